"""Products with 4-bit weights on the GPU against their definition in 64 bits."""
import numpy as np
import pytest
import torch
from kv8_ref import bf16

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu


def bits(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to("cuda")


def quantize(w, group):
    """w float64 [N][K] of bf16 values: codes int8 and scales (bits, values), in binary32."""
    g = w.astype(np.float32).reshape(w.shape[0], -1, group)
    sb, s = bf16(np.abs(g).max(-1) / np.float32(7))
    s32 = s.astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s32[..., None] > 0, np.rint(g / s32[..., None]), 0)
    return np.clip(q, -7, 7).astype(np.int8).reshape(w.shape), sb, s


class Linear:
    def __init__(self, N, K, group):
        self.N, self.K, self.group = N, K, group
        self.w = qtts.qtts_w4_create(N, K, group)

    def __enter__(self):
        return self

    def __exit__(self, *e):
        qtts.qtts_w4_destroy(self.w)

    def export(self):
        q = np.zeros((self.N, self.K), np.int8)
        s = np.zeros((self.N, self.K // self.group), np.uint16)
        qtts.qtts_w4_export(self.w, q, s)
        return q, s


def check(y, x, q, s, group, f32):
    """fp32 sums of exact products: each of the at most K + 2 K / 32 + 80
    additions and scale products rounds by 2^-24 (the tensor core's own sums
    within one MMA are cut, not rounded: 2^-23) of a running sum that is at
    most the sum of magnitudes; then the result's own rounding, 2^-8 for bf16."""
    wide = q.astype(np.float64) * np.repeat(s, group, 1)
    want = x @ wide.T
    mag = np.abs(x) @ np.abs(wide).T
    steps = x.shape[1] / 16 * 2 + 2 * x.shape[1] / 32 + 80  # one MMA sums 16 products at once
    tol = mag * steps * 2.0 ** -23 + (0 if f32 else 2.0 ** -8) * np.abs(want) + 1e-37
    assert np.all(np.abs(y - want) <= tol), np.max(np.abs(y - want) / (tol + 1e-300))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 1), (17, 3), (40, 5), (129, 7), (1000, 9), (2048, 16), (333, 49)])
@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 32, 33, 64])
def test_products(M, N, K, group):
    K *= group
    rng = np.random.default_rng(N * 1000 + K + M)
    w = rng.standard_normal((N, K)) * 0.02
    w[N // 2] = 0  # a row of zeros
    wb, w = bf16(w)
    q, sb, s = quantize(w, group)
    xb, x = bf16(rng.standard_normal((M, K)))
    with Linear(N, K, group) as L:
        qtts.qtts_w4_quantize(L.w, wb)
        gq, gs = L.export()
        assert np.array_equal(gq, q) and np.array_equal(gs, sb)
        for f32 in (0, 1):
            y = torch.full((M + 1, N + 3), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
            qtts.qtts_w4_linear(L.w, M, bits(xb), K, y, N + 3, qtts.QTTS_DTYPE_F32 if f32 else qtts.QTTS_DTYPE_BF16)
            y = y.double().cpu().numpy()
            assert np.all(y[M] == 7.0) and np.all(y[:, N:] == 7.0)
            check(y[:M, :N], x, q, s, group, f32)


def test_given_codes_from_device_and_strided_rows():
    rng = np.random.default_rng(5)
    N, K, group, M = 200, 320, 64, 5
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    sb, s = bf16(np.exp(rng.standard_normal((N, K // group)) * 3))
    xb, x = bf16(rng.standard_normal((M, K + 32)))
    with Linear(N, K, group) as L:
        qtts.qtts_w4_load(L.w, torch.from_numpy(q).cuda(), bits(sb))
        assert all(np.array_equal(a, b) for a, b in zip(L.export(), (q, sb)))
        y = torch.zeros(M, N, device="cuda")
        qtts.qtts_w4_linear(L.w, M, bits(xb)[:, 16:], K + 32, y, N, qtts.QTTS_DTYPE_F32)
        check(y.double().cpu().numpy(), x[:, 16:16 + K], q, s, group, True)
        q[3, 4] = 8
        with pytest.raises(qtts.QttsError) as e:
            qtts.qtts_w4_load(L.w, q, sb)
        assert e.value.code == qtts.QTTS_E_INVALID
        with pytest.raises(qtts.QttsError) as e:  # nothing is loaded after a refused load
            qtts.qtts_w4_linear(L.w, M, bits(xb), K + 32, y, N, qtts.QTTS_DTYPE_F32)
        assert e.value.code == qtts.QTTS_E_STATE


def test_non_finite_values_stay_in_their_row_and_group():
    rng = np.random.default_rng(6)
    wb, w = bf16(rng.standard_normal((40, 256)))
    wb = wb.copy()
    wb[7, 200] = 0x7F80
    xb, x = bf16(rng.standard_normal((3, 256)))
    xb = xb.copy()
    xb[1, 5] = 0x7FC0
    with Linear(40, 256, 128) as L:
        qtts.qtts_w4_quantize(L.w, wb)
        y = torch.zeros(3, 40, device="cuda")
        qtts.qtts_w4_linear(L.w, 3, bits(xb), 256, y, 40, qtts.QTTS_DTYPE_F32)
        y = y.cpu().numpy()
        assert np.isnan(y[1]).all() and np.isnan(y[:, 7]).all()
        assert np.isfinite(np.delete(y[[0, 2]], 7, 1)).all()


def test_refusals():
    with Linear(64, 128, 64) as L:
        x = torch.zeros(65, 136, dtype=torch.int16, device="cuda")
        y = torch.zeros(65, 64, device="cuda")
        f32 = qtts.QTTS_DTYPE_F32

        def code(*a):
            with pytest.raises(qtts.QttsError) as e:
                qtts.qtts_w4_linear(L.w, *a)
            return e.value.code

        assert code(1, x, 136, y, 64, f32) == qtts.QTTS_E_STATE
        qtts.qtts_w4_quantize(L.w, np.zeros((64, 128), np.uint16))
        assert code(65, x, 136, y, 64, f32) == qtts.QTTS_E_BATCH
        assert code(-1, x, 136, y, 64, f32) == qtts.QTTS_E_BATCH
        assert code(1, x, 136, y, 64, 2) == qtts.QTTS_E_INVALID
        assert code(1, None, 136, y, 64, f32) == qtts.QTTS_E_INVALID
        assert code(1, x, 136, None, 64, f32) == qtts.QTTS_E_INVALID
        assert code(1, x, 120, y, 64, f32) == qtts.QTTS_E_INVALID
        assert code(1, x, 132, y, 64, f32) == qtts.QTTS_E_INVALID
        assert code(1, x[:, 4:], 136, y, 64, f32) == qtts.QTTS_E_INVALID
        assert code(1, x, 136, y, 63, f32) == qtts.QTTS_E_INVALID
        assert qtts.qtts_w4_linear(L.w, 0, None, 136, None, 64, f32) == 0


@pytest.mark.parametrize("M,N,K,group", [(64, 40, 20000, 32), (33, 5000, 8192, 128), (8, 20, 60000 // 64 * 64, 64)])
def test_more_activations_than_shared_memory_holds(M, N, K, group):
    rng = np.random.default_rng(K)
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    sb, s = bf16(np.exp(rng.standard_normal((N, K // group))))
    xb, x = bf16(rng.standard_normal((M, K)))
    with Linear(N, K, group) as L:
        qtts.qtts_w4_load(L.w, q, sb)
        y = torch.zeros(M, N, device="cuda")
        qtts.qtts_w4_linear(L.w, M, bits(xb), K, y, N, qtts.QTTS_DTYPE_F32)
        check(y.double().cpu().numpy(), x, q, s, group, True)


def test_back_to_back_products_wait_for_their_input():
    """Products that start early read their activations only when the one before has written them."""
    rng = np.random.default_rng(9)
    N = 512
    wb, w = bf16(rng.standard_normal((N, N)) * N ** -0.5)
    q, sb, s = quantize(w, 64)
    xb, x = bf16(rng.standard_normal((4, N)))
    with Linear(N, N, 64) as L:
        qtts.qtts_w4_quantize(L.w, bits(wb))
        a, b = bits(xb), torch.zeros(4, N, dtype=torch.bfloat16, device="cuda")
        c = torch.zeros_like(b)
        for _ in range(50):
            b.fill_(float("nan"))
            qtts.qtts_w4_linear(L.w, 4, a, N, b, N, qtts.QTTS_DTYPE_BF16)
            qtts.qtts_w4_linear(L.w, 4, b, N, c, N, qtts.QTTS_DTYPE_BF16)
            qtts.qtts_w4_linear(L.w, 4, c, N, b, N, qtts.QTTS_DTYPE_BF16)
        check(c.double().cpu().numpy(), bf16_twice(L, a, N), q, s, 64, False)


def bf16_twice(L, a, N):
    y = torch.zeros(4, N, dtype=torch.bfloat16, device="cuda")
    qtts.qtts_w4_linear(L.w, 4, a, N, y, N, qtts.QTTS_DTYPE_BF16)
    torch.cuda.synchronize()
    return y.double().cpu().numpy()


@pytest.mark.parametrize("M,N,K,group", [
    (33, 3700, 32, 32), (64, 3700, 32 * 45, 32), (40, 20001, 32 * 6, 32),     # k tiles that end half full
    (64, 3700, 64, 64), (48, 4999, 64 * 33, 64), (64, 20001, 64 * 5, 64),
    (33, 3700, 128, 128), (64, 4999, 128 * 17, 128), (64, 20001, 128 * 3, 128),
    (12, 6001, 64 * 20, 64), (16, 30001, 64 * 3, 64), (24, 6001, 128 * 9, 128), (32, 12289, 32 * 33, 32)])
def test_many_rows_of_weights(M, N, K, group):
    """The variants of large layers, with strided rows and rows behind the last left as they were."""
    rng = np.random.default_rng(N + K + M)
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    sb, s = bf16(np.exp(rng.standard_normal((N, K // group))))
    xb, x = bf16(rng.standard_normal((M + 1, K + 8)))
    xb = xb.copy()
    xb[:, K:] = 0x7FC0  # between the rows, and behind the last: not read
    xb[M] = 0x7FC0
    with Linear(N, K, group) as L:
        qtts.qtts_w4_load(L.w, q, sb)
        d = bits(xb)
        for f32 in (0, 1):
            y = torch.full((M + 1, N + 3), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
            for _ in range(2):
                qtts.qtts_w4_linear(L.w, M, d, K + 8, y, N + 3, qtts.QTTS_DTYPE_F32 if f32 else qtts.QTTS_DTYPE_BF16)
            y = y.double().cpu().numpy()
            assert (y[M] == 7).all() and (y[:, N:] == 7).all()
            check(y[:M, :N], x[:M, :K], q, s, group, f32)


def test_non_finite_values_of_many_rows_stay_in_their_row_and_group():
    rng = np.random.default_rng(16)
    N, K = 3700, 256
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    sb, _ = bf16(np.exp(rng.standard_normal((N, K // 64))))
    sb = sb.copy()
    sb[133, 2] = 0x7FC0
    xb, _ = bf16(rng.standard_normal((50, K)))
    xb = xb.copy()
    xb[17, 5] = 0x7FC0
    with Linear(N, K, 64) as L:
        qtts.qtts_w4_load(L.w, q, sb)
        y = torch.zeros(50, N, device="cuda")
        qtts.qtts_w4_linear(L.w, 50, bits(xb), K, y, N, qtts.QTTS_DTYPE_F32)
        y = y.cpu().numpy()
        assert np.isnan(y[17]).all() and np.isnan(y[:, 133]).all()
        assert np.isfinite(np.delete(np.delete(y, 17, 0), 133, 1)).all()


def test_large_products_on_two_streams_and_in_a_graph():
    rng = np.random.default_rng(17)
    N, K = 5000, 512
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    sb, s = bf16(np.exp(rng.standard_normal((N, K // 128))))
    xb, x = bf16(rng.standard_normal((64, K)))
    with Linear(N, K, 128) as L:
        qtts.qtts_w4_load(L.w, q, sb)
        d, f32 = bits(xb), qtts.QTTS_DTYPE_F32
        y = [torch.zeros(64, N, device="cuda") for _ in range(3)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(10):
            for out, st in zip(y, streams):
                qtts.qtts_w4_linear(L.w, 64, d, K, out, N, f32, st.cuda_stream)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                qtts.qtts_w4_linear(L.w, 64, d, K, y[2], N, f32, torch.cuda.current_stream().cuda_stream)
        g.replay()
        torch.cuda.synchronize()
        check(y[0].double().cpu().numpy(), x, q, s, 128, True)
        assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
