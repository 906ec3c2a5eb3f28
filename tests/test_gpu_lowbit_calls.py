"""Calls of the low-bit operators that their description allows: rows at any
8-byte boundary, pages shared by sessions, contexts that end inside a page,
queries that are not finite, prompts replayed from a graph."""
import kv8_exact as ex
import kv8_ref as ref
import numpy as np
import pytest
import torch
from test_gpu_kv8 import Rig, bits, dev
from test_gpu_kv8_exact import Held
from test_gpu_w4 import Linear, check, quantize

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu


def padded(rows, stride, at):
    """rows [n][heads][d] (bits) in a buffer with `stride` elements between rows, from element `at` on."""
    n, w = rows.shape[0], rows.shape[1] * rows.shape[2]
    buf = torch.full((n * stride + at,), 0x7FC0, dtype=torch.int16, device="cuda")
    view = torch.as_strided(buf, (n, w), (stride, 1), at)
    view.copy_(bits(rows).view(n, w))
    return buf, view


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 7, 50])
def test_rows_at_any_eight_byte_boundary(d, new):
    with Rig(2, 160, nq=6, nkv=2, d=d) as r:
        n = 2 * (90 + new)
        k, v, q = r.rows(n), r.rows(n), r.rows(2 * new, 6)
        start = dev(np.array([0, n // 2, n], np.int32))
        (kb, kv), (vb, vv), (qb, qv) = padded(k[0], 2 * d + 4, 4), padded(v[0], 2 * d + 12, 12), padded(q[0], 6 * d + 20, 4)
        qtts.qtts_kv8_append(r.c, 0, 2, n, n // 2, start, dev(np.zeros(2, np.int32)), r.bt, r.stride, kv, 2 * d + 4, vv,
                             2 * d + 12)
        for b in range(2):
            r.ref.append(r.tables[b], 0, k[1][b * n // 2:(b + 1) * n // 2], v[1][b * n // 2:(b + 1) * n // 2])
        r.check_cache([n // 2] * 2)
        out = torch.full((2 * new * (6 * d + 28) + 4,), 7.0, dtype=torch.bfloat16, device="cuda")
        view = torch.as_strided(out, (2 * new, 6 * d), (6 * d + 28, 1), 4)
        starts = np.array([0, new, 2 * new])
        qtts.qtts_kv8_attention(r.c, 0, 2, 2 * new, new, dev(starts.astype(np.int32)), dev(np.array([90, 90], np.int32)),
                                r.bt, r.stride, qv, 6 * d + 20, 0.1, view, 6 * d + 28, r.work)
        got = view.double().cpu().numpy().reshape(2 * new, 6, d)
        r.check_out(got, starts, [90, 90], [new, new], q[1], 0.1)
        view.fill_(7.0)
        assert bool((out == 7.0).all()) and r.status() == (0, 0)


@pytest.mark.parametrize("new", [1, 8, 40])
def test_sessions_that_share_the_pages_of_a_prefix(new):
    """Three sessions behind the same 64 tokens, then tokens of their own; the mean of marked pages."""
    nq, nkv, d, pages = 4, 2, 64, 4 + 3 * 4
    bt = np.array([[0, 1, 2, 3, 4 + 4 * b, 5 + 4 * b, 6 + 4 * b, 7 + 4 * b] for b in range(3)], np.int32)
    c = qtts.qtts_kv8_create(qtts.Kv8Config(1, nq, nkv, d, 0.0, 16, 3, 128, pages))
    try:
        work = torch.zeros(qtts.qtts_kv8_workspace_bytes(c), dtype=torch.uint8, device="cuda")
        rng, w, table = np.random.default_rng(3), nkv * d, dev(bt)
        v = ex.marks(128, nkv, d)
        k = bits(ref.bf16(rng.standard_normal((128, nkv, d)))[0])
        vb = bits(ref.bf16(v)[0])
        qtts.qtts_kv8_append(c, 0, 1, 64, 64, dev(np.array([0, 64], np.int32)), dev(np.zeros(1, np.int32)), table, 8, k, w,
                             vb, w)
        own = [64 - 9 * b for b in range(3)]
        start = np.concatenate(([0], np.cumsum(own))).astype(np.int32)
        rows = np.concatenate([np.arange(64, 64 + n) for n in own])
        qtts.qtts_kv8_append(c, 0, 3, int(start[-1]), 64, dev(start), dev(np.full(3, 64, np.int32)), table, 8,
                             k[torch.from_numpy(rows)].contiguous(), w, vb[torch.from_numpy(rows)].contiguous(), w)
        lens = [64 + n - new for n in own]
        q = bits(ref.bf16(rng.standard_normal((3 * new, nq, d)))[0])
        out = torch.zeros(3 * new, nq, d, dtype=torch.bfloat16, device="cuda")
        qtts.qtts_kv8_attention(c, 0, 3, 3 * new, new, dev((np.arange(4) * new).astype(np.int32)),
                                dev(np.array(lens, np.int32)), table, 8, q, nq * d, 0.0, out, nq * d, work)
        got = out.double().cpu().numpy()
        for b in range(3):
            want = np.repeat(ex.mean_of_marks(lens[b] + np.arange(new), nkv, d), nq // nkv, 1)
            assert np.all(np.abs(got[b * new:(b + 1) * new] - want) <= ex.mean_bound(want))
        assert qtts.qtts_kv8_status(c) == (0, 0)
    finally:
        qtts.qtts_kv8_destroy(c)


@pytest.mark.parametrize("context", [1, 17, 50, 200])
def test_contexts_that_end_inside_a_page(context):
    """The last position of max_context is used, the next one is refused on the device."""
    pages = -(-context // 16)
    with Rig(1, 16, nq=2, nkv=1, d=64) as r:
        qtts.qtts_kv8_destroy(r.c)
        r.c = qtts.qtts_kv8_create(qtts.Kv8Config(1, 2, 1, 64, 1e6, 16, 1, context, pages))
        r.ref, r.tables, r.stride, r.cap = ref.Cache(pages, 1, 64, 1e6), np.arange(pages, dtype=np.int32)[None], pages, context
        r.bt = dev(r.tables)
        r.append([0], [context])
        r.check_cache([context])
        for new in sorted({1, min(context, 17), context}):
            r.attend([context - new], [new])
        assert r.status() == (0, 0)
        past = dev(np.array([context], np.int32))
        x = bits(r.rows(1)[0])
        qtts.qtts_kv8_append(r.c, 0, 1, 1, 1, None, past, r.bt, r.stride, x, 64, x, 64)
        assert r.status()[1] == qtts.QTTS_DEV_BAD_SESSION
        r.check_cache([context])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 30])
def test_the_farthest_positions(d, new):
    """The last tokens of a context of 262144, behind one page of zeros that stands in every earlier place of the
    table: K read back, and attention with sharp scores, whose rows see each other's rotations only."""
    far, pages = 262144 - 48, 16384
    c = qtts.qtts_kv8_create(qtts.Kv8Config(1, 2, 1, d, 1e6, 16, 1, 262144, 4))
    try:
        table = np.zeros((1, pages), np.int32)
        table[0, -3:] = [1, 2, 3]
        bt, one = dev(table), lambda *a: dev(np.array(a, np.int32))
        z = torch.zeros(16, d, dtype=torch.int16, device="cuda")
        qtts.qtts_kv8_append(c, 0, 1, 16, 16, one(0, 16), one(0), bt, pages, z, d, z, d)
        rng = np.random.default_rng(d)
        (kb, k), (vb, v), (qb, q) = (ref.bf16(rng.standard_normal((m, h, d))) for m, h in ((48, 1), (48, 1), (new, 2)))
        qtts.qtts_kv8_append(c, 0, 1, 48, 48, one(0, 48), one(far), bt, pages, bits(kb), d, bits(vb), d)
        want = ref.Cache(3, 1, d, 1e6)
        rotated = ref.rotate(k, far + np.arange(48), 1e6)
        for p in range(3):  # as three pages of rotated rows
            want.theta = 0.0
            want.append([p], 0, rotated[16 * p:16 * p + 16], v[16 * p:16 * p + 16])
        wk, wv, ks, vs = want.values(np.arange(3), 48)
        back = [torch.zeros(48, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        qtts.qtts_kv8_read(c, 0, 1, 48, 48, one(0, 48), one(far), bt, pages, *back)
        for got, x, step in zip(back, (wk, wv), (ks, vs)):
            off = np.abs(got.double().cpu().numpy() - x)
            near = off <= 2.0 ** -8 * np.abs(x)
            assert np.all(near | (off <= 1.01 * step + 2.0 ** -8 * np.abs(x))) and np.sum(~near) <= 1 + 1e-3 * near.size
        work = torch.zeros(qtts.qtts_kv8_workspace_bytes(c), dtype=torch.uint8, device="cuda")
        out = torch.zeros(new, 2, d, dtype=torch.bfloat16, device="cuda")
        lens = 262144 - new
        qtts.qtts_kv8_attention(c, 0, 1, new, new, one(0, new), one(lens), bt, pages, bits(qb), 2 * d, 2.0, out, 2 * d, work)
        got = out.double().cpu().numpy()
        qr = ref.rotate(q, lens + np.arange(new), 1e6)
        for i in range(new):
            seen = 48 - new + i + 1
            for h in range(2):
                x = 2.0 * wk[:seen, 0] @ qr[i, h]
                top = max(x.max(), 0.0)
                p = np.exp(x - top)
                l = p.sum() + far * np.exp(-top)
                res = p @ wv[:seen, 0] / l
                # a score is off by at most: queries in half 2^-11, fp32 sums 2^-20, a code a step off in two dims
                e = 2.0 * (np.abs(wk[:seen, 0]) @ np.abs(qr[i, h]) * (2.0 ** -11 + 2.0 ** -20)
                           + 2 * np.abs(qr[i, h]).max() * ks[:seen, 0, 0])
                tol = 2.0 ** -8 * np.abs(res) + np.expm1(2 * e.max()) * np.abs(res) \
                    + (np.expm1(e) * p) @ np.abs(wv[:seen, 0]) / l + 2.0 ** -10 * (p @ np.abs(wv[:seen, 0])) / l \
                    + vs.max() * p.max() / l
                assert np.all(np.abs(got[i, h] - res) <= tol), (i, h)
        assert qtts.qtts_kv8_status(c) == (0, 0)
    finally:
        qtts.qtts_kv8_destroy(c)


@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_a_query_that_is_not_finite_spoils_its_own_row_and_head(new, bad):
    n = 300
    rng = np.random.default_rng(5)
    k = ex.integers(rng, n, 2, 64, ex.steps(rng, n, 2, -7, -7))
    v = ex.integers(rng, n, 2, 64, ex.steps(rng, n, 2, -7, -7))
    qb, q = ref.bf16(rng.standard_normal((new, 4, 64)))
    qb = qb.copy()
    qb[new // 2, 1, 9] = bad
    with Held([n], 4, 2, 64, [k], [v]) as c:
        got, _ = c.attend(qb, [n - new], [new], 0.125)
    want, tol = ex.attention(q, k, v, n - new, 0.125)
    assert np.isnan(got[new // 2, 1]).all()
    keep = np.ones((new, 4), bool)
    keep[new // 2, 1] = False
    assert np.all(np.abs(got - want)[keep] <= tol[keep])


def test_prompts_of_a_layer_replayed_from_a_graph():
    """A chunk of two prompts through a layer's attention block: products of 33 to 64 rows, append, attention of many
    rows; replayed for the next chunk with lengths advanced on the device."""
    hidden, nq, nkv, d, new = 256, 32, 8, 64, 30
    wide = (nq + 2 * nkv) * d
    rng = np.random.default_rng(8)
    with Rig(2, 160, nq=nq, nkv=nkv, d=d) as r, Linear(wide, hidden, 64) as qkv, Linear(hidden, nq * d, 64) as proj:
        mats = []
        for L in (qkv, proj):
            wb, w = ref.bf16(rng.standard_normal((L.N, L.K)) * L.K ** -0.5)
            qtts.qtts_w4_quantize(L.w, wb)
            mats.append(quantize(w, 64))
        lens = [0, 21]
        r.append([0, 0], [0, 21])
        x = torch.zeros(2 * new, hidden, dtype=torch.int16, device="cuda")
        rows = torch.zeros(2 * new, wide, dtype=torch.bfloat16, device="cuda")
        att = torch.zeros(2 * new, nq * d, dtype=torch.bfloat16, device="cuda")
        y = torch.zeros(2 * new, hidden, device="cuda")
        kv_len, start = dev(np.array(lens, np.int32)), dev(np.array([0, new, 2 * new], np.int32))
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            qtts.qtts_w4_linear(qkv.w, 2 * new, x, hidden, rows, wide, qtts.QTTS_DTYPE_BF16, s)
            qtts.qtts_kv8_append(r.c, 0, 2, 2 * new, new, start, kv_len, r.bt, r.stride, rows[:, nq * d:], wide,
                                 rows[:, (nq + nkv) * d:], wide, s)
            qtts.qtts_kv8_attention(r.c, 0, 2, 2 * new, new, start, kv_len, r.bt, r.stride, rows, wide, d ** -0.5, att,
                                    nq * d, r.work, s)
            qtts.qtts_w4_linear(proj.w, 2 * new, att, nq * d, y, hidden, qtts.QTTS_DTYPE_F32, s)
            kv_len.add_(new)
        for i in range(4):
            xb, xv = ref.bf16(rng.standard_normal((2 * new, hidden)))
            x.copy_(bits(xb))
            g.replay()
            torch.cuda.synchronize()
            fused = rows.double().cpu().numpy()
            check(fused, xv, mats[0][0], mats[0][2], 64, False)
            fused = fused.reshape(2 * new, nq + 2 * nkv, d)
            at = [n + i * new for n in lens]
            for b in range(2):
                p = slice(b * new, (b + 1) * new)
                r.ref.append(r.tables[b], at[b], fused[p, nq:nq + nkv], fused[p, nq + nkv:])
            got = att.double().cpu().numpy()
            r.check_out(got.reshape(2 * new, nq, d), np.array([0, new, 2 * new]), at, [new] * 2, fused[:, :nq], d ** -0.5)
            check(y.double().cpu().numpy(), got, mats[1][0], mats[1][2], 64, True)
        r.check_cache([n + 4 * new for n in lens])
        assert r.status() == (0, 0)
