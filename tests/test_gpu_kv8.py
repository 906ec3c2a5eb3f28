"""The 8-bit paged K/V cache on the GPU (append, read-back, attention) against
its definition in 64 bits (kv8_ref)."""
import math

import kv8_ref as ref
import numpy as np
import pytest
import torch

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu

PAGE = 16
THETA = 1e6


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def bits(a):
    return dev(a.view(np.int16))


class Rig:
    """A cache on the GPU and its definition beside it, with shuffled pages."""

    def __init__(self, B, cap, nq=4, nkv=2, d=128, theta=THETA, layers=1, layer=0, seed=0, spare=0):
        self.rng = np.random.default_rng(seed)
        per = -(-cap // PAGE)
        self.B, self.nq, self.nkv, self.d, self.theta, self.layer, self.cap = B, nq, nkv, d, theta, layer, cap
        self.c = qtts.qtts_kv8_create(qtts.Kv8Config(layers, nq, nkv, d, theta, PAGE, B, per * PAGE, B * per + spare))
        ids = np.zeros(B * per, np.int32)
        qtts.qtts_kv8_alloc_pages(self.c, ids)
        self.rng.shuffle(ids)
        self.tables = ids.reshape(B, per)
        self.bt, self.stride = dev(self.tables), per
        self.ref = ref.Cache(B * per + spare, nkv, d, theta)
        self.work = torch.zeros(qtts.qtts_kv8_workspace_bytes(self.c), dtype=torch.uint8, device="cuda")

    def close(self):
        qtts.qtts_kv8_destroy(self.c)

    def __enter__(self):
        return self

    def __exit__(self, *e):
        self.close()

    def rows(self, n, heads=None, size=1.0):
        return ref.bf16(self.rng.standard_normal((n, heads or self.nkv, self.d)) * size)

    def append(self, lens, new, k=None, v=None, stream=None, one=False):
        """Appends new[b] random rows behind lens[b] tokens, on both sides."""
        start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        k, v = k or self.rows(start[-1]), v or self.rows(start[-1])
        w = self.nkv * self.d
        keep = dev(start), dev(np.asarray(lens, np.int32)), bits(k[0]), bits(v[0])
        qtts.qtts_kv8_append(self.c, self.layer, self.B, int(start[-1]), max(max(new), 1), None if one else keep[0],
                             keep[1], self.bt, self.stride, keep[2], w, keep[3], w, stream)
        for b in range(self.B):
            if lens[b] >= 0:
                s = slice(start[b], start[b + 1])
                self.ref.append(self.tables[b], lens[b], k[1][s], v[1][s])
        torch.cuda.synchronize()

    def read(self, lens, new):
        start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        k = torch.zeros(int(start[-1]), self.nkv, self.d, dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        qtts.qtts_kv8_read(self.c, self.layer, self.B, int(start[-1]), max(new), dev(start),
                           dev(np.asarray(lens, np.int32)), self.bt, self.stride, k, v)
        torch.cuda.synchronize()
        return k.double().cpu().numpy(), v.double().cpu().numpy(), start

    def check_cache(self, totals):
        """Every position of every session. A value is the definition's to the
        read-back's bf16 rounding, 2^-8 of it; a code whose exact quotient lies
        within the binary32 products' error of a rounding border (2^-22 * 127
        of 1, 6e-5 of all) may be one step off, and one rescaled later once more."""
        k, v, start = self.read([0] * self.B, totals)
        for b, n in enumerate(totals):
            want = self.ref.values(self.tables[b], n)
            for got, x, step in ((k, want[0], want[2]), (v, want[1], want[3])):
                g = got[start[b]:start[b + 1]]
                off = np.abs(g - x)
                near = off <= 2.0 ** -8 * np.abs(x)
                assert np.all(near | (off <= 2.01 * step + 2.0 ** -8 * np.abs(x))), off.max()
                assert np.sum(~near) <= 1 + 1e-3 * near.size

    def attend(self, lens, new, scale=None, one=False, q=None, stream=None, pad=0, check=True):
        start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        n = int(start[-1])
        scale = scale or 1 / math.sqrt(self.d)
        q = q or self.rows(n, self.nq)
        out = torch.full((n + pad, self.nq, self.d), 7.0, dtype=torch.bfloat16, device="cuda")
        qd = torch.cat((bits(q[0]), torch.zeros(pad, self.nq, self.d, dtype=torch.int16, device="cuda")))
        w = self.nq * self.d
        keep = dev(start), dev(np.asarray(lens, np.int32))
        qtts.qtts_kv8_attention(self.c, self.layer, self.B, n + pad, max(max(new), 1), None if one else keep[0],
                                keep[1], self.bt, self.stride, qd, w, scale, out, w, self.work, stream)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        assert np.all(got[n:] == 7.0)
        if check:
            self.check_out(got, start, lens, new, q[1], scale)
        return out

    def check_out(self, got, start, lens, new, q, scale):
        """|out - exact| is at most: the result's rounding to bf16, 2^-8 |out|;
        the weights' rounding to half, 2^-11, of at most max|v|; and scores off
        by e move weights by a factor of at most exp(2 e), out by 2.2 e max|v|
        for small e. e: queries rounded to half (2^-11 of each product), a
        K code a step off at a rounding border in two dims of a token, and the
        fp32 arithmetic of score and exponential (2^-20 of the score's terms);
        V codes a step off count as their weight, at most one step."""
        for b in range(self.B):
            if lens[b] < 0 or not new[b]:
                continue
            k, v, ks, vs = self.ref.values(self.tables[b], lens[b] + new[b])
            want, qr = ref.attention(q[start[b]:start[b + 1]], k, v, lens[b], scale, self.theta)
            g = got[start[b]:start[b + 1]]
            group = self.nq // self.nkv
            for h in range(self.nq):
                kh, vh = k[:, h // group], v[:, h // group]
                terms = (np.abs(kh) @ np.abs(qr[:, h]).T).max() * abs(scale)
                e = terms * (2.0 ** -11 + 2.0 ** -20) + 2 * abs(scale) * np.abs(qr[:, h]).max() * ks[:, h // group].max()
                tol = 2.0 ** -8 * np.abs(want[:, h]) + (2.2 * e + 2.0 ** -10) * np.abs(vh).max() + 1e-30
                assert np.all(np.abs(g[:, h] - want[:, h]) <= tol), (b, h, np.max(np.abs(g[:, h] - want[:, h]) - tol))

    def status(self):
        return qtts.qtts_kv8_status(self.c, raise_on_error=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [[1, 1, 1], [5, 16, 33], [0, 47, 1], [100, 3, 64]])
def test_append_from_empty_and_onto_partial_pages(d, new):
    with Rig(3, 200, d=d) as r:
        r.append([0, 0, 0], new)
        r.check_cache(new)
        more = [7, 1, 20]
        r.append(new, more)
        r.check_cache([a + b for a, b in zip(new, more)])
        assert r.status() == (0, 0)


def test_append_token_by_token_grows_the_scale_and_restarts_it_on_the_next_page():
    with Rig(2, 64, nkv=3, nq=3) as r:
        for i in range(37):
            size = 2.0 ** (i % 5) if i < 20 else 1e-3  # growth inside a page, and a small page after large ones
            r.append([i, i], [1, 1], r.rows(2, size=size), r.rows(2, size=size), one=True)
        r.check_cache([37, 37])


def test_append_of_zeros_and_of_tiny_values_reads_as_zeros():
    with Rig(1, 32) as r:
        z = ref.bf16(np.zeros((5, 2, 128)))
        t = ref.bf16(np.full((5, 2, 128), 1e-32))
        r.append([0], [5], z, z)
        r.append([5], [5], t, t)
        k, v, _ = r.read([0], [10])
        assert not k.any() and not v.any()
        r.append([10], [6])
        r.check_cache([16])


def test_append_after_a_rollback_and_a_reused_page():
    with Rig(1, 48) as r:
        r.append([0], [30], r.rows(30, size=50.0), r.rows(30, size=50.0))
        r.append([18], [2])  # the last 12 tokens were rejected; their scale still counts
        r.check_cache([20])
        r.append([0], [3], r.rows(3, size=0.1), r.rows(3, size=0.1))  # the pages are given to another session
        r.check_cache([3])


@pytest.mark.parametrize("bad", [np.inf, np.nan])
def test_a_non_finite_value_shows_in_its_own_block_only(bad):
    with Rig(2, 40) as r:
        k, v = r.rows(40), r.rows(40)
        kb = k[0].copy()
        kb[3, 0, 17] = ref.bf16(np.array([bad]))[0][0]
        w = r.nkv * r.d
        start, zero = dev(np.array([0, 20, 40], np.int32)), dev(np.zeros(2, np.int32))
        qtts.qtts_kv8_append(r.c, 0, 2, 40, 20, start, zero, r.bt, r.stride, bits(kb), w, bits(v[0]), w)
        gk, gv, _ = r.read([0, 0], [20, 20])
        assert np.isnan(gk[:16, 0]).all() and np.isfinite(gk[16:]).all() and np.isfinite(gk[:, 1]).all()
        assert np.isfinite(gv).all()
        out = r.attend([19, 19], [1, 1], check=False).float().cpu().numpy()
        assert np.isnan(out[0, :2]).all() and np.isfinite(out[0, 2:]).all() and np.isfinite(out[1]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (2, 2), (4, 2), (8, 2), (8, 1), (10, 2), (16, 1), (24, 1), (32, 1)])
def test_single_tokens_over_ragged_contexts(d, nq, nkv):
    lens = [0, 1, 15, 16, 17, 127, 128, 300]
    with Rig(len(lens), 320, nq=nq, nkv=nkv, d=d) as r:
        r.append([0] * 8, [x + 1 for x in lens])
        r.attend(lens, [1] * 8, one=True)
        r.attend(lens, [1] * 8)
        assert r.status() == (0, 0)


@pytest.mark.parametrize("B,nq,nkv,top", [(300, 4, 2, 40), (300, 16, 2, 20), (150, 32, 2, 60), (40, 3, 3, 3), (1, 8, 8, 700)])
def test_many_short_sessions(B, nq, nkv, top):
    """More tiles than CTAs: a CTA goes through several, some of them shared with its neighbours."""
    with Rig(B, top + 1, nq=nq, nkv=nkv, d=64) as r:
        lens = [int(x) for x in r.rng.integers(0, top + 1, B)]
        r.append([0] * B, [x + 1 for x in lens])
        r.attend(lens, [1] * B, one=True)
        some = [int(x) for x in r.rng.integers(0, 2, B)]
        r.attend([x if s else -1 for x, s in zip(lens, some)], [1] * B)
        assert r.status() == (0, 0)


@pytest.mark.parametrize("n", [1023, 4000])
def test_one_long_session_is_split_and_joined(n):
    with Rig(1, n + 1, nq=4, nkv=2) as r:
        r.append([0], [n + 1])
        a = r.attend([n], [1], q=(q := r.rows(1, 4)))
        b = r.attend([n], [1], q=q, check=False)
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,nq,nkv", [(64, 4, 2), (128, 4, 2), (128, 3, 3), (128, 10, 2), (64, 17, 1), (128, 8, 1)])
@pytest.mark.parametrize("lens,new", [([0, 5, 40], [3, 2, 1]), ([0, 33, 7], [50, 1, 17]), ([100, 0, 31], [0, 130, 64]),
                                      ([0, 200, 16], [1, 40, 129])])
def test_chunks_of_rows_are_causal(d, nq, nkv, lens, new):
    with Rig(3, 260, nq=nq, nkv=nkv, d=d) as r:
        r.append([0, 0, 0], [a + b for a, b in zip(lens, new)])
        r.attend(lens, new, pad=5)
        assert r.status() == (0, 0)


@pytest.mark.parametrize("size,vsize", [(30.0, 1.0), (1.0, 1e30), (1.0, 1e-25), (1e-20, 1e-20), (300.0, 100.0)])
def test_scales_far_from_one(size, vsize):
    """Sharp softmaxes, and values whose products with a weight leave half's range."""
    with Rig(2, 100, nq=4, nkv=2, theta=0.0) as r:
        for lo, n in ((0, 60), (60, 38)):
            f = vsize * (1e-3 if lo else 1.0)  # pages of very different V scales
            r.append([lo, lo], [n, n], r.rows(2 * n, size=math.sqrt(size)), r.rows(2 * n, size=f))
        q = r.rows(2, 4, size=math.sqrt(size))
        out = r.attend([97, 97], [1, 1], q=q, check=False).double().cpu().numpy()
        r.check_out(out, np.array([0, 1, 2]), [97, 97], [1, 1], q[1], 1 / math.sqrt(128))


def test_layers_do_not_touch_each_other_and_no_rotation():
    with Rig(2, 64, theta=0.0, layers=3, layer=1) as r:
        r.append([0, 0], [20, 41])
        r.check_cache([20, 41])
        r.attend([19, 40], [1, 1])
        r.layer = 2
        k, v, _ = r.read([0, 0], [20, 41])
        assert not k.any() and not v.any()
        r.layer = 0
        k, v, _ = r.read([0, 0], [20, 41])
        assert not k.any() and not v.any()


def test_inactive_sessions_and_rows_behind_the_last_are_left():
    with Rig(4, 64) as r:
        r.append([0] * 4, [10, 20, 30, 40])
        r.append([10, -1, 30, 40], [1, 1, 0, 2])
        r.check_cache([11, 20, 30, 42])
        start = np.array([0, 1, 2, 2, 4], np.int32)
        out = torch.full((6, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        q = r.rows(6, 4)
        qtts.qtts_kv8_attention(r.c, 0, 4, 6, 2, dev(start), dev(np.array([10, -1, 30, 40], np.int32)), r.bt, r.stride,
                                bits(q[0]), 512, 0.1, out, 512, r.work)
        got = out.double().cpu().numpy()
        assert np.all(got[1] == 7.0) and np.all(got[4:] == 7.0)
        r.check_out(got, start, [10, -1, 30, 40], [1, 1, 0, 2], q[1], 0.1)
        assert r.status() == (0, 0)


def test_rows_as_slices_of_one_projection():
    """q, k and v as strided views of a fused projection's output, out into a wider buffer."""
    with Rig(2, 64, nq=4, nkv=2) as r:
        x, fused = ref.bf16(r.rng.standard_normal((30, 8, 128)))
        f = bits(x)
        lens, start, kv0 = [0, 0], dev(np.array([0, 12, 30], np.int32)), dev(np.zeros(2, np.int32))
        qtts.qtts_kv8_append(r.c, 0, 2, 30, 18, start, kv0, r.bt, r.stride, f[:, 4:6], 1024, f[:, 6:], 1024)
        for b, s in ((0, slice(0, 12)), (1, slice(12, 30))):
            r.ref.append(r.tables[b], 0, fused[s, 4:6], fused[s, 6:])
        r.check_cache([12, 18])
        out = torch.full((30, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        qtts.qtts_kv8_attention(r.c, 0, 2, 30, 18, start, kv0, r.bt, r.stride, f, 1024, 0.09, out[:, 1:], 768, r.work)
        got = out.double().cpu().numpy()
        assert np.all(got[:, 0] == 7.0) and np.all(got[:, 5] == 7.0)
        r.check_out(got[:, 1:5], np.array([0, 12, 30]), lens, [12, 18], fused[:, :4], 0.09)


def test_device_checks_report_and_spare_the_others():
    with Rig(2, 64) as r:
        r.append([0, 0], [20, 20])
        # a page outside the pool: not written
        bt = r.tables.copy()
        bt[0, 1] = 10 ** 6
        k = r.rows(2)
        w = r.nkv * r.d
        lens = dev(np.array([20, 20], np.int32))
        qtts.qtts_kv8_append(r.c, 0, 2, 2, 1, None, lens, dev(bt), r.stride, bits(k[0]), w, bits(k[0]), w)
        r.ref.append(r.tables[1], 20, k[1][1:], k[1][1:])
        assert r.status() == (qtts.QTTS_E_DEVICE, qtts.QTTS_DEV_BAD_PAGE)
        assert r.status() == (0, 0)
        r.check_cache([20, 21])
        # a session past its block table, one past row_start's promise
        qtts.qtts_kv8_append(r.c, 0, 2, 2, 1, None, dev(np.array([64, 2 ** 31 - 1], np.int32)), r.bt, r.stride,
                             bits(k[0]), w, bits(k[0]), w)
        assert r.status()[1] == qtts.QTTS_DEV_BAD_SESSION
        qtts.qtts_kv8_append(r.c, 0, 2, 2, 1, dev(np.array([0, 2, 1], np.int32)), lens, r.bt, r.stride, bits(k[0]), w,
                             bits(k[0]), w)
        assert r.status()[1] == qtts.QTTS_DEV_BAD_SESSION
        r.check_cache([20, 21])
        out = torch.full((2, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        q = r.rows(2, 4)
        qtts.qtts_kv8_attention(r.c, 0, 2, 2, 1, None, dev(np.array([64, 20], np.int32)), r.bt, r.stride, bits(q[0]),
                                512, 0.1, out, 512, r.work)
        assert r.status()[1] == qtts.QTTS_DEV_BAD_SESSION
        got = out.double().cpu().numpy()
        assert np.all(got[0] == 7.0)
        r.check_out(got, np.array([0, 1, 2]), [-1, 20], [1, 1], q[1], 0.1)


def test_append_and_attention_in_a_captured_graph_on_another_stream():
    """Two decode steps replayed from one graph, lengths advanced on the device between them."""
    with Rig(3, 64, nq=4, nkv=2) as r:
        lens = [5, 31, 17]
        r.append([0] * 3, lens)
        k, v, q = bits(r.rows(3)[0]), bits(r.rows(3)[0]), bits(r.rows(3, 4)[0])
        kv_len = dev(np.array(lens, np.int32))
        out = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qtts.qtts_kv8_append(r.c, 0, 3, 3, 1, None, kv_len, r.bt, r.stride, k, 256, v, 256, s)
            qtts.qtts_kv8_attention(r.c, 0, 3, 3, 1, None, kv_len, r.bt, r.stride, q, 512, 0.1, out, 512, r.work, s)
            kv_len.add_(1)
        for step in range(3):
            kk, vv, qq = r.rows(3), r.rows(3), r.rows(3, 4)
            k.copy_(bits(kk[0]))
            v.copy_(bits(vv[0]))
            q.copy_(bits(qq[0]))
            g.replay()
            torch.cuda.synchronize()
            at = [x + step for x in lens]
            for b in range(3):
                r.ref.append(r.tables[b], at[b], kk[1][b:b + 1], vv[1][b:b + 1])
            r.check_out(out.double().cpu().numpy(), np.arange(4), at, [1] * 3, qq[1], 0.1)
        assert r.status() == (0, 0)


@pytest.mark.parametrize("nq,nkv,d,lens,new", [
    (1, 1, 128, [7990], [64]),             # one tile, its key steps cut over many CTAs
    (2, 2, 64, [5000, 3], [70, 300]),      # and beside it tiles of another length
    (1, 1, 128, [3], [333]),               # a group of one: the queries come in two passes
    (5, 1, 128, [700], [128]),             # a group that does not divide 128
    (32, 1, 64, [100, 2000], [9, 40]),
    (64, 8, 64, [200], [1250]),            # enough tiles for 256 rows each
    (16, 8, 128, [50], [4900]),
    (48, 16, 64, [0, 9, 31], [600, 700, 500]),
])
def test_many_rows(nq, nkv, d, lens, new):
    with Rig(len(lens), max(a + b for a, b in zip(lens, new)), nq=nq, nkv=nkv, d=d) as r:
        r.append([0] * len(lens), [a + b for a, b in zip(lens, new)])
        a = r.attend(lens, new, q=(q := r.rows(sum(new), nq)), pad=3)
        b = r.attend(lens, new, q=q, pad=3, check=False)
        assert torch.equal(a, b) and r.status() == (0, 0)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [-0.1, 1e-30])
def test_odd_softmax_scales(new, scale):
    with Rig(1, 200, nq=4, nkv=2) as r:
        r.append([0], [150])
        r.attend([150 - new], [new], scale=scale)


@pytest.mark.parametrize("new", [12, 60])
def test_rows_before_a_nan_do_not_see_it(new):
    """The last page's first token is a NaN in K and V: only rows on that page may show it."""
    n = 80
    with Rig(1, 96, nq=2, nkv=2) as r:
        r.append([0], [n])
        k, v = r.rows(1), r.rows(1)
        k[0][0, 1, 5] = v[0][0, 0, 9] = 0x7FC0
        w = r.nkv * r.d
        one, q = dev(np.array([n], np.int32)), r.rows(new, 2)
        qtts.qtts_kv8_append(r.c, 0, 1, 1, 1, None, one, r.bt, r.stride, bits(k[0]), w, bits(v[0]), w)
        out = torch.zeros(new, 2, 128, dtype=torch.bfloat16, device="cuda")
        lens = n + 1 - new
        qtts.qtts_kv8_attention(r.c, 0, 1, new, new, dev(np.array([0, new], np.int32)), dev(np.array([lens], np.int32)),
                                r.bt, r.stride, bits(q[0]), 256, 0.1, out, 256, r.work)
        got = out.double().cpu().numpy()
        assert np.isnan(got[-1]).all() and np.isfinite(got[:-1]).all()
        r.check_out(got[:-1], np.array([0, new - 1]), [lens], [new - 1], q[1][:-1], 0.1)


def test_blocks_beyond_four_gigabytes():
    """A layer's blocks start, and a page's lie, more than 2^32 bytes into the pool."""
    pages, per = 140000, 8  # 8 kv heads x 4 KiB: 4.6 GB a layer
    c = qtts.qtts_kv8_create(qtts.Kv8Config(2, 8, 8, 128, THETA, PAGE, 2, per * PAGE, pages))
    try:
        ids = np.concatenate((np.arange(pages - per, pages), np.arange(per))).astype(np.int32).reshape(2, per)
        rng = np.random.default_rng(3)
        k, v, q = (ref.bf16(rng.standard_normal((200, 8, 128))) for _ in range(3))
        want = ref.Cache(16, 8, 128, THETA)
        start, zero, bt = dev(np.array([0, 100, 200], np.int32)), dev(np.zeros(2, np.int32)), dev(ids)
        work = torch.zeros(qtts.qtts_kv8_workspace_bytes(c), dtype=torch.uint8, device="cuda")
        for layer in (1, 0):
            qtts.qtts_kv8_append(c, layer, 2, 200, 100, start, zero, bt, per, bits(k[0]), 1024, bits(v[0]), 1024)
        for b in range(2):
            want.append(np.arange(8) + 8 * b, 0, k[1][100 * b:100 * b + 100], v[1][100 * b:100 * b + 100])
        r = Rig.__new__(Rig)
        r.B, r.nq, r.nkv, r.d, r.theta, r.ref, r.tables = 2, 8, 8, 128, THETA, want, np.arange(16).reshape(2, 8)
        lens = dev(np.array([99, 99], np.int32))
        for layer in (0, 1):
            out = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
            qtts.qtts_kv8_attention(c, layer, 2, 2, 1, None, lens, bt, per, bits(q[0]), 1024, 0.1, out, 1024, work)
            r.check_out(out.double().cpu().numpy(), np.arange(3), [99, 99], [1, 1], q[1][:2], 0.1)
            out = torch.zeros(200, 8, 128, dtype=torch.bfloat16, device="cuda")
            qtts.qtts_kv8_attention(c, layer, 2, 200, 100, start, zero, bt, per, bits(q[0]), 1024, 0.1, out, 1024, work)
            r.check_out(out.double().cpu().numpy(), np.array([0, 100, 200]), [0, 0], [100, 100], q[1], 0.1)
    finally:
        qtts.qtts_kv8_destroy(c)


def test_two_streams_with_a_workspace_each():
    with Rig(2, 2100, nq=4, nkv=2) as r:
        r.append([0, 0], [2100, 2100])
        lens = [dev(np.array(x, np.int32)) for x in ([2099, 2000], [1500, 1999])]
        qs = [r.rows(2, 4) for _ in range(2)]
        works = [torch.zeros_like(r.work) for _ in range(2)]
        outs = [torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        dq = [bits(q[0]) for q in qs]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(20):
            for i, s in enumerate(streams):
                qtts.qtts_kv8_attention(r.c, 0, 2, 2, 1, None, lens[i], r.bt, r.stride, dq[i], 512, 0.1, outs[i], 512,
                                        works[i], s)
        torch.cuda.synchronize()
        for i, at in enumerate(([2099, 2000], [1500, 1999])):
            r.check_out(outs[i].double().cpu().numpy(), np.arange(3), at, [1, 1], qs[i][1], 0.1)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_over_a_page_outside_the_pool_reports_it(new):
    with Rig(3, 128) as r:
        r.append([0] * 3, [100] * 3)
        bt = r.tables.copy()
        bt[1, 2] = -1
        bt[1, 4] = 2 ** 31 - 1
        q, lens = r.rows(3 * new, 4), [100 - new] * 3
        out = torch.zeros(3 * new, 4, 128, dtype=torch.bfloat16, device="cuda")
        start = np.arange(4) * new
        qtts.qtts_kv8_attention(r.c, 0, 3, 3 * new, new, dev(start.astype(np.int32)), dev(np.array(lens, np.int32)),
                                dev(bt), r.stride, bits(q[0]), 512, 0.1, out, 512, r.work)
        assert r.status() == (qtts.QTTS_E_DEVICE, qtts.QTTS_DEV_BAD_PAGE)
        r.check_out(out.double().cpu().numpy(), start, [lens[0], -1, lens[2]], [new] * 3, q[1], 0.1)
        r.attend(lens, [new] * 3)
        assert r.status() == (0, 0)


def test_the_largest_batch():
    with Rig(1024, 20, nq=2, nkv=1, d=64) as r:
        lens = [int(x) for x in r.rng.integers(0, 19, 1024)]
        r.append([0] * 1024, [x + 1 for x in lens])
        r.attend(lens, [1] * 1024, one=True)
        r.append([-1] * 1023 + [lens[-1] + 1], [0] * 1023 + [1])
        assert r.status() == (0, 0)


def test_sessions_that_share_rows_are_reported():
    with Rig(3, 128) as r:
        r.append([0] * 3, [100] * 3)
        q, lens = r.rows(40, 4), dev(np.array([60] * 3, np.int32))
        out = torch.zeros(40, 4, 128, dtype=torch.bfloat16, device="cuda")
        start = dev(np.array([0, 40, 0, 40], np.int32))
        qtts.qtts_kv8_attention(r.c, 0, 3, 40, 40, start, lens, dev(r.tables), r.stride, bits(q[0]), 512, 0.1, out, 512,
                                r.work)
        assert r.status() == (qtts.QTTS_E_DEVICE, qtts.QTTS_DEV_BAD_SESSION)
        r.attend([60] * 3, [40] * 3)
        assert r.status() == (0, 0)


@pytest.mark.parametrize("d,cap,lens,new", [(64, 40000, [1500], [8]), (128, 40000, [2100], [5]), (128, 14000, [900, 0, 1700], [8, 3, 6])])
def test_nine_to_sixteen_columns_of_tables_for_long_sessions(d, cap, lens, new):
    """Tiles cut over CTAs, 16 columns each: where the tables could hold long sessions."""
    with Rig(len(lens), cap, nq=16, nkv=8, d=d) as r:
        r.append([0] * len(lens), [a + b for a, b in zip(lens, new)])
        q = r.rows(sum(new), 16)
        a, b = r.attend(lens, new, q=q, pad=2), r.attend(lens, new, q=q, pad=2, check=False)
        assert torch.equal(a, b) and r.status() == (0, 0)
