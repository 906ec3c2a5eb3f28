"""Attention over the 8-bit cache on contents that it holds without loss: no
page is lost, counted twice or taken for another, in any of the ways in which
the work is cut, and weights are right to the roundings that remain."""
import kv8_exact as ex
import numpy as np
import pytest
import torch
from kv8_ref import bf16
from test_gpu_kv8 import bits, dev

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu

PAGE = 16


class Held:
    """A cache whose sessions hold totals[b] tokens of the given K and V, pages shuffled. width: of the block
    tables (the entries behind a session's pages are -1)."""

    def __init__(self, totals, nq, nkv, d, k, v, width=0):
        pages = [-(-n // PAGE) for n in totals]
        self.B, self.nq, self.nkv, self.d = len(totals), nq, nkv, d
        self.stride = max(max(pages), width)
        self.c = qtts.qtts_kv8_create(qtts.Kv8Config(1, nq, nkv, d, 0.0, PAGE, self.B, self.stride * PAGE, sum(pages)))
        order = np.random.default_rng(sum(totals)).permutation(sum(pages)).astype(np.int32)
        bt = np.full((self.B, self.stride), -1, np.int32)
        at = 0
        for b, p in enumerate(pages):
            bt[b, :p] = order[at:at + p]
            at += p
        self.bt = dev(bt)
        self.work = torch.zeros(qtts.qtts_kv8_workspace_bytes(self.c), dtype=torch.uint8, device="cuda")
        start = np.concatenate(([0], np.cumsum(totals))).astype(np.int32)
        zero = torch.zeros(self.B, dtype=torch.int32, device="cuda")
        kb, vb, w = bits(bf16(np.concatenate(k))[0]), bits(bf16(np.concatenate(v))[0]), nkv * d
        qtts.qtts_kv8_append(self.c, 0, self.B, int(start[-1]), max(totals), dev(start), zero, self.bt, self.stride, kb,
                             w, vb, w)
        torch.cuda.synchronize()

    def __enter__(self):
        return self

    def __exit__(self, *e):
        qtts.qtts_kv8_destroy(self.c)

    def attend(self, q, lens, new, scale, max_new=0):
        """q: bf16 bits [rows][nq][d], rows packed. max_new: larger than what the sessions have."""
        start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        n, w = int(start[-1]), self.nq * self.d
        out = torch.full((n, self.nq, self.d), float("nan"), dtype=torch.bfloat16, device="cuda")
        qtts.qtts_kv8_attention(self.c, 0, self.B, n, max(max_new, max(new)), dev(start), dev(np.asarray(lens, np.int32)),
                                self.bt, self.stride, bits(q), w, scale, out, w, self.work)
        assert qtts.qtts_kv8_status(self.c, raise_on_error=False) == (0, qtts.QTTS_DEV_OK)
        return out.double().cpu().numpy(), start


def ragged(B, lo, hi):
    return [lo + (hi - lo) * ((b * 7 + 3) % B) // max(B - 1, 1) for b in range(B)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,nq,nkv,width,max_new", [
    ([129999], [1], 2, 1, 0, 0),                      # one long session, cut over all CTAs
    ([15999, 31], [1, 1], 8, 2, 0, 0),
    (ragged(8, 0, 511), [1] * 8, 16, 8, 0, 0),
    (ragged(32, 100, 1200), [1] * 32, 16, 8, 0, 0),   # a CTA for each tile
    (ragged(32, 100, 1200), [1] * 32, 16, 8, 16384, 0),   # the same from tables for long sessions
    (ragged(300, 0, 900), [1] * 300, 4, 2, 0, 0),     # more tiles than CTAs
    (ragged(300, 0, 40), [1] * 300, 16, 2, 16384, 0),
    (ragged(16, 0, 3000), [1] * 16, 64, 4, 0, 0),     # 16 columns
    (ragged(16, 0, 3000), [1] * 16, 64, 4, 16384, 0),
    (ragged(8, 900, 3000), [8] * 8, 16, 8, 0, 0),     # 16 columns of 8 rows
    (ragged(5, 0, 2000), [1, 3, 0, 2, 1], 32, 1, 0, 0),   # up to 96 columns
    (ragged(32, 100, 1200), [1] * 32, 16, 8, 0, 4),   # single tokens of calls that allow for more
    (ragged(32, 100, 1200), [1] * 32, 16, 8, 0, 8),
    (ragged(32, 100, 1200), [1] * 32, 16, 8, 0, 512),
    ([700, 0, 33], [90, 1, 1], 16, 8, 0, 0),          # a prompt beside single tokens
    ([8000], [100], 2, 2, 0, 0),                      # one tile's key steps over many CTAs
    ([0, 100, 1000], [1300, 900, 40], 64, 8, 0, 0),   # tiles of 256 rows
    ([3000], [1500], 6, 2, 0, 0),
])
def test_means_of_marked_pages(d, lens, new, nq, nkv, width, max_new):
    """A softmax scale of 0: the mean of V over the tokens seen; every page marks a dim."""
    totals = [a + b for a, b in zip(lens, new)]
    rng = np.random.default_rng(7)
    k = [ex.integers(rng, n, nkv, d, np.ones((-(-n // PAGE), nkv))) if n else np.zeros((0, nkv, d)) for n in totals]
    v = [ex.marks(n, nkv, d, 11 * b) for b, n in enumerate(totals)]
    q = bf16(rng.standard_normal((sum(new), nq, d)))[0]
    with Held(totals, nq, nkv, d, k, v, width) as c:
        got, start = c.attend(q, lens, new, 0.0, max_new)
    for b, n in enumerate(new):
        want = np.repeat(ex.mean_of_marks(lens[b] + np.arange(n), nkv, d, 11 * b), nq // nkv, 1)
        bad = np.abs(got[start[b]:start[b + 1]] - want) > ex.mean_bound(want)
        assert not bad.any(), (b, np.argwhere(bad)[:5])
        assert not np.isnan(got[start[b]:start[b + 1]]).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1.0, -1.0, 8.0])  # of 1 / sqrt(d)
@pytest.mark.parametrize("lens,new,nq,nkv,width", [
    ([0, 15, 100, 1023], [1] * 4, 4, 2, 0),
    ([4000], [1], 2, 1, 0),
    ([20, 300, 999], [1] * 3, 32, 2, 0),
    ([20, 300, 999], [1] * 3, 32, 2, 4096),
    ([60, 0, 700], [9, 1, 4], 4, 2, 0),
    ([5, 200, 0], [20, 60, 130], 4, 2, 0),
    ([1500], [70], 4, 2, 0),
    ([100, 0], [700, 600], 64, 8, 0),
])
def test_weights_of_real_scores(d, scale, lens, new, nq, nkv, width):
    """K and V blocks of sizes 16 times apart."""
    totals = [a + b for a, b in zip(lens, new)]
    rng = np.random.default_rng(len(lens) * 100 + nq)
    k = [ex.integers(rng, n, nkv, d, ex.steps(rng, n, nkv, -8, -6)) for n in totals]
    v = [ex.integers(rng, n, nkv, d, ex.steps(rng, n, nkv, -9, -5)) for n in totals]
    qb, q = bf16(rng.standard_normal((sum(new), nq, d)))
    s = scale * d ** -0.5
    with Held(totals, nq, nkv, d, k, v, width) as c:
        got, start = c.attend(qb, lens, new, s)
    for b in range(len(new)):
        rows = slice(start[b], start[b + 1])
        want, tol = ex.attention(q[rows], k[b], v[b], lens[b], np.float64(np.float32(s)))
        off = np.abs(got[rows] - want)
        assert np.all(off <= tol), (b, np.max(off - tol), np.argwhere(~(off <= tol))[:3])
