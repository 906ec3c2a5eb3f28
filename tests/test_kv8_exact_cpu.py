"""What the checks of kv8_exact would catch: results of nothing, of a page left
out, of a page counted twice and of a page taken for another are outside their
bounds, at the lengths that they are used at."""
import kv8_exact as ex
import numpy as np
import pytest
from kv8_ref import Cache, bf16


def test_the_cache_holds_the_values_without_loss():
    rng = np.random.default_rng(1)
    n = 70
    k, v = ex.integers(rng, n, 2, 64, ex.steps(rng, n, 2, -9, 3)), ex.marks(n, 2, 64, 5)
    assert np.array_equal(bf16(k)[1], k) and np.array_equal(bf16(v)[1], v)
    c = Cache(5, 2, 64, 0.0)
    c.append(np.arange(5), 0, k, v)
    assert all(np.array_equal(a, b) for a, b in zip(c.values(np.arange(5), n), (k, v)))


@pytest.mark.parametrize("pos", [0, 15, 16, 100, 1023, 4000])
@pytest.mark.parametrize("d,first", [(64, 0), (128, 77)])
def test_marks_have_the_mean_that_is_said(pos, d, first):
    v = ex.marks(pos + 1, 2, d, first)
    assert np.allclose(ex.mean_of_marks([pos], 2, d, first)[0], v.mean(0), rtol=1e-12, atol=0)


@pytest.mark.parametrize("n", [20, 500, 4000, 130000])
def test_flat_weights_show_every_page(n):
    """Of 130000 tokens a whole page (at that length less than a page is within the rounding to bf16)."""
    d = 64
    want = ex.mean_of_marks([n - 1], 1, d)[0]
    tol = ex.mean_bound(want)
    v = ex.marks(n, 1, d)
    total = v.sum(0)
    for page in sorted({0, 1, (n - 1) // 16 // 2, (n - 1) // 16}):
        here = v[page * 16:page * 16 + 16]
        for got in (total * 0, (total - here.sum(0)) / (n - len(here)), (total - here.sum(0)) / n,
                    (total + here.sum(0)) / (n + len(here)), (total - here.sum(0) + np.roll(here.sum(0), 1, -1)) / n):
            if len(here) < n or not got.any():
                assert np.any(np.abs(got - want) > tol), page


@pytest.mark.parametrize("n", [100, 300, 1023, 4000])
def test_weights_of_real_scores_show_every_page(n):
    rng = np.random.default_rng(n)
    nq, nkv, d, new = 4, 2, 64, 2
    k, v = (ex.integers(rng, n, nkv, d, ex.steps(rng, n, nkv, -6, -6)) for _ in range(2))
    q = bf16(rng.standard_normal((new, nq, d)))[1]
    scale = d ** -0.5
    want, tol = ex.attention(q, k, v, n - new, scale)
    assert np.all(np.abs(0 * want - want).max(-1) > tol.max(-1))
    pages = -(-n // 16)
    for page in range(0, pages, max(1, pages // 8)):
        rows = np.arange(n)
        for keep in (rows[rows // 16 != page], np.sort(np.concatenate((rows, rows[rows // 16 == page])))):
            for h in range(nq):
                kh, vh = k[keep, h // 2], v[keep, h // 2]
                x = q[0, h] @ kh.T * scale + np.where(keep > n - new, -np.inf, 0)
                p = np.exp(x - x.max())
                assert np.any(np.abs(p @ vh / p.sum() - want[0, h]) > tol[0, h]), (page, h)
