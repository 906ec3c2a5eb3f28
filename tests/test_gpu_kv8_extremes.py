"""Attention over the 8-bit cache where weights or values leave the usual range."""
import kv8_exact as ex
import numpy as np
import pytest
from kv8_ref import bf16
from test_gpu_kv8_exact import Held

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv,new", [(2, 1, 1), (2, 1, 40), (64, 8, 1100)])
@pytest.mark.parametrize("big", [0, 30, 60])
def test_blocks_of_zeros_keep_their_weights(d, nq, nkv, new, big):
    """V blocks of zeros (four pages of every eight) beside blocks of 127 * 2^big: the zeros' tokens count in the mean.
    Beyond mean_bound: exponentials of 2^+-100 (2^-22), and sums that moved with the maximum, twice at most in a
    warp and in each join (two factors of 2^-22): below 2^-18."""
    n = 1200 + new
    page = np.arange(n) // 16
    k = np.full((n, nkv, d), 1.0)
    v = np.zeros((n, nkv, d))
    v[page % 8 >= 4] = 127 * 2.0 ** big
    q = bf16(np.ones((new, nq, d)))[0]
    lens = n - new
    with Held([n], nq, nkv, d, [k], [v]) as c:
        got, _ = c.attend(q, [lens], [new], 0.0)
    seen = lens + np.arange(new)
    want = (np.cumsum(v[:, 0, 0])[seen] / (seen + 1))[:, None, None]
    assert np.all(np.abs(got - want) <= ex.mean_bound(want) + 2.0 ** -18 * want)


@pytest.mark.parametrize("at", [0, 20, 39])
@pytest.mark.parametrize("new", [1, 12, 40])
def test_a_nan_shows_however_small_its_weight(new, at):
    """A block of V with a NaN in page `at` of 40 or more, whose keys' scores are 127 * 64 below the others': 0 * NaN."""
    n, d = 40 * 16 - 4 + new, 64
    k = np.full((n, 2, d), 0.5 * 127)
    k[at * 16:at * 16 + 16] *= -1
    v = ex.marks(n, 2, d)
    v[at * 16, 1, 9] = np.nan
    q = bf16(np.ones((new, 2, d)))[0]
    lens = n - new
    with Held([n], 2, 2, d, [k], [v]) as c:
        got, _ = c.attend(q, [lens], [new], 1.0)
    sees = lens + np.arange(new) >= at * 16
    assert np.isnan(got[sees, 1]).all()
    assert np.isfinite(got[~sees]).all() and np.isfinite(got[:, 0]).all()
