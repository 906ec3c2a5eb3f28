"""Attention of many rows over the 8-bit cache gives the same bits call after
call, whatever the order in which a CTA's warps come along."""
import pytest
import torch
from test_gpu_kv8 import Rig

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv,lo,span,new", [(16, 8, 0, 51, 20), (8, 8, 0, 96, 33), (32, 2, 20, 51, 8), (16, 8, 80, 80, 40)])
def test_tiles_of_one_and_two_key_steps(d, nq, nkv, lo, span, new):
    """Tiles of at most 128 keys are one key step: one of the two softmax groups of the
    128-row form has no step in them and is done while the other has just begun. 32
    sessions of such tiles (the last case: of one and of two steps), 60 times."""
    lens = [lo + (7 * b) % span for b in range(32)]
    with Rig(32, 256, nq=nq, nkv=nkv, d=d) as r:
        r.append([0] * 32, [n + new for n in lens])
        q = r.rows(32 * new, nq)
        first = r.attend(lens, [new] * 32, q=q)
        for _ in range(60):
            assert torch.equal(first, r.attend(lens, [new] * 32, q=q, check=False))
        assert r.status() == (0, qtts.QTTS_DEV_OK)
