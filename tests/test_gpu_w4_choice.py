"""Products of 33 to 64 rows on both sides of the sizes at which another kernel takes them."""
import numpy as np
import pytest
import torch
from kv8_ref import bf16
from test_gpu_w4 import Linear, bits, check

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [3584, 3585, 9728, 9729])
@pytest.mark.parametrize("tiles", [7, 8, 15, 16])  # of 64 k; the 32nd k of the last is missing in groups of 32
@pytest.mark.parametrize("M,group", [(33, 32), (64, 64)])
def test_products(N, tiles, M, group):
    K = tiles * 64 - (32 if group == 32 else 0)
    rng = np.random.default_rng(N + K)
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    sb, s = bf16(np.exp(rng.standard_normal((N, K // group))))
    xb, x = bf16(rng.standard_normal((M, K)))
    with Linear(N, K, group) as L:
        qtts.qtts_w4_load(L.w, q, sb)
        y = torch.full((M + 1, N), 7.0, device="cuda")
        qtts.qtts_w4_linear(L.w, M, bits(xb), K, y, N, qtts.QTTS_DTYPE_F32)
        y = y.double().cpu().numpy()
        assert (y[M] == 7).all()
        check(y[:M], x, q, s, group, True)
