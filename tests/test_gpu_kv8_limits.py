"""Calls of the 8-bit cache with row counts and bounds far above what its sessions have."""
import numpy as np
import pytest
import torch
from test_gpu_kv8 import Rig, bits, dev

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu

MAX = 2 ** 31 - 1


@pytest.mark.parametrize("n_rows,max_new", [(21, MAX), (MAX, 16), (MAX, MAX), (MAX - 7, MAX - 20)])
def test_append_and_read_with_bounds_of_any_size(n_rows, max_new):
    with Rig(2, 64) as r:
        k, v, w = r.rows(21), r.rows(21), r.nkv * r.d
        start, lens = dev(np.array([0, 5, 21], np.int32)), dev(np.array([0, 0], np.int32))
        qtts.qtts_kv8_append(r.c, 0, 2, n_rows, max_new, start, lens, r.bt, r.stride, bits(k[0]), w, bits(v[0]), w)
        for b, s in ((0, slice(0, 5)), (1, slice(5, 21))):
            r.ref.append(r.tables[b], 0, k[1][s], v[1][s])
        r.check_cache([5, 16])
        tight = r.read([0, 0], [5, 16])
        got = [torch.zeros(21, r.nkv, r.d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        qtts.qtts_kv8_read(r.c, 0, 2, n_rows, max_new, start, lens, r.bt, r.stride, got[0], got[1])
        assert all(np.array_equal(a.double().cpu().numpy(), b) for a, b in zip(got, tight))
        assert r.status() == (0, 0)


@pytest.mark.parametrize("n_rows,max_new", [(25, MAX), (MAX, 1), (MAX, 8), (MAX, 16), (MAX, MAX), (MAX - 7, MAX - 20)])
def test_attention_with_bounds_of_any_size(n_rows, max_new):
    """Up to 2, 9 to 16 and more columns of bounds; one row, or 25 rows of 16 at most."""
    new = [1, 0, 0] if max_new == 1 else [8, 0, 3] if max_new == 8 else [9, 0, 16]
    lens = [60, 7, 33]
    with Rig(3, 128) as r:
        r.append([0] * 3, [a + b for a, b in zip(lens, new)])
        start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        q = r.rows(int(start[-1]), r.nq)
        out = torch.zeros(int(start[-1]), r.nq, r.d, dtype=torch.bfloat16, device="cuda")
        w = r.nq * r.d
        qtts.qtts_kv8_attention(r.c, 0, 3, n_rows, max_new, dev(start), dev(np.array(lens, np.int32)), r.bt, r.stride,
                                bits(q[0]), w, 0.1, out, w, r.work)
        r.check_out(out.double().cpu().numpy(), start, lens, new, q[1], 0.1)
        assert r.status() == (0, 0)
