"""The low-bit operators as a decode step runs them: a layer's fused QKV
projection in 4 bits, its keys and values appended to the 8-bit cache straight
from that projection's rows, attention over the cache, and the output
projection in 4 bits with fp32 results: captured once, replayed step by step.
Each stage is held to its definition on the inputs that it got."""
import kv8_ref as ref
import numpy as np
import pytest
import torch
from test_gpu_kv8 import Rig, bits, dev
from test_gpu_w4 import Linear, check, quantize

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,lens,group", [(1, [0], 128), (5, [3, 100, 15, 16, 47], 32), (12, [60] * 12, 64)])
def test_a_layer_step_replayed_from_a_graph(B, lens, group):
    hidden, nq, nkv, d, steps = 512, 8, 4, 64, 3
    wide = (nq + 2 * nkv) * d
    rng = np.random.default_rng(B)
    with Rig(B, max(lens) + steps, nq=nq, nkv=nkv, d=d) as r, Linear(wide, hidden, group) as qkv, \
            Linear(hidden, nq * d, group) as proj:
        mats = []
        for L in (qkv, proj):
            wb, w = ref.bf16(rng.standard_normal((L.N, L.K)) * L.K ** -0.5)
            qtts.qtts_w4_quantize(L.w, bits(wb))
            mats.append(quantize(w, group))
        if max(lens):
            r.append([0] * B, lens)
        x = torch.zeros(B, hidden, dtype=torch.int16, device="cuda")
        rows = torch.zeros(B, wide, dtype=torch.bfloat16, device="cuda")
        att = torch.zeros(B, nq * d, dtype=torch.bfloat16, device="cuda")
        y = torch.zeros(B, hidden, device="cuda")
        kv_len = dev(np.array(lens, np.int32))
        k, v = rows[:, nq * d:], rows[:, (nq + nkv) * d:]

        def step(s):
            qtts.qtts_w4_linear(qkv.w, B, x, hidden, rows, wide, qtts.QTTS_DTYPE_BF16, s)
            qtts.qtts_kv8_append(r.c, 0, B, B, 1, None, kv_len, r.bt, r.stride, k, wide, v, wide, s)
            qtts.qtts_kv8_attention(r.c, 0, B, B, 1, None, kv_len, r.bt, r.stride, rows, wide, d ** -0.5, att, nq * d,
                                    r.work, s)
            qtts.qtts_w4_linear(proj.w, B, att, nq * d, y, hidden, qtts.QTTS_DTYPE_F32, s)
            kv_len.add_(1)

        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(s)
        for i in range(steps):
            xb, xv = ref.bf16(rng.standard_normal((B, hidden)))
            x.copy_(bits(xb))
            g.replay()
            torch.cuda.synchronize()
            fused = rows.double().cpu().numpy()
            check(fused, xv, mats[0][0], mats[0][2], group, False)
            fused = fused.reshape(B, nq + 2 * nkv, d)
            at = [n + i for n in lens]
            for b in range(B):
                r.ref.append(r.tables[b], at[b], fused[b:b + 1, nq:nq + nkv], fused[b:b + 1, nq + nkv:])
            got = att.double().cpu().numpy()
            r.check_out(got.reshape(B, nq, d), np.arange(B + 1), at, [1] * B, fused[:, :nq], d ** -0.5)
            check(y.double().cpu().numpy(), got, mats[1][0], mats[1][2], group, True)
        r.check_cache([n + steps for n in lens])
        assert r.status() == (0, 0)


def test_a_prompt_then_tokens():
    """A prompt in two chunks and then single tokens, next to a session that only decodes."""
    nq, nkv, d = 4, 2, 128
    with Rig(2, 400, nq=nq, nkv=nkv, d=d) as r:
        lens = [0, 90]
        r.append([0, 0], [0, 90])
        for new in ([150, 1], [37, 1], [1, 1], [1, 1]):
            r.append(lens, new)
            r.attend(lens, new)
            lens = [a + b for a, b in zip(lens, new)]
        r.check_cache(lens)
        assert r.status() == (0, 0)
