"""What the low-bit decode operators are measured on: the 8-bit paged K/V
cache (append with the position rotation, attention over it) and products with
4-bit weights. `run` computes each in plain torch operations where `own` is
false and calls the library where it is true.

A cache block is one page (16 tokens) of one kv head's K or V; it holds int8
codes and one fp32 scale. Appending to a block: scale = max(the scale of the
tokens already in it, max|new values| / 127), codes = round(x / scale), and the
codes already there are rescaled where the scale grew.
"""
import math
import weakref

import torch

own = False

PAGE = 16
THETA = 1e6
DEV = "cuda"


# ---------------------------------------------------------------- the cases

def _append(name, B, ctx, new, nkv=8, d=128):
    return {"name": name, "op": "append", "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
            "new_hi": new[1], "nkv": nkv, "d": d}


def _attend(name, B, ctx, new, nq=16, nkv=8, d=128):
    return {"name": name, "op": "attention", "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
            "new_hi": new[1], "nq": nq, "nkv": nkv, "d": d}


def _linear(name, M, N, K, group=128, fp32=False):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "group": group, "fp32": fp32}


def listed():
    return [
        # one decode step of the largest batch: every session appends the token of one frame
        _append("append 32 x 1 token", 32, (100, 1200), (1, 1)),
        # one prompt placed behind a short prefix, starting and ending inside a page
        _append("append 1 x 501 tokens", 1, (37, 37), (501, 501)),
        # a batch of long ragged prompts
        _append("append 32 x 60..1000 tokens", 32, (0, 300), (60, 1000)),
        # the first frames of a single session: latency
        _attend("attend 1 x 1, 128 back", 1, (128, 128), (1, 1)),
        # a small ragged batch of sessions
        _attend("attend 8 x 1, 64..512 back", 8, (64, 512), (1, 1)),
        # the largest batch, sessions of very different ages
        _attend("attend 32 x 1, 100..1200 back", 32, (100, 1200), (1, 1)),
        # one very long session, the work of one token split over the machine
        _attend("attend 1 x 1, 130001 back", 1, (130001, 130001), (1, 1)),
        # many long sessions: the cache's own bandwidth
        _attend("attend 32 x 1, 4k..16k back", 32, (4001, 16003), (1, 1)),
        # a prompt chunk of the prompt pass's size behind an earlier one
        _attend("attend 1 x 1024, 1000 back", 1, (1000, 1000), (1024, 1024)),
        # one session's fused QKV projection: latency
        _linear("w4 1 x 4096 x 2048", 1, 4096, 2048),
        # one session's gate and up projections, with the finest groups
        _linear("w4 1 x 12288 x 2048, groups of 32", 1, 12288, 2048, group=32),
        # the largest batch through the down projection, added to an fp32 residual by the caller
        _linear("w4 32 x 2048 x 6144, fp32 out", 32, 2048, 6144, group=64, fp32=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "linear"])
    if op == "linear":
        group = rng.choice([32, 64, 128])
        return {"op": op, "M": _log(rng, 1, 64), "N": _log(rng, 40, 12288), "K": group * _log(rng, 3, 6144 // group),
                "group": group, "fp32": rng.random() < 0.5}
    B = _log(rng, 1, 32)
    nkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "append":
        new = rng.choice([1, _log(rng, 2, 1000)])
        ctx = _log(rng, 1, 2000)
        return {"op": op, "B": B, "ctx_lo": ctx // 3, "ctx_hi": ctx, "new_lo": (new + 1) // 2, "new_hi": new,
                "nkv": nkv, "d": d}
    new = rng.choice([1, 1, 1, _log(rng, 2, 1024)])
    if new == 1:
        ctx = min(_log(rng, 1, 130001), 300000 // B)
    else:
        ctx = min(_log(rng, 1, 4000), 2000000 // (B * new))
    new = min(new, max(1, 1024 // B))
    return {"op": op, "B": B, "ctx_lo": ctx // 3, "ctx_hi": ctx, "new_lo": (new + 1) // 2, "new_hi": new,
            "nq": nkv * rng.choice([1, 2, 4, 8]), "nkv": nkv, "d": d}


def _ragged(lo, hi, B, step):
    """B lengths spread over lo..hi, in no order."""
    return [lo + (hi - lo) * ((b * step + 3) % B) // max(B - 1, 1) if B > 1 else hi for b in range(B)]


def _lengths(case):
    B = case["B"]
    return _ragged(case["ctx_lo"], case["ctx_hi"], B, 7), _ragged(case["new_lo"], case["new_hi"], B, 5)


# --------------------------------------------------------------- the inputs

def _inputs(case, seed):
    """The data a step brings: random tensors made from the seed alone."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["op"] == "linear":
        w = (randn(case["N"], case["K"]) * 0.02).bfloat16()
        return {"w": w, "x": randn(case["M"], case["K"]).bfloat16()}
    ctx, new = _lengths(case)
    nkv, d = case["nkv"], case["d"]
    gain = torch.exp(0.5 * randn(nkv, d))  # keys have channels of different size

    def rows(n):
        k, v = randn(n, nkv, d), randn(n, nkv, d)
        return (k * gain / gain.square().mean(-1, keepdim=True).sqrt()).bfloat16(), v.bfloat16()

    pages = [-(-(c + n) // PAGE) for c, n in zip(ctx, new)]
    order = torch.randperm(sum(pages), generator=g, device=DEV).int()
    bt = torch.full((case["B"], max(pages)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, p in enumerate(pages):
        bt[b, :p] = order[at:at + p]
        at += p
    held = ctx if case["op"] == "append" else [c + n for c, n in zip(ctx, new)]
    i = {"pages": sum(pages), "bt": bt, "held": held, "ctx": ctx, "new": new}
    i["held_k"], i["held_v"] = rows(sum(held))
    if case["op"] == "append":
        i["k"], i["v"] = rows(sum(new))
    else:
        i["q"] = randn(sum(new), case["nq"], d).bfloat16()
    return i


def _starts(n):
    s = [0]
    for x in n:
        s.append(s[-1] + x)
    return torch.tensor(s, dtype=torch.int32, device=DEV)


class _State:
    pass


def prepare(case, seed):
    i = _inputs(case, seed)
    s = _State()
    s.op = case["op"]
    if s.op == "linear":
        s.x = i["x"]
        s.M, s.N, s.K, s.group, s.fp32 = case["M"], case["N"], case["K"], case["group"], case["fp32"]
        s.y = torch.empty(s.M, s.N, dtype=torch.float32 if s.fp32 else torch.bfloat16, device=DEV)
        if own:
            from codebook_decode_gb300 import qtts
            s.qtts = qtts
            s.w = qtts.qtts_w4_create(s.N, s.K, s.group)
            s.free = weakref.finalize(s, qtts.qtts_w4_destroy, s.w)
            qtts.qtts_w4_quantize(s.w, i["w"])
        else:
            s.codes, s.scale = _quantize4(i["w"], s.group)
        return s
    B = case["B"]
    s.B, s.nkv, s.d, s.nq = B, case["nkv"], case["d"], case.get("nq", case["nkv"])
    s.bt = i["bt"]
    s.kv_len = torch.tensor(i["ctx"], dtype=torch.int32, device=DEV)
    s.row_start = _starts(i["new"])
    s.rows, s.max_new = sum(i["new"]), max(i["new"])
    s.one = s.max_new == 1 and min(i["new"]) == 1
    held, held_start = i["held"], _starts(i["held"])
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    if s.op == "append":
        s.k, s.v = i["k"], i["v"]
        # what a step touches is read back from the start of its first page
        back = [c % PAGE + n for c, n in zip(i["ctx"], i["new"])]
        s.back_len = s.kv_len // PAGE * PAGE
        s.back_start = _starts(back)
        s.back_rows, s.back_max = sum(back), max(back)
        s.k_back = torch.empty(s.back_rows, s.nkv, s.d, dtype=torch.bfloat16, device=DEV)
        s.v_back = torch.empty_like(s.k_back)
    else:
        s.q, s.out = i["q"], torch.empty_like(i["q"])
    if own:
        from codebook_decode_gb300 import qtts
        s.qtts = qtts
        c = qtts.Kv8Config(n_layers=1, n_q_heads=s.nq, n_kv_heads=s.nkv, head_dim=s.d, rope_theta=THETA,
                           page_size=PAGE, max_batch=B, max_context=max(a + n for a, n in zip(i["ctx"], i["new"])),
                           pool_pages=i["pages"])
        s.cache = qtts.qtts_kv8_create(c)
        s.free = weakref.finalize(s, qtts.qtts_kv8_destroy, s.cache)
        s.work = torch.zeros(qtts.qtts_kv8_workspace_bytes(s.cache), dtype=torch.uint8, device=DEV)
        if sum(held):
            qtts.qtts_kv8_append(s.cache, 0, B, sum(held), max(held), held_start, zero, s.bt, s.bt.shape[1],
                                 i["held_k"], s.nkv * s.d, i["held_v"], s.nkv * s.d)
    else:
        s.codes = torch.zeros(i["pages"], s.nkv, 2, PAGE, s.d, dtype=torch.int8, device=DEV)
        s.scale = torch.zeros(i["pages"], s.nkv, 2, device=DEV)
        if sum(held):
            _append_plain(s, i["held_k"], i["held_v"], held_start, zero)
    torch.cuda.synchronize()
    return s


# ------------------------------------------------------------ the operators

def run(s):
    return {"append": _run_append, "attention": _run_attention, "linear": _run_linear}[s.op](s)


def _run_append(s):
    """Append, then read the pages that were touched: the cache's new state."""
    if own:
        n = s.nkv * s.d
        s.qtts.qtts_kv8_append(s.cache, 0, s.B, s.rows, s.max_new, None if s.one else s.row_start, s.kv_len, s.bt,
                               s.bt.shape[1], s.k, n, s.v, n, _stream())
        s.qtts.qtts_kv8_read(s.cache, 0, s.B, s.back_rows, s.back_max, s.back_start, s.back_len, s.bt,
                             s.bt.shape[1], s.k_back, s.v_back, _stream())
        return s.k_back, s.v_back
    _append_plain(s, s.k, s.v, s.row_start, s.kv_len)
    b, pos = _positions(s.back_start, s.back_len, s.back_rows)
    page = s.bt[b, pos // PAGE].long()
    got = s.codes[page, :, :, pos % PAGE].float() * s.scale[page][..., None]
    return got[:, :, 0].bfloat16(), got[:, :, 1].bfloat16()


def _run_attention(s):
    if own:
        s.qtts.qtts_kv8_attention(s.cache, 0, s.B, s.rows, s.max_new, None if s.one else s.row_start, s.kv_len, s.bt,
                                  s.bt.shape[1], s.q, s.nq * s.d, 1 / math.sqrt(s.d), s.out, s.nq * s.d, s.work,
                                  _stream())
        return s.out
    B, P, nkv, d, n = s.B, s.bt.shape[1], s.nkv, s.d, s.max_new
    page = s.bt.clamp_min(0).long()
    held = s.codes[page].float() * s.scale[page][..., None, None]  # [B, P, nkv, 2, PAGE, d]
    k = held[:, :, :, 0].transpose(1, 2).reshape(B, nkv, P * PAGE, d)
    v = held[:, :, :, 1].transpose(1, 2).reshape(B, nkv, P * PAGE, d)
    b, pos = _positions(s.row_start, s.kv_len, s.rows)
    i = pos - s.kv_len[b]
    q = torch.zeros(B, n, s.nq, d, device=DEV)
    q[b, i] = _rotate(s.q.float(), pos)
    q = q.reshape(B, n, nkv, s.nq // nkv, d).permute(0, 2, 1, 3, 4).reshape(B, nkv, -1, d)
    x = q @ k.transpose(-1, -2) / math.sqrt(d)  # [B, nkv, n * group, P * PAGE]
    last = s.kv_len[:, None] + torch.arange(n, device=DEV)
    seen = torch.arange(P * PAGE, device=DEV) <= last[..., None]  # [B, n, P * PAGE]
    x = x.view(B, nkv, n, -1, P * PAGE).masked_fill(~seen[:, None, :, None], -math.inf).view(B, nkv, -1, P * PAGE)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    y = p @ v / p.sum(-1, keepdim=True)
    y = y.view(B, nkv, n, s.nq // nkv, d).permute(0, 2, 1, 3, 4).reshape(B, n, s.nq, d)
    s.out.copy_(y[b, i])
    return s.out


def _run_linear(s):
    if own:
        s.qtts.qtts_w4_linear(s.w, s.M, s.x, s.K, s.y, s.N, s.qtts.QTTS_DTYPE_F32 if s.fp32 else s.qtts.QTTS_DTYPE_BF16,
                              _stream())
        return s.y
    w = torch.stack((s.codes & 15, s.codes >> 4), -1).view(s.N, -1, s.group).float() - 8
    w = (w * s.scale.float()[..., None]).view(s.N, s.K)
    s.y.copy_(s.x.float() @ w.t())
    return s.y


def _stream():
    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------- the plain forms' own parts

def _positions(start, pos0, rows):
    """The session and the position of each packed row."""
    r = torch.arange(rows, device=DEV, dtype=torch.int32)
    b = torch.bucketize(r, start[1:], right=True)
    return b, pos0[b] + r - start[b]


def _rotate(x, pos):
    """Rotate-half position rotation of x [rows, heads, d]; angles in 64 bits."""
    h = x.shape[-1] // 2
    a = pos[:, None].double() * THETA ** (-torch.arange(h, device=DEV, dtype=torch.float64) / h)
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    return torch.cat((x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s), -1)


def _append_plain(s, k, v, start, pos0):
    rows = k.shape[0]
    b, pos = _positions(start, pos0, rows)
    x = torch.stack((_rotate(k.float(), pos), v.float()), 2)  # [rows, nkv, 2, d]
    page, slot = s.bt[b, pos // PAGE].long(), pos % PAGE
    new = torch.zeros_like(s.scale)
    new.index_reduce_(0, page, x.abs().amax(-1) / 127, "amax")
    # the block that a session's first new row falls into keeps the tokens before it
    there = (slot > 0) & (pos == pos0[b])
    first = page[there]
    old = s.scale[first]
    scale = new.clone()
    scale[first] = torch.maximum(new[first], old)
    grown = torch.where(old > 0, old / scale[first], 1.0)
    s.codes[first] = torch.round(s.codes[first].float() * grown[..., None, None]).to(torch.int8)
    s.scale[page] = scale[page]
    inv = torch.where(scale > 0, 1 / scale, 0.0)[page]
    s.codes[page, :, :, slot] = torch.round(x * inv[..., None]).clamp(-127, 127).to(torch.int8)


def _quantize4(w, group):
    """codes + 8, two to a byte along K, and bf16 scales [N, K / group]."""
    N, K = w.shape
    w = w.float().view(N, K // group, group)
    scale = (w.abs().amax(-1) / 7).bfloat16()
    q = torch.round(w / scale.float()[..., None]).nan_to_num(0).clamp(-7, 7).to(torch.int32).view(N, K // 2, 2) + 8
    return (q[..., 0] | q[..., 1] << 4).to(torch.uint8), scale


# ------------------------------------------------- what cannot be done without

def work(case):
    if case["op"] == "linear":
        M, N, K, group = case["M"], case["N"], case["K"], case["group"]
        return {"bytes": N * K / 2 + N * (K // group) * 2 + M * K * 2 + M * N * (4 if case["fp32"] else 2),
                "flops": 2 * M * N * K}
    ctx, new = _lengths(case)
    nkv, d = case["nkv"], case["d"]
    if case["op"] == "append":
        rows, back = sum(new), sum(c % PAGE + n for c, n in zip(ctx, new))
        per = nkv * d * 2
        return {"bytes": rows * per * (2 + 1) + back * per * (1 + 2), "flops": rows * nkv * d * 8}
    nq = case["nq"]
    seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    held = sum(c + n for c, n in zip(ctx, new))
    return {"bytes": held * nkv * d * 2 + -(-held // PAGE) * nkv * 8 + sum(new) * nq * d * 4, "flops": seen * nq * d * 4}


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    i = _inputs(case, seed)
    if case["op"] == "linear":
        group = case["group"]
        w = i["w"].double().unflatten(1, (-1, group))
        s = (w.abs().amax(2, keepdim=True) / 7).bfloat16().double()
        q = (w / s).round().nan_to_num(0).clamp(-7, 7)
        return torch.einsum("mk,nk->mn", i["x"].double(), (q * s).flatten(1))
    ctx, new, out_k, out_v = i["ctx"], i["new"], [], []
    row = held = 0
    outs = []
    for c, n, h in zip(ctx, new, i["held"]):
        k, v = i["held_k"][held:held + h].double(), i["held_v"][held:held + h].double()
        held += h
        k, ks = _blocks(_turn(k, 0))
        v, vs = _blocks(v)
        if case["op"] == "append":
            k2, v2 = i["k"][row:row + n].double(), i["v"][row:row + n].double()
            row += n
            out_k.append(_extend(k, ks, _turn(k2, c), c))
            out_v.append(_extend(v, vs, v2, c))
            continue
        k, v = (k * ks).flatten(0, 1)[:h], (v * vs).flatten(0, 1)[:h]
        q = _turn(i["q"][row:row + n].double(), c).unflatten(1, (case["nkv"], -1))
        row += n
        x = torch.einsum("ihgd,jhd->hgij", q, k) / case["d"] ** 0.5
        j, t = torch.arange(h, device=DEV), torch.arange(n, device=DEV)
        x = torch.softmax(x.masked_fill(j[None] > c + t[:, None], -math.inf), -1)
        outs.append(torch.einsum("hgij,jhd->ihgd", x, v).flatten(1, 2))
    if case["op"] == "append":
        return torch.cat(out_k), torch.cat(out_v)
    return torch.cat(outs)


def _turn(x, pos0):
    """x [rows, heads, d] at positions pos0.., pairs (i, i + d/2) as complex numbers."""
    h = x.shape[2] // 2
    f = THETA ** (-torch.arange(h, device=DEV, dtype=torch.float64) / h)
    a = torch.outer(torch.arange(pos0, pos0 + x.shape[0], device=DEV, dtype=torch.float64), f)[:, None]
    z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(torch.ones_like(a), a)
    return torch.cat((z.real, z.imag), 2)


def _blocks(x):
    """x [rows, heads, d] as codes [blocks, PAGE, heads, d] and scales [blocks, 1, heads, 1]."""
    x = torch.cat((x, x.new_zeros(-x.shape[0] % PAGE, *x.shape[1:]))).unflatten(0, (-1, PAGE))
    s = x.abs().amax((1, 3), keepdim=True) / 127
    return (x / s).nan_to_num(0).round(), s


def _extend(q, s, x, pos):
    """The block that holds `pos` and those behind it after x was appended at `pos`: values [rows, heads, d]."""
    r = pos % PAGE
    if not r:
        q, s = _blocks(x)
        return (q * s).flatten(0, 1)[:x.shape[0]]
    old, so = q[pos // PAGE, :r], s[pos // PAGE]
    head = x[:PAGE - r]
    sn = torch.maximum(so, head.abs().amax((0, 2), keepdim=True) / 127)
    first = torch.cat(((old * so / sn).round(), (head / sn).round())) * sn
    q, s = _blocks(x[PAGE - r:])
    return torch.cat((first, (q * s).flatten(0, 1)[:max(0, x.shape[0] - (PAGE - r))]))
