"""Cases of the decoder-layer operators around the rotated W8A8 linear: the norm that feeds it, the append into
a paged 4-bit attention cache, and the attention that reads that cache.

`run` computes an operator in its plain form (elementary torch operations in f32), or, where `own` is true, through
the library's entry points.  The formats both follow:

  norm     h' = h + x rounded to the type of x; n = h' / sqrt(mean(h'^2) + eps) * gamma; n~ = n rotated per 128
           by the unnormalised Hadamard matrix; s = amax |n~| / 127; codes = rne(n~ / s).
  append   k and q are turned by their position's angles (a table of cosines and sines), then k, v and q are rotated
           per 128 (q times 2^-7, which undoes H.H^T = 128 I in q.k); k and v are kept as e2m1 codes (levels
           0, .5, 1, 1.5, 2, 3, 4, 6 and a sign bit) with s = f16(amax / 6) per token and head.
  attn     o = softmax(sm_scale * q.k) v over the tokens that a row sees.

Cache layout: k_codes [pages][heads][page][D/2] (element 2j in byte j's low nibble, 2j + 1 in its high one),
v_codes [pages][heads][page/8][D][4] (byte j holds tokens 2j and 2j + 1 of the octet), scales f16
[pages][heads][page].  Sequence b owns rows q_start[b] .. q_start[b + 1] of q, k, v and o: its last tokens of
seq_len[b].
"""
import functools
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------------------ cases --

def _norm(name, dtype, M, K):
    return {"name": name, "op": "norm", "dtype": dtype, "M": M, "K": K}


def _append(name, dtype, B, n, ragged, ctx, q_heads=40, heads=8, D=128, page=64, rot=128, style=0):
    return {"name": name, "op": "append", "dtype": dtype, "B": B, "n": n, "ragged": ragged, "ctx": ctx,
            "q_heads": q_heads, "heads": heads, "D": D, "page": page, "rot": rot, "style": style,
            "rotate": D % 128 == 0}


def _attn(name, dtype, B, n, ragged, ctx, q_heads=40, heads=8, D=128, page=64, causal=True, window=0):
    return {"name": name, "op": "attn", "dtype": dtype, "B": B, "n": n, "ragged": ragged, "ctx": ctx,
            "q_heads": q_heads, "heads": heads, "D": D, "page": page, "causal": causal, "window": window}


def listed():
    return [
        # one decoded token in front of a trunk linear of 5120 inputs: a call that latency bounds
        _norm("norm_decode", "f32", 1, 5120),
        # 8 sequences x 16-token draft block, activations kept in bf16 between the layers
        _norm("norm_verify", "bf16", 128, 5120),
        # an 8K-token prefill
        _norm("norm_prefill", "f32", 8192, 5120),
        # one new token for each of 8 sequences, up to 200K tokens into them (40 query and 8 KV heads of 128)
        _append("append_decode", "f32", 8, 1, False, 200000),
        # 8 ragged draft blocks of up to 16 tokens, angles on adjacent pairs of half the head
        _append("append_verify", "bf16", 8, 16, True, 30000, rot=64, style=1),
        # an 8K-token prefill of one sequence behind an odd prefix
        _append("append_prefill", "f32", 1, 8192, False, 37),
        # one token over a short context: latency again
        _attn("attn_short", "f32", 1, 1, False, 996),
        # one token over the 200K-token context
        _attn("attn_200k", "f32", 1, 1, False, 199999),
        # 64 decoding sequences of very different lengths
        _attn("attn_batch", "bf16", 64, 1, False, 16000),
        # 8 sequences x 16-token draft block over 8K-token contexts
        _attn("attn_verify", "bf16", 8, 16, False, 8192),
        # an 8K-token prefill
        _attn("attn_prefill", "bf16", 1, 8192, False, 0),
        # chunks of four ragged prompts in a model of 64-wide heads with a sliding window
        _attn("attn_window", "f16", 4, 1500, True, 9000, q_heads=32, heads=4, D=64, page=32, window=4096),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "append", "attn", "attn"))
    dtype = rng.choice(("f32", "bf16", "f16"))
    if op == "norm":
        c = _norm("", dtype, _log(rng, 1, 8192), 128 * _log(rng, 1, 160))
        c["M"] = max(1, min(c["M"], 8192 * 5120 // c["K"]))
    else:
        D = rng.choice((64, 128, 128, 256))
        heads = rng.choice((1, 2, 4, 8, 8))
        q_heads = heads * rng.randint(1, 8)
        page = rng.choice((32, 64, 128))
        shape = rng.choice(("decode", "block", "prompt"))
        n = {"decode": 1, "block": rng.randint(2, 32), "prompt": _log(rng, 33, 4096)}[shape]
        most = {"append": 8192, "attn": 4096}[op]
        B = max(1, min(_log(rng, 1, 64), most // n))
        if op == "append":
            c = _append("", dtype, B, n, n > 1 and rng.random() < 0.6, _log(rng, 1, 200000), q_heads, heads, D, page,
                        rng.choice((D, D, D // 2)), rng.randint(0, 1))
        else:
            # every (row, head) pair meets the whole context: hold their product under the largest listed case's
            room = 8192 * 8192 * 40 // 2 * 128 // (B * n * q_heads * D) - n
            ctx = _log(rng, 1, max(2, min(200000 // B, room)))
            c = _attn("", dtype, B, n, n > 1 and rng.random() < 0.6, ctx, q_heads, heads, D, page,
                      rng.random() < 0.8, rng.choice((0, 0, 0, _log(rng, 16, 8192))))
    del c["name"]
    return c


def _lengths(c):
    """New tokens and cached tokens before them, of each sequence: of the case alone, not of a seed."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    if c["B"] == 1:
        return [c["n"]], [c["ctx"]]
    new = [r.randint(0, c["n"]) if c["ragged"] else c["n"] for _ in range(c["B"])]
    new[0] = c["n"]
    return new, [r.randint(c["ctx"] // 16, c["ctx"]) for _ in range(c["B"])]


# ----------------------------------------------------------------------------------------------- inputs --

def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "norm":
        _prepare_norm(s, c, g)
    elif c["op"] == "append":
        _prepare_append(s, c, g)
    else:
        _prepare_attn(s, c, g)
    if own:
        _handles(s)
    return s


def _activations(shape, g):
    """Normal values with 1% outliers x20, as the repository's workloads draw them."""
    x = torch.randn(shape, generator=g, device=DEV)
    return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.01, 20 * x, x)


def _prepare_norm(s, c, g):
    M, K, dt = c["M"], c["K"], DTYPES[c["dtype"]]
    s["x"] = torch.randn((M, K), generator=g, device=DEV).to(dt)
    s["h"] = _activations((M, K), g).to(dt)
    s["gamma"] = 1 + 0.2 * torch.randn((K,), generator=g, device=DEV)
    # output buffers, as a serving program keeps them
    s["h_out"] = torch.empty_like(s["h"])
    s["q"] = torch.empty((M, K), dtype=torch.int8, device=DEV)
    s["scale"] = torch.empty((M,), device=DEV)


def _prepare_batch(s, c, g, fixed=None):
    """q_start, seq_len and a block table over shuffled pages.  `fixed`: pages before the first new token all
    stand for one shared page (an append never touches them)."""
    new, ctx = _lengths(c)
    page, B = c["page"], c["B"]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s["T"] = start[-1]
    s["seq_len"] = torch.tensor([a + b for a, b in zip(new, ctx)], dtype=torch.int32, device=DEV)
    s["q_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
    first = [a // page if fixed else 0 for a in ctx]
    last = [(a + b + page - 1) // page for a, b in zip(new, ctx)]
    width = max(1, max(last))
    pages = 1 + sum(max(0, z - a) for a, z in zip(first, last))
    order = 1 + torch.randperm(pages - 1, generator=g, device=DEV).to(torch.int32) if pages > 1 else None
    table = torch.zeros((B, width), dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        k = max(0, last[b] - first[b])
        if k:
            table[b, first[b]:last[b]] = order[at:at + k]
        at += k
    s["block_table"], s["pages"], s["max_q"] = table, pages, max(new)


def _prepare_append(s, c, g):
    _prepare_batch(s, c, g, fixed=True)
    dt, T, H, D, page = DTYPES[c["dtype"]], s["T"], c["heads"], c["D"], c["page"]
    # q, k and v are columns of one projection's output, as the fused linear writes them
    qkv = torch.randn((T, c["q_heads"] + 2 * H, D), generator=g, device=DEV)
    qkv *= torch.exp(torch.rand((T, c["q_heads"] + 2 * H, 1), generator=g, device=DEV) * 2 - 1)
    qkv[..., 3] *= 8                                        # an outlier channel
    qkv = qkv.to(dt)
    s["q"], s["k"], s["v"] = qkv.split([c["q_heads"], H, H], dim=1)
    rows, half = int(s["block_table"].shape[1]) * page, c["rot"] // 2
    freq = 1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * freq
    s["rope"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    s["k_codes"] = torch.zeros((s["pages"], H, page, D // 2), dtype=torch.uint8, device=DEV)
    s["v_codes"] = torch.zeros((s["pages"], H, page // 8, D, 4), dtype=torch.uint8, device=DEV)
    s["k_scale"] = torch.zeros((s["pages"], H, page), dtype=torch.float16, device=DEV)
    s["v_scale"] = torch.zeros((s["pages"], H, page), dtype=torch.float16, device=DEV)
    s["q_out"] = torch.empty((T, c["q_heads"], D), dtype=dt, device=DEV)


def _prepare_attn(s, c, g):
    _prepare_batch(s, c, g)
    H, D, page, n = c["heads"], c["D"], c["page"], s["pages"]
    k = torch.randn((n, H, page, D), generator=g, device=DEV)
    k *= torch.exp(torch.rand((n, H, page, 1), generator=g, device=DEV) - 0.5)
    kc, s["k_scale"] = _quantise(k)
    s["k_codes"] = _pack(kc)
    del k, kc
    v = torch.randn((n, H, page, D), generator=g, device=DEV) + 0.25
    v *= torch.exp(torch.rand((n, H, page, 1), generator=g, device=DEV) * 2 - 1)
    vc, s["v_scale"] = _quantise(v)
    del v
    s["v_codes"] = _pack(vc.view(n, H, page // 8, 8, D).transpose(3, 4).contiguous())
    s["q"] = (2 * torch.randn((s["T"], c["q_heads"], D), generator=g, device=DEV)).to(DTYPES[c["dtype"]])
    s["o"] = torch.empty_like(s["q"])


def _handles(s):
    """What a program that uses the library keeps beside its tensors."""
    from rotated_w8a8_int8_amd import binding as B
    if "k_codes" in s:
        s["cache"] = B.KV4Cache(s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"])
        s["batch"] = B.KVBatch(s["block_table"], s["seq_len"], s["q_start"] if s["max_q"] != 1 else None,
                               rows=s["T"], max_q=s["max_q"])


# ------------------------------------------------------------------------------------- one pass through --

def run(s):
    return {"norm": _run_norm, "append": _run_append, "attn": _run_attn}[s["case"]["op"]](s)


def _run_norm(s):
    if own:
        from rotated_w8a8_int8_amd import binding as B
        q, scale, h = B.add_rmsnorm_quant_i8(s["x"], s["gamma"], s["h"], eps=EPS, q=s["q"], scale=s["scale"],
                                             residual_out=s["h_out"])
    else:
        h = (s["h"].float() + s["x"].float()).to(s["x"].dtype)
        f = h.float()
        n = f * torch.rsqrt(f.square().mean(dim=1, keepdim=True) + EPS) * s["gamma"]
        n = _rotate(n)
        scale = n.abs().amax(dim=1) / 127
        q = torch.where(scale[:, None] > 0, torch.round(n / scale[:, None]), 0).clamp(-127, 127)
    values = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    return h, torch.mul(q, scale[:, None], out=values), scale


def _run_append(s):
    c = s["case"]
    if own:
        from rotated_w8a8_int8_amd import binding as B
        q = B.kv4_append(s["cache"], s["batch"], s["k"], s["v"], s["q"], rope=s["rope"], rope_style=c["style"],
                         rotate=c["rotate"], q_out=s["q_out"])
        return (q, *B.kv4_read(s["cache"], s["batch"]))
    page, H, D = c["page"], c["heads"], c["D"]
    row = torch.arange(s["T"], device=DEV)
    b = (row[:, None] >= s["q_start"][None, 1:]).sum(dim=1)
    pos = s["seq_len"][b] - s["q_start"][b + 1] + row
    q, k, v = _turn(s["q"].float(), s["rope"][pos], c), _turn(s["k"].float(), s["rope"][pos], c), s["v"].float()
    if c["rotate"]:
        q, k, v = _rotate(q) * 2.0 ** -7, _rotate(k), _rotate(v)
    at, off = s["block_table"][b, pos // page].long(), pos % page
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    s["k_codes"][at, :, off] = _pack(kc)
    s["k_scale"][at, :, off] = ks
    s["v_scale"][at, :, off] = vs
    # a token's codes are one nibble of each of D dwords: add what the nibble changes by (exact modulo 2^32)
    words = s["v_codes"].view(torch.int32).view(-1)
    head, dim = torch.arange(H, device=DEV)[:, None], torch.arange(D, device=DEV)
    word = (((at * H)[:, None, None] + head) * (page // 8) + (off // 8)[:, None, None]) * D + dim
    shift = (4 * (off % 8))[:, None, None]
    change = (vc.to(torch.int64) - ((words[word] >> shift) & 15)) << shift
    words.index_add_(0, word.view(-1), change.view(-1).to(torch.int32))
    back = (words[word] >> shift) & 15
    return (q.to(s["q"].dtype), (_values(_unpack(s["k_codes"][at, :, off]), s["k_scale"][at, :, off])).bfloat16(),
            _values(back, s["v_scale"][at, :, off]).bfloat16())


def _run_attn(s):
    c = s["case"]
    if own:
        from rotated_w8a8_int8_amd import binding as B
        return B.attn_kv4(s["cache"], s["batch"], s["q"], sm_scale=c["D"] ** -0.5, causal=c["causal"],
                          window=c["window"], o=s["o"])
    B, H, D, G = c["B"], c["heads"], c["D"], c["q_heads"] // c["heads"]
    k, v = _gather(s, c)                                            # [B][H][L][D]
    i = torch.arange(s["max_q"], device=DEV)
    row = (s["q_start"][:-1, None] + i).clamp(max=s["T"] - 1).long()    # [B][max_q], padded
    new = s["q_start"][1:] - s["q_start"][:-1]
    q = s["q"].float()[row].view(B, -1, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    score = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(B, H, G, s["max_q"], -1)
    t, pos = torch.arange(k.shape[2], device=DEV), (s["seq_len"] - new)[:, None] + i
    sees = (t < s["seq_len"][:, None, None]) & ((t <= pos[:, :, None]) if c["causal"] else (t >= 0))
    if c["window"]:
        sees = sees & (t > pos[:, :, None] - c["window"])
    score.masked_fill_(~sees[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    p = score.sub_(torch.where(top > -math.inf, top, 0)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(B, H, -1, k.shape[2]), v).view(B, H, G, s["max_q"], D)
    o = torch.where(total > 0, o / total, 0).permute(0, 3, 1, 2, 4).reshape(B, s["max_q"], -1, D)
    at = torch.arange(s["T"], device=DEV)
    b = (at[:, None] >= s["q_start"][None, 1:]).sum(dim=1)
    return o[b, at - s["q_start"][b]].to(s["q"].dtype)


# ------------------------------------------------------------------------------- parts of the plain form --

def _butterfly(x, h):
    x = x.view(*x.shape[:-1], -1, 2, h) if x.shape[-1] != 2 * h else x.view(*x.shape[:-1], 1, 2, h)
    a, b = x[..., 0, :], x[..., 1, :]
    return torch.stack([a + b, a - b], dim=-2).flatten(-3)


def _rotate(x):
    """Each 128 of the last dim times the unnormalised Hadamard matrix, stage by stage."""
    return functools.reduce(_butterfly, (1, 2, 4, 8, 16, 32, 64), x.reshape(*x.shape[:-1], -1, 128)).view(x.shape)


def _turn(x, table, c):
    """Rotary angles on the first `rot` values of each head: pairs (d, d + rot/2), or (2d, 2d + 1) in style 1."""
    half = c["rot"] // 2
    cos, sin = table[:, None, :half], table[:, None, half:]
    if c["style"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., 2 * half:]], dim=-1)


def _quantise(x):
    """e2m1 codes (uint8, one a value) and f16 scales of the last dim's vectors; ties go to the even level."""
    s = (x.abs().amax(dim=-1) / 6).clamp(max=65504.0).half()
    r = torch.where(s[..., None] > 0, x / s[..., None].float(), 0)
    a = r.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8))
    return torch.where((code > 0) & (r < 0), code + 8, code), s


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(packed):
    return torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2)


def _values(code, scale):
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=DEV)
    return level[code.int()] * scale[..., None].float()


def _gather(s, c):
    """K and V of each sequence in f32 [B][heads][L][D], L the longest's tokens to a whole page."""
    B, H, D = c["B"], c["heads"], c["D"]
    at = s["block_table"].long()
    k = _values(_unpack(s["k_codes"][at]), s["k_scale"][at]).transpose(1, 2).reshape(B, H, -1, D)
    v = _unpack(s["v_codes"][at]).transpose(4, 5).reshape(B, at.shape[1], H, -1, D)
    return k, _values(v, s["v_scale"][at]).transpose(1, 2).reshape(B, H, -1, D)


# ------------------------------------------------------------------------------------------------- work --

def work(c):
    e = SIZE[c["dtype"]]
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        # x, h and gamma in, h', codes and scales out; the norm, 7 stages of sums and the codes
        return {"bytes": M * K * (3 * e + 1) + 4 * K + 4 * M, "flops": M * K * (5 + 7 + 2)}
    new, ctx = _lengths(c)
    T, H, Hq, D = sum(new), c["heads"], c["q_heads"], c["D"]
    if c["op"] == "append":
        # q, k, v and a row of angles in; q, codes and scales out, and the bf16 values these stand for
        kv = T * H * 2 * (D // 2 + 2)
        return {"bytes": T * (Hq + 2 * H) * D * e + 4 * T * c["rot"] + T * Hq * D * e + kv + 4 * T * H * D,
                "flops": T * (Hq + 2 * H) * D * 12}
    pairs = tokens = 0
    for n, before in zip(new, ctx):
        # row i (of n) stands at position before + i
        lo = [max(0, before + i + 1 - c["window"]) if c["window"] else 0 for i in range(n)]
        hi = [before + i + 1 if c["causal"] else before + n for i in range(n)]
        pairs += sum(z - a for a, z in zip(lo, hi))
        tokens += hi[-1] - lo[0] if n else 0
    return {"bytes": tokens * H * 2 * (D // 2 + 2) + 2 * T * Hq * D * e, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------------------------------- in 64 bits --

def exact(c, seed):
    with torch.no_grad():
        s = prepare(c, seed)
        return {"norm": _exact_norm, "append": _exact_append, "attn": _exact_attn}[c["op"]](s, c)


def _hadamard64(x):
    i = torch.arange(128, device=DEV)
    bits = i[:, None] & i
    sign = torch.zeros_like(bits)
    for k in range(7):
        sign ^= (bits >> k) & 1
    return (x.reshape(-1, 128) @ (1 - 2 * sign).double()).view(x.shape)


def _exact_norm(s, c):
    h = (s["h"].double() + s["x"].double()).to(s["x"].dtype)           # the sum is kept in its own type
    f = h.double()
    n = _hadamard64(f / torch.sqrt((f * f).sum(1, keepdim=True) / c["K"] + EPS) * s["gamma"].double())
    scale = n.abs().max(dim=1).values / 127
    q = torch.round(n / scale[:, None]).clamp(-127, 127)
    return h.double(), q * scale[:, None], scale


def _nearest64(x):
    """The e2m1 values of vectors under their f16 scales: among the two levels around |x| / s the nearer one, in the
    middle the one of even index."""
    s = (x.abs().max(dim=-1, keepdim=True).values / 6).clamp(max=65504.0).half().double()
    a = torch.where(s > 0, x.abs() / s.clamp(min=1e-30), 0.0)
    level = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
    up = torch.searchsorted(level, a.contiguous()).clamp(1, 7)
    low = up - 1
    over, under = level[up] - a, a - level[low]
    pick = torch.where((over < under) | ((over == under) & (up % 2 == 0)), up, low)
    return torch.sign(x) * level[pick] * s


def _exact_append(s, c):
    start, total = s["q_start"].tolist(), s["seq_len"].tolist()
    parts = []
    for b, n in enumerate(total):
        m = start[b + 1] - start[b]
        parts.append(torch.arange(n - m, n, device=DEV))
    table = s["rope"].double()[torch.cat(parts)]
    half = c["rot"] // 2
    z = torch.complex(table[:, :half], table[:, half:])[:, None]
    out = []
    for x in (s["q"].double(), s["k"].double()):
        y, r = x.clone(), x[..., :c["rot"]]
        if c["style"]:
            w = torch.view_as_complex(r.reshape(*r.shape[:-1], half, 2).contiguous()) * z
            y[..., :c["rot"]] = torch.view_as_real(w).flatten(-2)
        else:
            w = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * z
            y[..., :c["rot"]] = torch.cat([w.real, w.imag], dim=-1)
        out.append(y)
    q, k = out
    v = s["v"].double().contiguous()
    if c["rotate"]:
        q, k, v = _hadamard64(q) / 128, _hadamard64(k), _hadamard64(v)
    return q, _nearest64(k), _nearest64(v)


def _exact_attn(s, c):
    H, D, page, G = c["heads"], c["D"], c["page"], c["q_heads"] // c["heads"]
    start, total = s["q_start"].tolist(), s["seq_len"].tolist()
    signed = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64, device=DEV)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, L in enumerate(total):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        at = s["block_table"][b, :(L + page - 1) // page].long()
        q = s["q"][start[b]:start[b + 1]].double().view(n, H, G, D)
        pos = torch.arange(L - n, L, device=DEV)
        for h in range(H):
            kc, vc = s["k_codes"][at, h], s["v_codes"][at, h]
            k = torch.empty((len(at) * page, D), dtype=torch.float64, device=DEV)
            k[:, 0::2] = signed[(kc & 15).long()].view(-1, D // 2)
            k[:, 1::2] = signed[(kc >> 4).long()].view(-1, D // 2)
            k *= s["k_scale"][at, h].double().view(-1, 1)
            v = torch.empty((len(at) * page // 8, 8, D), dtype=torch.float64, device=DEV)
            for j in range(4):
                v[:, 2 * j] = signed[(vc[..., j] & 15).long()].view(-1, D)
                v[:, 2 * j + 1] = signed[(vc[..., j] >> 4).long()].view(-1, D)
            v = v.view(-1, D) * s["v_scale"][at, h].double().view(-1, 1)
            k, v = k[:L], v[:L]
            for r in range(0, n, 2048):                       # rows in pieces, for memory
                p = pos[r:r + 2048]
                w = torch.einsum("ngd,td->ngt", q[r:r + 2048, h], k) / math.sqrt(D)
                t = torch.arange(L, device=DEV)
                hide = torch.zeros((len(p), L), dtype=torch.bool, device=DEV)
                if c["causal"]:
                    hide |= t > p[:, None]
                if c["window"]:
                    hide |= t <= p[:, None] - c["window"]
                w = torch.softmax(w.masked_fill(hide[:, None], -math.inf), dim=-1)
                o[start[b] + r:start[b] + r + len(p)].view(len(p), H, G, D)[:, h] = torch.nan_to_num(w @ v)
    return o
