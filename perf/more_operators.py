"""Cases of the token mixers beside causal attention: attention for trees of drafted tokens over the paged 4-bit
cache, eviction from that cache by accumulated attention weight, and linear attention with a decay for each head.

`run` computes an operator in its plain form (elementary torch operations in f32), or, where `own` is true, through
the library's entry points:

  tree     o_i = softmax(sm_scale * q_i.k) v, row i being drafted node i of its sequence: it sees the tokens before the
           drafted ones, and those of the drafted ones whose bit is set in its mask (its ancestors and itself).  With a
           window it sees the tokens t >= base + c - window before the drafted ones, which begin at token base, c being
           the drafted tokens that it sees.
  weights  causal attention, and for each token and KV head w = factor * w + the probabilities that the last `observe`
           rows (0: every row) of its sequence gave it, summed over the query heads of the group; the call's own tokens
           begin at 0, a sequence without rows keeps its weights.
  evict    of each sequence and KV head the `budget` tokens of greatest weight, the first `first` and the last `recent`
           ones always among them, in their order, to pages of their own; returned with the cached values as they are
           read back.
  linear   S = exp(g_h) * S + k v^T, o = scale * S^T q, token by token; value head h reads key head
           h / (heads / qk_heads); S is f32 and updated in place.

Cache layout: k_codes [pages][heads][page][D/2] (element 2j in byte j's low nibble, 2j + 1 in its high one),
v_codes [pages][heads][page/8][D][4] (byte j holds tokens 2j and 2j + 1 of the octet), scales f16
[pages][heads][page].  Sequence b owns rows q_start[b] .. q_start[b + 1]: its last tokens of seq_len[b].
"""
import math
import random

import torch

own = False

DEV = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 64                      # tokens a chunk in the plain form of linear attention


# ------------------------------------------------------------------------------------------------ cases --

def _tree(name, dtype, B, n, ragged, ctx, q_heads=40, heads=8, D=128, page=64, window=0):
    return {"name": name, "op": "tree", "dtype": dtype, "B": B, "n": n, "ragged": ragged, "ctx": ctx,
            "q_heads": q_heads, "heads": heads, "D": D, "page": page, "window": window}


def _weights(name, dtype, B, n, ragged, ctx, observe=0, factor=1.0, q_heads=40, heads=8, D=128, page=64):
    return {"name": name, "op": "weights", "dtype": dtype, "B": B, "n": n, "ragged": ragged, "ctx": ctx,
            "observe": observe, "factor": factor, "q_heads": q_heads, "heads": heads, "D": D, "page": page}


def _evict(name, B, ctx, budget, first, recent, heads=8, D=128, page=64):
    return {"name": name, "op": "evict", "B": B, "n": 1, "ragged": False, "ctx": ctx, "budget": budget, "first": first,
            "recent": recent, "heads": heads, "D": D, "page": page}


def _linear(name, dtype, B, n, ragged, heads=40, qk_heads=40, D=128):
    return {"name": name, "op": "linear", "dtype": dtype, "B": B, "n": n, "ragged": ragged, "heads": heads,
            "qk_heads": qk_heads, "D": D}


def listed():
    return [
        # a small tree over a short context: a call that latency bounds
        _tree("tree_small", "f32", 1, 8, False, 500),
        # trees of up to 60 drafted tokens for each of 8 sequences, contexts of up to 16K tokens
        _tree("tree_verify", "bf16", 8, 60, True, 16000),
        # one tree over the 200K-token context
        _tree("tree_long", "bf16", 1, 64, False, 199936),
        # one decoded token, its weights added to those of the 4K tokens before it
        _weights("weights_decode", "f32", 1, 1, False, 4096),
        # 32 decoding sequences of very different lengths, older weights fading
        _weights("weights_batch", "bf16", 32, 1, False, 30000, factor=0.96875),
        # four ragged prompts in a model of 64-wide heads, observed from their last 32 rows before their first eviction
        _weights("weights_prompt", "f16", 4, 3000, True, 0, observe=32, factor=0.0, q_heads=32, heads=4, D=64, page=32),
        # a short session cut to 256 tokens a head
        _evict("evict_short", 1, 1000, 256, 4, 64),
        # 8 sessions of up to 32K tokens cut to 4096
        _evict("evict_batch", 8, 32768, 4096, 4, 512),
        # a 200K-token session cut to 16K
        _evict("evict_long", 1, 199998, 16384, 16, 1024),
        # one token of each of 64 sequences: the states pass by once
        _linear("linear_decode", "bf16", 64, 1, False),
        # an 8K-token prefill
        _linear("linear_prompt", "bf16", 1, 8192, False),
        # six ragged chunks of prompts in f32, 64-wide heads, value heads that share key heads
        _linear("linear_ragged", "f32", 6, 1500, True, heads=32, qk_heads=8, D=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tree", "weights", "evict", "linear"))
    dtype = rng.choice(("f32", "bf16", "f16"))
    D = rng.choice((64, 128, 128, 256))
    if op == "linear":
        heads = rng.choice((4, 8, 16, 32, 40))
        shape = rng.choice(("decode", "block", "prompt"))
        n = {"decode": 1, "block": rng.randint(2, 48), "prompt": _log(rng, 49, 4096)}[shape]
        B = max(1, min(_log(rng, 1, 64), 4096 // n, 64 * 40 * 128 * 128 // (heads * D * D)))
        c = _linear("", dtype, B, n, n > 1 and rng.random() < 0.6, heads, heads // rng.choice((1, 1, 2, 4)), D)
    else:
        heads = rng.choice((1, 2, 4, 8, 8))
        q_heads = heads * rng.randint(1, 8)
        page = rng.choice((32, 64, 128, 256))
        if op == "evict":
            B = _log(rng, 1, 16)
            ctx = _log(rng, 16, 199998 // B)
            budget = _log(rng, 8, max(8, min(16384, 2 * ctx // 3)))
            c = _evict("", B, ctx, budget, rng.randint(0, min(8, budget // 4)), rng.randint(0, budget // 2), heads, D, page)
        elif op == "tree":
            n = rng.randint(2, 128)
            B = _log(rng, 1, max(1, min(16, 480 // n)))
            # every (row, head) pair meets the whole context: hold their product under the largest listed case's
            room = 64 * 40 * 199936 * 128 // (B * n * q_heads * D)
            ctx = _log(rng, 1, max(2, min(199936 // B, room)))
            c = _tree("", dtype, B, n, rng.random() < 0.6, ctx, q_heads, heads, D, page, rng.choice((0, 0, _log(rng, 128, 8192))))
        else:
            n = rng.choice((1, 1, rng.randint(2, 32), _log(rng, 33, 2048)))
            B = max(1, min(_log(rng, 1, 32), 2048 // n))
            room = 64 * 40 * 199936 * 128 // (B * n * q_heads * D)
            ctx = _log(rng, 1, max(2, min(480000 // B, 100000, room)))
            c = _weights("", dtype, B, n, n > 1 and rng.random() < 0.6, ctx, rng.choice((0, 0, rng.randint(1, 64))),
                         rng.choice((0.0, 1.0, 0.9375)), q_heads, heads, D, page)
    del c["name"]
    return c


def _rng(c):
    return random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))


def _lengths(c):
    """New tokens and cached tokens before them, of each sequence: of the case alone, not of a seed."""
    r, ctx = _rng(c), c.get("ctx", 0)
    if c["B"] == 1:
        return [c["n"]], [ctx]
    new = [r.randint(0, c["n"]) if c["ragged"] else c["n"] for _ in range(c["B"])]
    new[0] = c["n"]
    return new, [r.randint(ctx // 16, ctx) for _ in range(c["B"])]


# ----------------------------------------------------------------------------------------------- inputs --

def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "linear":
        _prepare_linear(s, c, g)
    else:
        _prepare_cache(s, c, g)
        if c["op"] == "evict":
            _prepare_evict(s, c, g)
        else:
            s["q"] = (2 * torch.randn((s["T"], c["q_heads"], c["D"]), generator=g, device=DEV)).to(DTYPES[c["dtype"]])
            s["o"] = torch.empty_like(s["q"])
        if c["op"] == "tree":
            s["mask"] = _masks(c, seed)
        elif c["op"] == "weights":
            shape = (c["B"], c["heads"], s["block_table"].shape[1] * c["page"])
            s["weight"] = 4 * torch.rand(shape, generator=g, device=DEV) ** 8
        if own:
            _handles(s)
    return s


def _starts(new):
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return start


def _prepare_cache(s, c, g):
    """q_start, seq_len, a block table over shuffled pages, and a filled cache."""
    new, ctx = _lengths(c)
    H, D, page, B = c["heads"], c["D"], c["page"], c["B"]
    start = _starts(new)
    s["T"], s["max_q"] = start[-1], max(new)
    s["len"] = [a + b for a, b in zip(new, ctx)]
    s["seq_len"] = torch.tensor(s["len"], dtype=torch.int32, device=DEV)
    s["q_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
    s["block_table"], n = _table(s["len"], page, g)
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


def _table(lengths, page, g):
    count = [(n + page - 1) // page for n in lengths]
    pages, width = max(1, sum(count)), max(1, max(count))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((len(lengths), width), dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(count):
        table[b, :k] = order[at:at + k]
        at += k
    return table, pages


def _masks(c, seed):
    """A random tree a sequence: bit j of row i is set where node j is node i or an ancestor of it."""
    r = random.Random(seed)
    words = (c["n"] + 63) // 64
    rows = []
    for n in _lengths(c)[0]:
        seen = []
        for i in range(n):
            parent = -1 if i == 0 else r.randint(max(-1, i - 6), i - 1)
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        rows += seen
    words64 = [[(m >> 64 * w) & (1 << 64) - 1 for w in range(words)] for m in rows]
    signed = [[x - (1 << 64) if x >> 63 else x for x in row] for row in words64]
    return torch.tensor(signed, dtype=torch.int64, device=DEV).view(-1, words)


def _prepare_evict(s, c, g):
    B, H, budget = c["B"], c["heads"], c["budget"]
    # weights as they come of many rows: most tokens a little, a few a lot, some none at all
    u = torch.rand((B, H, s["block_table"].shape[1] * c["page"]), generator=g, device=DEV)
    s["weight"] = torch.where(u < 0.02, 0, u.pow(12) * 8)
    s["to_table"], pages = _table([min(budget, n) for n in s["len"]], c["page"], g)
    s["to"] = [torch.zeros((pages, *t.shape[1:]), dtype=t.dtype, device=DEV)
               for t in (s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"])]
    # the kept tokens as rows of a batch, to be read back
    kept = [min(budget, n) for n in s["len"]]
    s["rows"] = sum(kept)
    s["row_start"] = torch.tensor(_starts(kept), dtype=torch.int32, device=DEV)
    s["kept"] = torch.zeros((B, H, budget), dtype=torch.int32, device=DEV)
    s["kept_weight"] = torch.zeros((B, H, budget), device=DEV)
    s["count"] = torch.zeros((B,), dtype=torch.int32, device=DEV)


def _prepare_linear(s, c, g):
    new, _ = _lengths(c)
    start = _starts(new)
    T, H, K, D = start[-1], c["heads"], c["qk_heads"], c["D"]
    s["T"], s["max_q"] = T, max(new)
    s["q_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
    # q, k and v are columns of one projection's output, as the linear writes them
    qkv = torch.randn((T, 2 * K + H, D), generator=g, device=DEV)
    qkv[:, :2 * K] = torch.nn.functional.silu(qkv[:, :2 * K])
    s["q"], s["k"], s["v"] = qkv.to(DTYPES[c["dtype"]]).split([K, K, H], dim=1)
    # decays from one that forgets within a few tokens to one that holds for hundreds
    s["log_decay"] = -torch.exp2(-8 * torch.arange(1, H + 1, device=DEV) / H)
    s["state"] = torch.randn((c["B"], H, D, D), generator=g, device=DEV)
    s["o"] = torch.empty((T, H, D), dtype=DTYPES[c["dtype"]], device=DEV)


def _handles(s):
    """What a program that uses the library keeps beside its tensors."""
    from rotated_w8a8_int8_amd import binding as B
    s["cache"] = B.KV4Cache(s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"])
    s["batch"] = B.KVBatch(s["block_table"], s["seq_len"], s["q_start"] if s["max_q"] != 1 else None, rows=s["T"],
                           max_q=s["max_q"])
    if "to" in s:
        s["to_cache"] = B.KV4Cache(*s["to"])
        s["to_batch"] = B.KVBatch(s["to_table"], s["count"], s["row_start"], rows=s["rows"])


# ------------------------------------------------------------------------------------- one pass through --

def run(s):
    return {"tree": _run_tree, "weights": _run_weights, "evict": _run_evict, "linear": _run_linear}[s["case"]["op"]](s)


def _run_tree(s):
    c = s["case"]
    if own:
        from rotated_w8a8_int8_amd import binding as B
        return B.attn_kv4_tree(s["cache"], s["batch"], s["q"], s["mask"], sm_scale=c["D"] ** -0.5, window=c["window"],
                               o=s["o"])
    k, v, row, t, base = _padded(s, c)
    j = torch.arange(s["max_q"], device=DEV)
    bit = (s["mask"][row][:, :, j // 64] >> (j % 64)) & 1                             # [B][max_q][max_q]
    drafted = torch.gather(bit, 2, (t - base[:, None]).clamp(0, s["max_q"] - 1)[:, None].expand(-1, s["max_q"], -1)) > 0
    before = t < base[:, None, None]
    if c["window"]:
        before = before & (t >= base[:, None, None] + bit.sum(dim=2, keepdim=True) - c["window"])
    sees = before | (drafted & (t >= base[:, None, None]) & (t < s["seq_len"][:, None, None]))
    return _rows(s, _attend(s, c, k, v, row, sees)[0])


def _run_weights(s):
    c = s["case"]
    if own:
        from rotated_w8a8_int8_amd import binding as B
        return B.attn_kv4_weights(s["cache"], s["batch"], s["q"], s["weight"], sm_scale=c["D"] ** -0.5,
                                  observe=c["observe"], factor=c["factor"], o=s["o"])
    k, v, row, t, base = _padded(s, c)
    i = torch.arange(s["max_q"], device=DEV)
    pos, new = base[:, None] + i, s["seq_len"] - base
    sees = (t <= pos[:, :, None]) & (t < s["seq_len"][:, None, None])
    o, p = _attend(s, c, k, v, row, sees)                                              # p [B][H][G][max_q][L]
    counts = (i < new[:, None]) & ((i >= new[:, None] - c["observe"]) if c["observe"] else (i >= 0))
    given = torch.matmul(counts.float()[:, None, None, None], p).sum(dim=2)[:, :, 0]   # [B][H][L]
    old = torch.where(t < base[:, None, None], c["factor"] * s["weight"], 0) if c["factor"] else 0
    changed = (t < s["seq_len"][:, None, None]) & (new > 0)[:, None, None]
    s["weight"].copy_(torch.where(changed, old + given, s["weight"]))
    return _rows(s, o), s["weight"]


def _run_evict(s):
    c = s["case"]
    if own:
        from rotated_w8a8_int8_amd import binding as B
        B.kv4_select(s["batch"], s["weight"], c["budget"], first=c["first"], recent=c["recent"], kept=s["kept"],
                     count=s["count"], kept_weight=s["kept_weight"])
        B.kv4_move(s["cache"], s["batch"], s["kept"], s["count"], to=s["to_cache"], to_table=s["to_table"])
        return (s["kept"], s["kept_weight"], *B.kv4_read(s["to_cache"], s["to_batch"]))
    B, H, D, page, budget = c["B"], c["heads"], c["D"], c["page"], c["budget"]
    n, t = s["seq_len"][:, None, None], torch.arange(s["weight"].shape[2], device=DEV)
    always = (t < c["first"]) | (t >= n - c["recent"])
    rank = torch.where(t < n, torch.where(always, math.inf, s["weight"]), -math.inf)
    most = min(budget, rank.shape[2])
    best = rank.sort(dim=2, descending=True, stable=True).indices[:, :, :most]
    count = s["seq_len"].clamp(max=budget)
    here = torch.arange(most, device=DEV) < count[:, None, None]                       # [B][1][most]
    # shorter sequences end with places past their count: they go behind, and stay zero
    kept = torch.where(here, best, rank.shape[2]).sort(dim=2).values
    kept = torch.where(here, kept, 0)
    s["count"].copy_(count)
    s["kept"][:, :, :most] = kept.int()
    s["kept_weight"][:, :, :most] = torch.where(here, torch.gather(s["weight"], 2, kept), 0)
    b, h = torch.arange(B, device=DEV)[:, None, None], torch.arange(H, device=DEV)[:, None]
    at, off = s["block_table"][b, kept // page].long(), kept % page                    # [B][H][most]
    kc, ks, vs = s["k_codes"][at, h, off], s["k_scale"][at, h, off], s["v_scale"][at, h, off]
    words = s["v_codes"].view(torch.int32)[..., 0][at, h, off // 8]                    # [B][H][most][D]
    vc = ((words >> (4 * (off % 8))[..., None]) & 15).to(torch.uint8)
    # into their new pages: whole octets of values
    width = s["to_table"].shape[1] * page
    pad = (0, 0, 0, width - most)
    fill = [torch.nn.functional.pad(x, pad[-2 * (x.dim() - 2):]).view(B, H, -1, page, *x.shape[3:]).transpose(1, 2)
            for x in (kc, ks, vc, vs)]
    fill[2] = _pack(fill[2].reshape(B, -1, H, page // 8, 8, D).transpose(4, 5).contiguous())
    real = (torch.arange(s["to_table"].shape[1], device=DEV) * page < count[:, None]).view(-1).nonzero()[:, 0]
    for to, x in zip(s["to"], fill):
        to[s["to_table"].view(-1)[real].long()] = x.flatten(0, 1)[real]
    pick = here[:, 0].reshape(-1).nonzero()[:, 0]
    rows = [_values(x, y).bfloat16().transpose(1, 2).reshape(-1, H, D)[pick] for x, y in ((_unpack(kc), ks), (vc, vs))]
    return s["kept"], s["kept_weight"], rows[0], rows[1]


def _run_linear(s):
    c = s["case"]
    if own:
        from rotated_w8a8_int8_amd import binding as B
        o, state = B.linear_attn(s["q"], s["k"], s["v"], s["log_decay"], state=s["state"], state_out=s["state"],
                                 q_start=s["q_start"] if s["max_q"] != 1 else None, max_q=s["max_q"],
                                 scale=c["D"] ** -0.5, o=s["o"])
        return o, state
    B, H, D, each = c["B"], c["heads"], c["D"], c["heads"] // c["qk_heads"]
    C = min(CHUNK, s["max_q"])
    N = (s["max_q"] + C - 1) // C
    i = torch.arange(N * C, device=DEV)
    new = s["q_start"][1:] - s["q_start"][:-1]
    row = (s["q_start"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    real = (i < new[:, None])[:, :, None, None]
    # [B][H][N][C][D]; rows past a sequence's end are zero and do not decay
    q, k, v = (torch.where(real, x[row].float(), 0).repeat_interleave(H // x.shape[2 - 1], dim=2)
               .view(B, N, C, H, D).permute(0, 3, 1, 2, 4) for x in (s["q"], s["k"], s["v"]))
    steps = torch.minimum(i + 1, new[:, None]).view(B, 1, N, C).float()                # tokens up to and with this one
    g = s["log_decay"][:, None, None]
    first = (torch.arange(N, device=DEV) * C).view(1, 1, N, 1)
    begin = torch.minimum(first, new[:, None, None, None]).float()                     # tokens before the chunk
    end = steps[..., -1:]
    age = steps[..., :, None] - steps[..., None, :]
    decay = torch.where(torch.ones((C, C), dtype=torch.bool, device=DEV).tril(), torch.exp(g[..., None] * age), 0)
    inside = torch.matmul(torch.matmul(q, k.transpose(3, 4)) * decay, v)
    new_part = torch.matmul((k * torch.exp(g * (end - steps))[..., None]).transpose(3, 4), v)   # [B][H][N][D][D]
    # the state before chunk n (n = N: at the end): the first state and the chunks before n, each aged to there
    ends = torch.cat([begin[..., 0], end[:, :, -1]], dim=2)                            # [B][1][N + 1] tokens before
    since = (ends[..., :, None] - ends[..., None, :]).clamp(min=0)
    by = torch.exp(g * since) * torch.ones((N + 1, N + 1), device=DEV).tril()
    parts = torch.cat([s["state"][:, :, None], new_part], dim=2).flatten(3)            # [B][H][N + 1][D * D]
    states = torch.matmul(by, parts).view(B, H, N + 1, D, D)
    across = torch.matmul(q * torch.exp(g * (steps - begin))[..., None], states[:, :, :-1])
    s["state"].copy_(states[:, :, -1])
    o = ((inside + across) * D ** -0.5).permute(0, 2, 3, 1, 4).reshape(B, N * C, H, D)
    return _rows(s, o.to(s["q"].dtype)), s["state"]


# ------------------------------------------------------------------------------- parts of the plain form --

def _padded(s, c):
    """K and V of each sequence in f32 [B][heads][L][D], L the longest's tokens to a whole page; the row of each
    sequence's i-th query; the tokens; the token of each sequence's first row."""
    B, H, D = c["B"], c["heads"], c["D"]
    at = s["block_table"].long()
    k = _values(_unpack(s["k_codes"][at]), s["k_scale"][at]).transpose(1, 2).reshape(B, H, -1, D)
    v = _unpack(s["v_codes"][at]).transpose(4, 5).reshape(B, at.shape[1], H, -1, D)
    v = _values(v, s["v_scale"][at]).transpose(1, 2).reshape(B, H, -1, D)
    i = torch.arange(s["max_q"], device=DEV)
    row = (s["q_start"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    return k, v, row, torch.arange(k.shape[2], device=DEV), s["seq_len"] - (s["q_start"][1:] - s["q_start"][:-1])


def _attend(s, c, k, v, row, sees):
    """Outputs [B][max_q][q_heads][D] and probabilities [B][heads][G][max_q][L]."""
    B, H, D, G = c["B"], c["heads"], c["D"], c["q_heads"] // c["heads"]
    q = s["q"].float()[row].view(B, -1, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    score = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(B, H, G, s["max_q"], -1)
    score.masked_fill_(~sees[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    p = score.sub_(torch.where(top > -math.inf, top, 0)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p = p.mul_(torch.where(total > 0, 1 / total, 0))
    o = torch.matmul(p.view(B, H, -1, k.shape[2]), v).view(B, H, G, s["max_q"], D)
    return o.permute(0, 3, 1, 2, 4).reshape(B, s["max_q"], -1, D).to(s["q"].dtype), p


def _rows(s, padded):
    """[B][max_q or more][..] back to the call's rows."""
    at = torch.arange(s["T"], device=DEV)
    b = (at[:, None] >= s["q_start"][None, 1:]).sum(dim=1)
    return padded[b, at - s["q_start"][b]]


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


# ------------------------------------------------------------------------------------------------- work --

def work(c):
    new, ctx = _lengths(c)
    T, H, D = sum(new), c["heads"], c["D"]
    if c["op"] == "linear":
        e = SIZE[c["dtype"]]
        # q, k and v in, o out, the states in and out; their update and the product with q, token by token
        return {"bytes": T * (2 * c["qk_heads"] + 2 * H) * D * e + 8 * c["B"] * H * D * D, "flops": 4 * T * H * D * D}
    if c["op"] == "evict":
        tokens, kept = sum(a + b for a, b in zip(new, ctx)), sum(min(c["budget"], a + b) for a, b in zip(new, ctx))
        # the weights in; the kept tokens' codes and scales in and out; their list, weights and values out
        return {"bytes": H * (4 * tokens + kept * (4 * (D // 2 + 2) + 8 + 4 * D)), "flops": H * tokens}
    e, Hq, n_w = SIZE[c["dtype"]], c["q_heads"], 0
    tokens = pairs = 0
    for n, before in zip(new, ctx):
        w = c.get("window", 0)
        tokens += (min(before, w) if w else before) + n if n else 0
        # about half of a chain's, and all of a tree's, own tokens
        pairs += n * (min(before, w) if w else before) + (n * (n + 1) // 2)
        n_w += before + n
    bytes_ = tokens * H * 2 * (D // 2 + 2) + 2 * T * Hq * D * e
    if c["op"] == "tree":
        return {"bytes": bytes_ + 8 * T * ((c["n"] + 63) // 64), "flops": 4 * D * Hq * pairs}
    # the weights in (where they count) and out
    return {"bytes": bytes_ + n_w * H * (8 if c["factor"] else 4), "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------------------------------- in 64 bits --

def exact(c, seed):
    with torch.no_grad():
        s = prepare(c, seed)
        return {"tree": _exact_attn, "weights": _exact_attn, "evict": _exact_evict, "linear": _exact_linear}[c["op"]](s, c)


def _cached64(s, b, h, L, page, D):
    """Keys and values of tokens 0 .. L - 1 of one sequence and head."""
    signed = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64, device=DEV)
    at = s["block_table"][b, :(L + page - 1) // page].long()
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
    return k[:L], v[:L]


def _exact_attn(s, c):
    H, D, page, G = c["heads"], c["D"], c["page"], c["q_heads"] // c["heads"]
    start = s["q_start"].tolist()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    weight = s["weight"].double() if c["op"] == "weights" else None
    for b, L in enumerate(s["len"]):
        n = start[b + 1] - start[b]
        base, t = L - n, torch.arange(L, device=DEV)
        if n == 0:
            continue
        if c["op"] == "weights":
            weight[b, :, :base] *= c["factor"]
            weight[b, :, base:L] = 0
        q = s["q"][start[b]:start[b + 1]].double().view(n, H, G, D)
        if c["op"] == "tree":
            bits = s["mask"][start[b]:start[b + 1]].tolist()
            hide = torch.zeros((n, L), dtype=torch.bool)
            for i, words in enumerate(bits):
                path = [j for j in range(n) if words[j // 64] >> (j % 64) & 1]
                hide[i, base:] = True
                hide[i, [base + j for j in path]] = False
                if c["window"]:
                    hide[i, :max(0, base + len(path) - c["window"])] = True
            hide = hide.to(DEV)
        for h in range(H):
            k, v = _cached64(s, b, h, L, page, D)
            for r in range(0, n, 1024):                                               # rows in pieces, for memory
                z = min(r + 1024, n)
                w = (q[r:z, h].reshape(-1, D) @ k.t()).view(z - r, G, L) / math.sqrt(D)
                if c["op"] == "tree":
                    gone = hide[r:z]
                else:
                    gone = t > base + torch.arange(r, z, device=DEV)[:, None]
                p = torch.nan_to_num(torch.softmax(w.masked_fill(gone[:, None], -math.inf), dim=-1))
                o[start[b] + r:start[b] + z].view(z - r, H, G, D)[:, h] = (p.view(-1, L) @ v).view(z - r, G, D)
                if c["op"] == "weights":
                    seen = n - c["observe"] if c["observe"] else 0
                    weight[b, h, :L] += p[max(0, seen - r):].sum(dim=(0, 1))
    return o if c["op"] == "tree" else (o, weight)


def _exact_evict(s, c):
    B, H, D, page = c["B"], c["heads"], c["D"], c["page"]
    kept = torch.zeros((B, H, c["budget"]), dtype=torch.int32, device=DEV)
    kept_weight = torch.zeros((B, H, c["budget"]), dtype=torch.float64, device=DEV)
    keys, values = [], []
    for b, L in enumerate(s["len"]):
        n = min(L, c["budget"])
        free = torch.arange(min(c["first"], L), max(L - c["recent"], min(c["first"], L)), device=DEV)
        outer = torch.tensor([t for t in range(L) if t < c["first"] or t >= L - c["recent"]], dtype=torch.int64, device=DEV)
        k_b, v_b = [], []
        for h in range(H):
            if n < L:
                w = s["weight"][b, h, free].double()
                order = torch.argsort(-w, stable=True)[:n - len(outer)]
                at = torch.cat([outer, free[order]]).sort().values
            else:
                at = torch.arange(L, device=DEV)
            kept[b, h, :n] = at.int()
            kept_weight[b, h, :n] = s["weight"][b, h, at].double()
            k, v = _cached64(s, b, h, L, page, D)
            k_b.append(k[at])
            v_b.append(v[at])
        keys.append(torch.stack(k_b, dim=1))
        values.append(torch.stack(v_b, dim=1))
    return kept, kept_weight, torch.cat(keys), torch.cat(values)


def _exact_linear(s, c):
    H, D = c["heads"], c["D"]
    start, decay = s["q_start"].tolist(), s["log_decay"].double()
    state, o = s["state"].double(), torch.zeros((s["T"], H, D), dtype=torch.float64, device=DEV)
    of = torch.arange(H, device=DEV) // (H // c["qk_heads"])
    if s["max_q"] == 1:                                                                # a token of each sequence
        q, k, v = s["q"].double()[:, of], s["k"].double()[:, of], s["v"].double()
        state = state * torch.exp(decay)[:, None, None] + k[..., None] * v[:, :, None]
        return (state * q[..., None]).sum(dim=2) / math.sqrt(D), state
    for b in range(c["B"]):
        for r in range(start[b], start[b + 1], 256):                                  # blocks of rows, the state between
            z = min(r + 256, start[b + 1])
            q, k, v = (x[r:z].double().transpose(0, 1) for x in (s["q"], s["k"], s["v"]))
            q, k = q[of], k[of]                                                        # [H][m][D]
            i = torch.arange(z - r, device=DEV, dtype=torch.float64)
            w = torch.bmm(q, k.transpose(1, 2).contiguous())
            w = w * torch.exp(decay[:, None, None] * (i[:, None] - i).clamp(min=0)) * (i[:, None] >= i)
            y = torch.bmm(w, v.contiguous())
            y += torch.bmm(q, state[b]) * torch.exp(decay[:, None] * (i + 1))[..., None]
            o[r:z] = y.transpose(0, 1) / math.sqrt(D)
            aged = k * torch.exp(decay[:, None] * (z - r - 1 - i))[..., None]
            state[b] = state[b] * torch.exp(decay * (z - r))[:, None, None] + torch.bmm(aged.transpose(1, 2).contiguous(), v.contiguous())
    return o, state
