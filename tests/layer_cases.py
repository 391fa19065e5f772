"""Inputs and comparisons shared by the GPU tests of the calls between a layer's linears."""
import numpy as np

from oracle import layer as O
from rotated_w8a8_int8_amd import binding as B

DTYPES = ("f32", "bf16", "f16")


def torch_dtype(torch, dtype):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]


def put(torch, a, dtype=None):
    """A host array on the GPU; `dtype` f32, bf16 or f16 for values (given as f32, already representable)."""
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(torch_dtype(torch, dtype))


def host(t):
    return t.float().cpu().numpy()


def ragged(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def page_table(rng, seq_len, page, width=None, spare=2):
    """Distinct shuffled pages for every sequence, -1 where it needs none, and the number of pages."""
    need = [(int(n) + page - 1) // page for n in seq_len]
    width = max(1, max(need, default=1)) if width is None else width
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    table, at = np.full((len(need), width), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def device_cache(torch, c):
    return B.KV4Cache(put(torch, c.k_codes), put(torch, c.k_scale), put(torch, c.v_codes), put(torch, c.v_scale))


def device_batch(torch, table, seq_len, q_start, rows, max_q=None):
    return B.KVBatch(put(torch, table), put(torch, np.asarray(seq_len, np.int32)),
                     None if q_start is None else put(torch, q_start), rows=rows, max_q=max_q)


def rope_table(rows, dim, base=1e6):
    half = dim // 2
    ang = np.arange(rows, dtype=np.float64)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def fill_cache(rng, c, table, seq_len, k_size=1.0, heavy=True):
    """Quantised normal keys and values in every token of every sequence; what lies past a length stays stale."""
    for b, n in enumerate(seq_len):
        for p in range((int(n) + c.page - 1) // c.page):
            page, lo = int(table[b, p]), p * c.page
            m = min(int(n), lo + c.page) - lo
            if not 0 <= page < c.pages:
                continue
            for t in range(m):
                k = rng.standard_normal((c.heads, c.D)) * k_size * np.exp(rng.uniform(-0.5, 0.5, (c.heads, 1)))
                v = (rng.standard_normal((c.heads, c.D)) + 0.25) * np.exp(rng.uniform(-1, 1, (c.heads, 1)))
                c.put(page, t, O.quantise_f32(k.astype(np.float32)), O.quantise_f32(v.astype(np.float32)))


def attention_tolerance(dtype, out, mass, reach, n_tokens):
    """How far an output may be from the 64-bit one, element by element.

    reach = max_t sm_scale sum_d |q_d k_d|: a query element enters the products with a relative error of at most
    2^-16 (f32: two 16-bit parts) or 0 (bf16 and f16 queries are taken
    exactly), the products are exact, the f32 sum of D of them rounds at most D times (D <= 256: 2^-16), and three more
    f32 roundings (scales, exponent) count 2^-22: a score is off by at most e = 2^-14.9 reach < 2^-14 reach, and
    every probability by a factor of at most exp(2 e) (its own score and the normaliser's).  The weight p * scale enters
    with 2^-16 (f32, two parts) or 2^-8 (one 16-bit part), exp2 and its products with 2^-21, and the f32 sum over n tokens, in
    partial sums, rounds at most 2 sqrt(n) + 64 times to first order (tiles of tokens, splits, waves).  The division and the
    output's own rounding end it.  Weights are f16 (f32: a sum of two) on a scale that puts the row's largest weight so
    far at 2^3 or more, so each is off by up to f16's smallest step, 2^-24, in itself: 2^-27 of the largest, whose token
    has a value of the highest level, 6, in some dimension, and thus n 2^-27 of the row's largest mass for n tokens.  All are relative to mass = sum_t p_t |v_t|.  An f16 output below 2^-14 is a multiple of
    2^-24, so its rounding is off by up to 2^-25 however small the value (f32 and bf16 reach down to 2^-126: 1e-30 covers
    them).
    """
    e = 2.0 ** -14 * reach[..., None]
    weight = (2.0 ** -16 if dtype == "f32" else 2.0 ** -8) + 2.0 ** -21 + (2 * np.sqrt(n_tokens) + 64) * 2.0 ** -24
    least = n_tokens * 2.0 ** -27 * np.max(mass, axis=-1, keepdims=True)
    return (np.expm1(2 * e) + 2 * weight) * mass + (O.EPS[dtype] / 2 + 2.0 ** -22) * np.abs(out) + least + (2.0 ** -25 if dtype == "f16" else 1e-30)
