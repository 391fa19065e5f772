"""CPU oracle of the calls between a layer's linears: the norm that feeds them, the paged 4-bit cache and its
attention.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it imports nothing from the GPU library.  Plain NumPy in
64 bits, written from the definitions in include/rad.h.  Where a call defines its f32 operations one by one (the
append's angles, rotation, scale and codes) ``append_f32`` does those operations in that order; everything else
is f64.
"""
from __future__ import annotations

import numpy as np

import oracle

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_round(v):
    """The nearest bf16 values (ties to even), as f32."""
    u = np.ascontiguousarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32) << 16).view(np.float32)


def to_dtype(v, dtype):
    """f32 or f64 values rounded to 'f32', 'bf16' or 'f16', as f32."""
    v = np.asarray(v, dtype=np.float32)
    if dtype == "bf16":
        return bf16_round(v)
    return v.astype(np.float16).astype(np.float32) if dtype == "f16" else v


EPS = {"f32": 2.0 ** -23, "bf16": 2.0 ** -7, "f16": 2.0 ** -10}     # spacing at 1; a rounding is off by half


def hadamard():
    i = np.arange(128)
    return np.array([[1.0 - 2.0 * (bin(a & b).count("1") & 1) for b in i] for a in i])


def rotate(v):
    v = np.asarray(v, dtype=np.float64)
    return (v.reshape(-1, 128) @ hadamard()).reshape(v.shape)


# ------------------------------------------------------------------------------------------------ norm --

def add_rmsnorm(x, residual, gamma, eps, dtype, rot):
    """h (f32, as stored), the f64 normalised (rotated) rows, and per row the f64 sums of |n| over each 128."""
    h = x if residual is None else to_dtype(residual.astype(np.float32) + x.astype(np.float32), dtype)
    f = h.astype(np.float64)
    n = f / np.sqrt(np.mean(f * f, axis=1, keepdims=True) + eps) * gamma.astype(np.float64)
    mass = np.abs(n).reshape(len(n), -1, 128).sum(axis=2)
    return h, (rotate(n) if rot else n), mass


# ----------------------------------------------------------------------------------------------- cache --

def e2m1_codes(r):
    """Codes of quotients r: the nearest level, ties to the even index, above 6 to 6; zero without a sign."""
    a = np.abs(np.asarray(r, dtype=np.float64))
    up = np.clip(np.searchsorted(LEVELS, a), 1, 7)
    over, under = LEVELS[up] - a, a - LEVELS[up - 1]
    code = np.where((over < under) | ((over == under) & (up % 2 == 0)), up, up - 1)
    return np.where((code > 0) & (np.asarray(r) < 0), code + 8, code).astype(np.uint8)


def e2m1_values(code):
    return np.where(code & 8, -1.0, 1.0) * LEVELS[code & 7]


def quantise_f32(y):
    """Codes and f16 scales of f32 vectors (last dim), in the call's own f32 operations."""
    amax = np.max(np.abs(y), axis=-1)
    with np.errstate(over="ignore"):
        s = np.minimum((amax / np.float32(6)).astype(np.float32), np.float32(65504)).astype(np.float16)
    s32 = s.astype(np.float32)[..., None]
    r = np.divide(y, s32, out=np.zeros_like(y), where=s32 > 0)
    return e2m1_codes(r), s


def turn_f32(x, table, style):
    """Angles on f32 [rows][heads][D] by f32 table rows [rows][dim], each operation rounded to f32."""
    half = table.shape[1] // 2
    c, s = table[:, None, :half], table[:, None, half:]
    y = x.copy()
    if style:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


def rotate_f32(x):
    """The f32 butterfly network of rad_fwht128."""
    return oracle.fwht128(np.ascontiguousarray(x, dtype=np.float32).reshape(-1, x.shape[-1])).reshape(x.shape)


def append_f32(q, k, v, table, style, rot):
    """Turned queries (f32), and (codes, scales) of keys and values, of f32 rows [rows][heads][D]."""
    if table is not None:
        q, k = turn_f32(q, table, style), turn_f32(k, table, style)
    if rot:
        q, k, v = rotate_f32(q) * np.float32(2.0 ** -7), rotate_f32(k), rotate_f32(v)
    return q, quantise_f32(k), quantise_f32(v)


class Cache:
    """The paged cache in host memory, in the layouts of include/rad.h."""

    def __init__(self, pages, heads, page, D, rng=None):
        shape = (pages, heads, page, D // 2)
        self.k_codes = np.zeros(shape, np.uint8)
        self.v_codes = np.zeros((pages, heads, page // 8, D, 4), np.uint8)
        self.k_scale = np.zeros((pages, heads, page), np.float16)
        self.v_scale = np.zeros((pages, heads, page), np.float16)
        if rng is not None:                       # stale contents: any code, scales of any bits (NaN among them)
            self.k_codes[:] = rng.integers(0, 256, shape)
            self.v_codes[:] = rng.integers(0, 256, self.v_codes.shape)
            self.k_scale[:] = rng.integers(0, 65536, self.k_scale.shape).astype(np.uint16).view(np.float16)
            self.v_scale[:] = rng.integers(0, 65536, self.v_scale.shape).astype(np.uint16).view(np.float16)
        self.pages, self.heads, self.page, self.D = pages, heads, page, D

    def put(self, page, off, k, v):
        """One token: (codes, scales) [heads][D] and [heads] of its keys and values."""
        self.k_codes[page, :, off] = k[0][:, 0::2] | (k[0][:, 1::2] << 4)
        self.k_scale[page, :, off], self.v_scale[page, :, off] = k[1], v[1]
        byte, shift = (off % 8) // 2, 4 * (off % 2)
        old = self.v_codes[page, :, off // 8, :, byte]
        self.v_codes[page, :, off // 8, :, byte] = (old & (0xF0 >> shift)) | (v[0] << shift)

    def get(self, page, off):
        """Keys and values [heads][D] of one token, f64."""
        kc = self.k_codes[page, :, off]
        k = np.empty((self.heads, self.D))
        k[:, 0::2], k[:, 1::2] = e2m1_values(kc & 15), e2m1_values(kc >> 4)
        vc = (self.v_codes[page, :, off // 8, :, (off % 8) // 2] >> (4 * (off % 2))) & 15
        return (k * self.k_scale[page, :, off].astype(np.float64)[:, None],
                e2m1_values(vc) * self.v_scale[page, :, off].astype(np.float64)[:, None])


def tokens_of(cache, table_row, n):
    """f64 keys, values [n][heads][D] and which of the first n tokens lie on a page of the cache."""
    K, V, on = np.zeros((n, cache.heads, cache.D)), np.zeros((n, cache.heads, cache.D)), np.zeros(n, bool)
    for p in range((n + cache.page - 1) // cache.page):
        page, lo = int(table_row[p]), p * cache.page
        m = min(n, lo + cache.page) - lo
        if not 0 <= page < cache.pages:
            continue
        kc = cache.k_codes[page][:, :m]
        K[lo:lo + m, :, 0::2] = e2m1_values(kc & 15).transpose(1, 0, 2)
        K[lo:lo + m, :, 1::2] = e2m1_values(kc >> 4).transpose(1, 0, 2)
        K[lo:lo + m] *= cache.k_scale[page][:, :m].T.astype(np.float64)[..., None]
        vc = cache.v_codes[page]                                            # [heads][page/8][D][4]
        nib = np.stack([vc & 15, vc >> 4], axis=-1).reshape(cache.heads, -1, cache.D, 8)
        vals = e2m1_values(nib).transpose(1, 3, 0, 2).reshape(-1, cache.heads, cache.D)[:m]
        V[lo:lo + m] = vals * cache.v_scale[page][:, :m].T.astype(np.float64)[..., None]
        on[lo:lo + m] = True
    return K, V, on


# ------------------------------------------------------------------------------------------- attention --

def attention(q, cache, table, seq_len, q_start, sm_scale, causal, window):
    """f64 outputs [rows][q_heads][D] (NaN in padding rows), sum_t p_t |v_t| alike, and per (row, head) the largest
    sm_scale * sum_d |q_d k_d| over the tokens seen."""
    rows, HQ, D = q.shape
    G = HQ // cache.heads
    out, mass = np.full(q.shape, np.nan), np.zeros(q.shape)
    reach = np.zeros((rows, HQ))
    cap = table.shape[1] * cache.page
    for b, n in enumerate(np.clip(seq_len, 0, cap)):
        lo, hi = int(q_start[b]), int(q_start[b + 1])
        if hi <= lo:
            continue
        n = int(n)
        K, V, on = tokens_of(cache, table[b], n)
        pos = n - (hi - lo) + np.arange(hi - lo)
        t = np.arange(n)
        sees = on[None] & (pos[:, None] >= 0) & np.ones((hi - lo, n), bool)
        if causal:
            sees &= t[None] <= pos[:, None]
        if window:
            sees &= t[None] > pos[:, None] - window
        for h in range(HQ):
            qh = q[lo:hi, h].astype(np.float64)
            s = np.where(sees, sm_scale * (qh @ K[:, h // G].T), -np.inf)
            top = np.max(s, axis=1, initial=-np.inf, keepdims=True)
            p = np.where(sees, np.exp(s - np.where(np.isfinite(top), top, 0)), 0.0)
            p /= np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
            out[lo:hi, h] = p @ V[:, h // G]
            mass[lo:hi, h] = p @ np.abs(V[:, h // G])
            reach[lo:hi, h] = np.max(np.where(sees, sm_scale * (np.abs(qh) @ np.abs(K[:, h // G]).T), 0.0), axis=1,
                                     initial=0.0)
    return out, mass, reach
