"""CPU oracle of the token mixers beside causal attention: attention for trees of drafted tokens, the weights that
attention gives to cached tokens, the selection by weight, the move of cached tokens, and linear attention.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it imports nothing from the GPU library.  Plain NumPy in
64 bits, written from the definitions in include/rad.h.
"""
from __future__ import annotations

import numpy as np

from oracle import layer as O


def mask_bits(words, n):
    """[rows][n] truth values of uint64 masks [rows][words]; nodes past the words are not seen."""
    out = np.zeros((len(words), n), bool)
    for j in range(min(n, 64 * words.shape[1])):
        out[:, j] = (words[:, j // 64] >> np.uint64(j % 64)) & np.uint64(1)
    return out


def sees_position(n, len_, on, causal, window):
    pos, t = len_ - n + np.arange(n)[:, None], np.arange(len_)[None]
    sees = on[None] & (pos >= 0) & np.ones((n, len_), bool)
    if causal:
        sees &= t <= pos
    if window:
        sees &= t > pos - window
    return sees


def sees_tree(n, len_, on, words, window):
    base, t = len_ - n, np.arange(len_)[None]
    bits = mask_bits(words, n) & ((base + np.arange(n)) >= 0)[None]
    sees = np.zeros((n, len_), bool)
    first = max(base, 0)
    sees[:, :first] = True
    if window:
        sees[:, :first] &= t[:, :first] >= base + bits.sum(axis=1)[:, None] - window
    sees[:, first:] = bits[:, first - base:]
    return sees & on[None] & ((base + np.arange(n)) >= 0)[:, None]


def attend(q, cache, table, seq_len, q_start, sm_scale, sees_of):
    """As oracle.layer.attention, with sees_of(b, n, len, on) telling what each row sees; and the probabilities
    [(b, h)] -> [n][len]."""
    rows, HQ, D = q.shape
    G = HQ // cache.heads
    out, mass, reach, probs = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros((rows, HQ)), {}
    cap = table.shape[1] * cache.page
    for b, len_ in enumerate(np.clip(seq_len, 0, cap)):
        lo, hi, len_ = int(q_start[b]), int(q_start[b + 1]), int(len_)
        if hi <= lo:
            continue
        K, V, on = O.tokens_of(cache, table[b], len_)
        sees = sees_of(b, hi - lo, len_, on)
        for h in range(HQ):
            qh = q[lo:hi, h].astype(np.float64)
            s = np.where(sees, sm_scale * (qh @ K[:, h // G].T), -np.inf)
            top = np.max(s, axis=1, initial=-np.inf, keepdims=True)
            p = np.where(sees, np.exp(s - np.where(np.isfinite(top), top, 0)), 0.0)
            p /= np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
            probs[b, h] = p
            out[lo:hi, h] = p @ V[:, h // G]
            mass[lo:hi, h] = p @ np.abs(V[:, h // G])
            reach[lo:hi, h] = np.max(np.where(sees, sm_scale * (np.abs(qh) @ np.abs(K[:, h // G]).T), 0.0), axis=1, initial=0.0)
    return out, mass, reach, probs


def weights(old, probs, reach, heads, G, seq_len, q_start, observe, factor):
    """f64 weights after a call, and the sum of each entry's probabilities times expm1(2^-13 reach) (what scores off by
    2^-14 reach may change)."""
    new, slack = old.astype(np.float64).copy(), np.zeros(old.shape)
    for (b, hq), p in probs.items():
        n, len_ = p.shape
        first = max(0, n - observe) if observe else 0
        if hq % G == 0:
            base = max(len_ - n, 0)
            new[b, hq // G, :base] = factor * new[b, hq // G, :base] if factor else 0.0
            new[b, hq // G, base:len_] = 0.0
        new[b, hq // G, :len_] += p[first:].sum(axis=0)
        r = reach[int(q_start[b]):int(q_start[b + 1]), hq]
        slack[b, hq // G, :len_] += (p * np.expm1(2.0 ** -13 * r)[:, None])[first:].sum(axis=0)
    return new, slack


def select(w, n_tokens, budget, first, recent):
    """Ascending tokens kept of one head's weights."""
    if n_tokens <= budget:
        return np.arange(n_tokens)
    free = np.arange(first, n_tokens - recent)
    key = np.where(np.isnan(w[free]), -np.inf, w[free]) + 0.0
    # NaN below -inf: a second key
    order = np.lexsort((free, np.isnan(w[free]), -key))
    take = free[order[:budget - first - recent]]
    return np.sort(np.concatenate([np.arange(first), take, np.arange(n_tokens - recent, n_tokens)]))


def nibble_tokens(cache, h, page, off):
    """One head's codes and scales of a token: [D] key codes, [D] value codes, scales as they are held."""
    kc = cache.k_codes[page, h, off]
    k = np.stack([kc & 15, kc >> 4], axis=-1).reshape(-1)
    v = (cache.v_codes[page, h, off // 8, :, (off % 8) // 2] >> (4 * (off % 2))) & 15
    return k, v, cache.k_scale[page, h, off:off + 1].view(np.uint16)[0], cache.v_scale[page, h, off:off + 1].view(np.uint16)[0]


def put_token(cache, h, page, off, token):
    k, v, ks, vs = token
    cache.k_codes[page, h, off] = k[0::2] | (k[1::2] << 4)
    byte, shift = (off % 8) // 2, 4 * (off % 2)
    old = cache.v_codes[page, h, off // 8, :, byte]
    cache.v_codes[page, h, off // 8, :, byte] = (old & (0xF0 >> shift)) | (v << shift)
    cache.k_scale[page, h, off:off + 1].view(np.uint16)[0] = ks
    cache.v_scale[page, h, off:off + 1].view(np.uint16)[0] = vs


def move(cache, table, seq_len, source, count, to, to_table, to_start):
    """Moves entry i of source [B][lists][n] to token to_start + i of the pages to_table of `to`."""
    cap = table.shape[1] * cache.page
    for b in range(len(table)):
        for h in range(cache.heads):
            lst, taken = source[b, h if source.shape[1] > 1 else 0], []
            for i in range(int(np.clip(count[b], 0, source.shape[2]))):
                t = int(lst[i])
                page = int(table[b, t // cache.page]) if 0 <= t < min(int(np.clip(seq_len[b], 0, cap)), cap) else -1
                taken.append(nibble_tokens(cache, h, page, t % cache.page) if 0 <= page < cache.pages else None)
            for i, token in enumerate(taken):
                t = int(to_start[b]) + i
                if token is None or t < 0 or t >= to_table.shape[1] * to.page:
                    continue
                page = int(to_table[b, t // to.page])
                if 0 <= page < to.pages:
                    put_token(to, h, page, t % to.page, token)


def linear(q, k, v, log_decay, state, q_start, scale, max_q=None):
    """f64 outputs [rows][heads][D] (NaN in rows of no sequence) and states, row by row, and the sums of magnitudes that
    both come of.  q_start None: one row a sequence."""
    rows, heads, D = v.shape
    B = len(state)
    each = heads // q.shape[1]
    start = np.arange(B + 1) if q_start is None else q_start
    S, big = state.astype(np.float64).copy(), np.abs(state.astype(np.float64))
    o, mass = np.full((rows, heads, D), np.nan), np.zeros((rows, heads, D))
    a = np.exp(log_decay.astype(np.float64))[:, None, None]
    of = np.arange(heads) // each
    for b in range(B):
        n = int(start[b + 1] - start[b]) if max_q is None else min(int(start[b + 1] - start[b]), max_q)
        for r in range(int(start[b]), int(start[b]) + n):
            qr, kr, vr = q[r].astype(np.float64)[of], k[r].astype(np.float64)[of], v[r].astype(np.float64)
            S[b] = a * S[b] + kr[:, :, None] * vr[:, None, :]
            big[b] = a * big[b] + np.abs(kr)[:, :, None] * np.abs(vr)[:, None, :]
            o[r] = scale * np.einsum("hd,hde->he", qr, S[b])
            mass[r] = abs(scale) * np.einsum("hd,hde->he", np.abs(qr), big[b])
    return o, S, mass, big
