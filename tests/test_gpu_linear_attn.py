"""GPU: rad_linear_attn against the recurrence in 64 bits: types, head sizes, shared keys, ragged batches, decays from none
to all, states absent, kept and in place, strides."""
import numpy as np
import pytest

import layer_cases as C
from oracle import layer as O
from oracle import mixers as X
from rotated_w8a8_int8_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    return _t


def tolerance(dtype, n, D, scale, o, mass, S, big):
    """How far outputs and states may be off.

    Row by row or in chunks, a term of a state passes at most 2 n roundings in f32 (its product, and a product and a sum
    a row or chunk), and its decay exp(g m), m <= n, is off by at most 4 roundings a row (exp, and its argument or its
    products).  An output adds D and chunk (64) roundings of its sums and a few more for scale: (6 n + D + 128) 2^-24 of
    the sum of magnitudes.  The 16-bit types take state and row weights as pairs of 16-bit parts, off by at most 2^-16
    each, and age values alike: 2^-14 for outputs, 2^-16 for states.  Then the output's own rounding.
    """
    f32 = (6 * n + D + 128) * 2.0 ** -24
    parts = 0.0 if dtype == "f32" else 2.0 ** -14
    to = (f32 + parts) * mass + O.EPS[dtype] / 2 * np.abs(o) + (2.0 ** -25 if dtype == "f16" else 1e-30)
    return to, (f32 + parts / 4) * big + 1e-30


def run(torch, new, heads, qk, D, dtype, seed=0, pad=0, decay=None, state=True, keep=True, in_place=False, single=False, scale=None,
        max_q=None, size=1.0):
    rng = np.random.default_rng(seed)
    start = C.ragged(new)
    T, Bn = int(start[-1]) + pad, len(new)
    x = O.to_dtype(size * rng.standard_normal((T, 2 * qk + heads, D)), dtype)
    g = -np.exp2(rng.uniform(-10, 0, heads)).astype(np.float32) if decay is None else np.resize(np.float32(decay), heads)
    S0 = rng.standard_normal((Bn, heads, D, D)).astype(np.float32) if state else None
    scale = D ** -0.5 if scale is None else scale
    xd = C.put(torch, x, dtype)
    q, k, v = xd.split([qk, qk, heads], dim=1)
    s_in = None if S0 is None else C.put(torch, S0)
    s_out = None if not keep else s_in if in_place else torch.full((Bn, heads, D, D), 44.0, device="cuda")
    o = torch.full((T, heads, D), 33.0, dtype=C.torch_dtype(torch, dtype), device="cuda")
    B.linear_attn(q, k, v, C.put(torch, g), state=s_in, state_out=s_out, q_start=None if single else C.put(torch, start),
                  max_q=max(new) if max_q is None else max_q, scale=scale, o=o)
    with np.errstate(under="ignore"):
        want, S, mass, big = X.linear(x[:, :qk], x[:, qk:2 * qk], x[:, 2 * qk:], g, np.zeros((Bn, heads, D, D)) if S0 is None else S0,
                                      start, scale, max_q)
    got, none = C.host(o), np.isnan(want)
    assert np.all(got[none] == 33.0), "rows of no sequence were written"
    to, ts = tolerance(dtype, max(1, max(new)), D, scale, np.nan_to_num(want), mass, S, big)
    off = np.where(none, 0, np.abs(got - np.nan_to_num(want)))
    if dtype == "f16":
        # f16 ends at 65504, its rounding at 65520: an exact output that may lie past that is that infinity's
        past = (np.abs(np.nan_to_num(want)) + to >= 65504) & np.isinf(got) & (np.sign(got) == np.sign(np.nan_to_num(want)))
        off = np.where(past, 0, off)
    assert np.all(off <= to), "off by %g of the tolerance at %s" % (np.max(off / to), np.unravel_index(np.argmax(off / to), off.shape))
    if keep:
        off = np.abs(s_out.cpu().numpy() - S)
        assert np.all(off <= ts), "state off by %g of the tolerance" % np.max(off / ts)
    if S0 is not None and not in_place:
        assert np.array_equal(s_in.cpu().numpy(), S0)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
@pytest.mark.parametrize("heads,qk", [(1, 1), (6, 6), (8, 2)])
def test_single_tokens(torch, heads, qk, D, dtype):
    run(torch, [1] * 5, heads, qk, D, dtype, seed=heads, single=True, in_place=True)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
@pytest.mark.parametrize("new", [[2], [7, 0, 1, 16], [31, 32, 33], [63, 64, 65, 5], [130, 1, 257]])
def test_ragged_rows(torch, new, D, dtype):
    print("linear", new, D, dtype, flush=True)
    run(torch, new, 4, 2, D, dtype, seed=D + len(new), pad=3)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("new,pad", [([256, 0, 128, 0, 0], 0), ([0, 0, 384, 128], 0), ([512], 0), ([129, 127, 0], 128), ([0, 700, 1, 0, 33], 5),
                                     ([128] * 9, 0), ([20] * 40 + [300], 1)])
def test_sequences_of_whole_segments_and_none(torch, new, pad, dtype):
    print("segments", new, pad, dtype, flush=True)
    run(torch, new, 4, 2, 64, dtype, seed=len(new), pad=pad)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("n", [1000, 2049])
def test_prompts(torch, n, dtype):
    print("prompt", n, dtype, flush=True)
    run(torch, [n], 2, 2, 64, dtype, seed=n)
    run(torch, [n, 70], 2, 1, 128, dtype, seed=n + 1, in_place=True)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("decay", [[0.0], [-1e-4, -30.0], [-np.inf, -0.5], [-1e30, -90.0]])
def test_decays_from_none_to_all(torch, decay, dtype):
    print("decay", decay, dtype, flush=True)
    run(torch, [1, 1], 2, 2, 64, dtype, decay=decay, single=True)
    run(torch, [150, 20, 300], 2, 2, 64, dtype, decay=decay, seed=1)


@pytest.mark.parametrize("state,keep", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("new,single", [([1, 1, 1], True), ([5, 0, 3], False), ([200, 0, 30], False)])
def test_states_absent_and_not_kept(torch, new, single, state, keep):
    run(torch, new, 4, 4, 128, "bf16", seed=2, state=state, keep=keep, single=single)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("size", [1e-3, 50.0])
def test_small_and_large_values(torch, size, dtype):
    run(torch, [100, 9], 2, 2, 128, dtype, seed=6, size=size, scale=1.0, state=False)


def test_rows_past_max_q(torch):
    run(torch, [90, 20], 2, 2, 64, "f32", seed=7, max_q=64)
    run(torch, [9, 2, 5], 2, 2, 64, "bf16", seed=8, max_q=4)


def test_no_rows_hand_the_state_on(torch):
    run(torch, [0, 0], 3, 3, 64, "f32", seed=3, pad=2, max_q=4)
    s = torch.randn((2, 2, 64, 64), device="cuda")
    out = torch.empty_like(s)
    empty = torch.empty((0, 2, 64), device="cuda")
    B.linear_attn(empty, empty, empty, torch.zeros(2, device="cuda"), state=s, state_out=out, q_start=torch.zeros(3, dtype=torch.int32, device="cuda"), max_q=8)
    assert torch.equal(out, s)


def test_a_prompt_in_chunks_is_the_prompt(torch):
    # 700 rows at once, and in calls of 200, 1, 320 and 179 with the state between
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((700, 4, 128), generator=g, device="cuda") for _ in range(3))
    decay = torch.tensor([-0.5, -0.05, -0.005, 0.0], device="cuda")
    zero = torch.tensor([0, 700], dtype=torch.int32, device="cuda")
    s_all = torch.empty((1, 4, 128, 128), device="cuda")
    o_all, _ = B.linear_attn(q, k, v, decay, state_out=s_all, q_start=zero, scale=0.1)
    s, parts, at = torch.zeros((1, 4, 128, 128), device="cuda"), [], 0
    for n in (200, 1, 320, 179):
        rows = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        parts.append(B.linear_attn(q[at:at + n], k[at:at + n], v[at:at + n], decay, state=s, state_out=s, q_start=rows, scale=0.1)[0])
        at += n
    # both within the tolerance of the exact result, which norms of 2^-13 of it bound
    for a, b in ((torch.cat(parts), o_all), (s, s_all)):
        assert float((a - b).norm()) <= 2.0 ** -13 * float(b.norm())


def test_a_block_verified_without_its_state_and_run_again_with_the_rows_accepted(torch):
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn((24, 4, 64), generator=g, device="cuda").bfloat16() for _ in range(3))
    decay, s0 = -torch.rand(4, generator=g, device="cuda"), torch.randn((3, 4, 64, 64), generator=g, device="cuda")
    start = torch.tensor([0, 8, 16, 24], dtype=torch.int32, device="cuda")
    s = s0.clone()
    o, none = B.linear_attn(q, k, v, decay, state=s, q_start=start, max_q=8)
    assert none is None and torch.equal(s, s0)
    accepted = torch.tensor([0, 3, 3, 11], dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 1, 2, 16, 17, 18, 19, 20, 21, 22, 23], device="cuda")
    o2, s2 = B.linear_attn(q[rows], k[rows], v[rows], decay, state=s, state_out=s, q_start=accepted, max_q=8)
    assert torch.allclose(o2.float(), o[rows].float(), rtol=2.0 ** -7, atol=2.0 ** -7 * float(o.float().abs().max()))
    assert torch.equal(s2[1], s0[1]) and not torch.equal(s2[0], s0[0])
