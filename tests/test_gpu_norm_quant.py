"""GPU: rad_add_rmsnorm_quant_i8 against the 64-bit norm: the stored sum bit-exact, codes and scales within what f32
arithmetic can lose; row counts from one to many, row lengths over every launch shape."""
import numpy as np
import pytest

import layer_cases as C
import oracle
from oracle import layer as O
from rotated_w8a8_int8_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    return _t


def inputs(M, K, dtype, seed, residual=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp(rng.uniform(-3, 3, (M, 1)))
    h = rng.standard_normal((M, K)) * np.where(rng.random((M, K)) < 0.01, 20, 1)
    gamma = (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)
    return O.to_dtype(x, dtype), O.to_dtype(h, dtype) if residual else None, gamma


def check(q, s, h, x, res, gamma, eps, dtype, rot):
    """h exact.  The f32 norm loses: the sum of K squares, in at most 128 additions one after the other per lane and a
    tree above, and its own roundings, 140 * 2^-24 relative, half of that in its root; the mean, root, quotient and two
    products 6 * 2^-24; the seven butterfly stages 7 * 2^-24 of the sum of the block's magnitudes.  Then s = amax / 127
    (one rounding) and |code * s - n| <= s / 2 plus that loss."""
    hr, n, mass = O.add_rmsnorm(x, res, gamma, eps, dtype, rot)
    if res is not None:
        assert np.array_equal(h, hr), "the stored sum differs"
    lost = np.abs(n) * 80 * 2.0 ** -24 + (np.repeat(mass, 128, axis=1) * 90 * 2.0 ** -24 if rot else 0)
    amax = np.max(np.abs(n), axis=1)
    worst = np.max(lost, axis=1)
    assert np.all(np.abs(s.astype(np.float64) * 127 - amax) <= worst + amax * 2.0 ** -23)
    off = np.abs(q.astype(np.float64) * s.astype(np.float64)[:, None] - n)
    assert np.all(off <= s.astype(np.float64)[:, None] * (0.5 + 2.0 ** -14) + lost)
    assert q.min() >= -127 and np.all(np.max(np.abs(q.astype(int)), axis=1)[amax > 0] == 127)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("M,K", [(1, 128), (1, 5120), (3, 640), (2, 8192), (2, 8320), (17, 1152), (2, 65536),
                                 (255, 384), (256, 384), (257, 2048), (300, 4096), (260, 6144), (259, 24576),
                                 (256, 24704), (1000, 5120)])
def test_norm_quant(torch, M, K, dtype):
    print("norm", M, K, dtype, flush=True)
    x, h, g = inputs(M, K, dtype, seed=M + K)
    q, s, out = B.add_rmsnorm_quant_i8(C.put(torch, x, dtype), C.put(torch, g), C.put(torch, h, dtype), eps=1e-6)
    check(q.cpu().numpy(), s.cpu().numpy(), C.host(out), x, h, g, 1e-6, dtype, True)


@pytest.mark.parametrize("rot", [True, False])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("dtype", C.DTYPES)
def test_forms(torch, dtype, residual, rot):
    x, h, g = inputs(9, 1024, dtype, seed=5, residual=residual)
    hd = None if h is None else C.put(torch, h, dtype)
    q, s, out = B.add_rmsnorm_quant_i8(C.put(torch, x, dtype), C.put(torch, g), hd, eps=1e-5, rotate=rot)
    assert (out is hd)                                          # in place
    check(q.cpu().numpy(), s.cpu().numpy(), None if out is None else C.host(out), x, h, g, 1e-5, dtype, rot)


def test_out_of_place_keeps_the_residual(torch):
    x, h, g = inputs(5, 512, "bf16", seed=6)
    hd, ho = C.put(torch, h, "bf16"), torch.empty((5, 512), dtype=torch.bfloat16, device="cuda")
    _, _, out = B.add_rmsnorm_quant_i8(C.put(torch, x, "bf16"), C.put(torch, g), hd, residual_out=ho)
    assert out is ho and np.array_equal(C.host(hd), h)
    assert np.array_equal(C.host(ho), O.to_dtype(x + h, "bf16"))


def test_zero_rows_and_tiny_rows(torch):
    x = np.zeros((4, 256), np.float32)
    x[1] = 1e-30                                               # the mean of squares vanishes beside eps
    x[2, 7] = 1.0
    g = np.ones(256, np.float32)
    q, s, _ = B.add_rmsnorm_quant_i8(C.put(torch, x), C.put(torch, g), eps=1e-6)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert s[0] == 0 and s[3] == 0 and not q[0].any() and not q[3].any()
    check(q[1:3], s[1:3], None, x[1:3], None, g, 1e-6, "f32", True)


def test_codes_equal_the_quantiser_on_the_same_rows(torch):
    # gamma = 1 and rows whose mean square is exactly 1 normalise to themselves: the codes are the quantiser's
    rng = np.random.default_rng(8)
    x = np.where(rng.random((6, 5120)) < 0.5, 1.0, -1.0).astype(np.float32)
    q, s, _ = B.add_rmsnorm_quant_i8(C.put(torch, x), torch.ones(5120, device="cuda"), eps=0.0)
    qo, so = oracle.quant_act_i8(x, rotate=True)
    assert np.array_equal(q.cpu().numpy(), qo) and np.array_equal(s.cpu().numpy().view(np.int32), so.view(np.int32))


def test_binding_refusals(torch):
    x, g = torch.zeros(4, 256, device="cuda"), torch.ones(256, device="cuda")
    with pytest.raises(ValueError, match="gamma"):
        B.add_rmsnorm_quant_i8(x, g[:128].contiguous())
    with pytest.raises(TypeError, match="residual"):
        B.add_rmsnorm_quant_i8(x, g, x.bfloat16())
    with pytest.raises(ValueError, match="residual_out"):
        B.add_rmsnorm_quant_i8(x, g, residual_out=x.clone())
    with pytest.raises(TypeError, match="f32, bf16 or f16"):
        B.add_rmsnorm_quant_i8(x.double(), g)
    with pytest.raises(ValueError, match="contiguous"):
        B.add_rmsnorm_quant_i8(torch.zeros(256, 4, device="cuda").t(), g)
    with pytest.raises(B.RadError):
        B.add_rmsnorm_quant_i8(x[:, :200].contiguous(), g[:200].contiguous())


@pytest.mark.parametrize("rot", [True, False])
@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("M,K", [(1023, 2176), (1024, 2176), (1025, 4096), (1024, 5120), (1100, 8192), (1024, 2048), (1024, 8320)])
def test_many_tokens(torch, M, K, dtype, rot):
    # from 1024 tokens on, rows of more than 2048 and up to 8192 values take half the waves, two steps each
    print("norm", M, K, dtype, rot, flush=True)
    x, h, g = inputs(M, K, dtype, seed=M + K)
    q, s, out = B.add_rmsnorm_quant_i8(C.put(torch, x, dtype), C.put(torch, g), C.put(torch, h, dtype), eps=1e-6, rotate=rot)
    check(q.cpu().numpy(), s.cpu().numpy(), C.host(out), x, h, g, 1e-6, dtype, rot)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(6, 640), (5, 8320), (1024, 4096)])
def test_rows_whose_squares_leave_f32(torch, M, K, dtype):
    # rows of about 2^63 and more (squares pass 2^128), and of 2^-75 and less without an eps to cover them
    print("range", M, K, dtype, flush=True)
    x, h, g = inputs(M, K, dtype, seed=K)
    for size, eps in ((1e25, 1e-6), (1e30, 1e-6), (1e30, 1e30), (3e18, 1e-6), (1e-25, 0.0), (1e-30, 0.0), (1e-20, 1e-40),
                      (1e-25, 1e-45), (1e-25, 1e-6)):
        xs, hs = O.to_dtype(x * np.float32(size), dtype), O.to_dtype(h * np.float32(size), dtype)
        xs[1], hs[1] = x[1], h[1]                              # an ordinary row among them
        q, s, out = B.add_rmsnorm_quant_i8(C.put(torch, xs, dtype), C.put(torch, g), C.put(torch, hs, dtype), eps=eps)
        check(q.cpu().numpy(), s.cpu().numpy(), C.host(out), xs, hs, g, float(np.float32(eps)), dtype, True)
