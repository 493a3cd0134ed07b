"""What the backward passes of include/iq_train.h keep of their operands.

bfloat16 calls form products of 32-bit arithmetic, and round once, at the end.
Gradients are sparse, so that few additions round and a bound on all roundings before the last stays far below a step
of bfloat16: then the result has to lie between the roundings of the 64-bit value less and plus that bound, which for
nearly all values are the same.  u = 2^-24:
  gradient times block scale   2^-23 of the product (two fp16 values), in steps of 2^-39 of the largest: 2^-40 each, with
                               4 bits for how far the token's and the payload's powers of two lie above them
  sums                         2u of the partial sum for each addition of a value that is not zero
  act, slope                   as in test_gpu_train.py: 2^-20 |g| and 2^-17, their sums' errors apart

float32 calls stay within 2^-20 of the result in the norm, which 32-bit arithmetic on decoded weights does not leave
either, also where a weight or an activation is far larger than the rest."""
import numpy as np
import pytest

from ggml_iq_codebook_imatrix_amd import inputs
from test_gpu_run import FORMATS, U, decoded, dev, f64, payload, round_to
from test_gpu_train import ACTS, act_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ggml_iq_codebook_imatrix_amd import api as a
    a.lib()
    return a


def sparse(T, cols, n, seed, size=1.0):
    """n values of bfloat16 a token, of about one size, at random places; zeros elsewhere."""
    g = inputs.rng(seed)
    x = np.zeros((T, cols), np.float32)
    at = np.argsort(g.random((T, cols)), 1)[:, :n]
    np.put_along_axis(x, at, (g.choice([-1, 1], (T, min(n, cols))) * g.uniform(1, 2, (T, min(n, cols))) * size).astype(
        np.float32), 1)
    return dev(x, torch.bfloat16)


def between(got, v, off):
    low, high = round_to(v - off, torch.bfloat16), round_to(v + off, torch.bfloat16)
    bad = (got < low) | (got > high)
    assert not bad.any(), bad.mean()
    # one result alone is right, but for sums of few values that nearly cancel (by the 64-bit values and the bounds alone
    # 0.79 to 0.90 of these gated blocks' results, and more of the projections')
    assert (low == high).mean() > 0.75


# rows, blocks, tokens: ends inside a tile; tiles of 128 and of 256 tokens
@pytest.mark.parametrize("rows,nb,T", [(70, 3, 40), (200, 20, 3000)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_backward_rounds_once(api, orc, fmt, rows, nb, T):
    print("[case] linear backward rounds once", fmt, rows, nb, T, flush=True)
    grid, p = inputs.grid_for(fmt, 41), payload(fmt, rows, nb, rows)
    w, dy = decoded(orc, fmt, p, grid), sparse(T, rows, 3, 7, 1e-3)
    got = f64(api.linear_backward(fmt, dev(p), dev(grid), dy))
    dd = f64(dy)
    v, S = dd @ w, np.abs(dd) @ np.abs(w)
    # 3 values of two parts each, and as many partial sums of splits: 9 additions
    between(got, v, (9 * 2 * U + 2.0 ** -23) * S + 3 * 2.0 ** -36 * np.abs(dd).max() * np.abs(w).max())


@pytest.mark.parametrize("inter,nb,T", [(70, 3, 40), (200, 20, 3000)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_glu_backward_rounds_once(api, orc, fmt, inter, nb, T):
    act = ACTS[FORMATS.index(fmt) % 3]
    print("[case] glu backward rounds once", fmt, inter, nb, T, act, flush=True)
    grid = inputs.grid_for(fmt, 41)
    gate, up = payload(fmt, inter, nb, inter), payload(fmt, inter, nb, inter + 1)
    wg, wu = decoded(orc, fmt, gate, grid), decoded(orc, fmt, up, grid)
    # x of 64 makes g of a few units, whose activation matters; dh has two values a token
    x, dh = sparse(T, nb * 256, 3, 8, 64.0), sparse(T, inter, 2, 9, 1e-3)
    got = f64(api.glu_backward(fmt, dev(gate), dev(up), dev(grid), x, dh, activation=act))
    xd, dd = f64(x), f64(dh)
    g, u = xd @ wg.T, xd @ wu.T
    og, ou = (12 * 2 * U * (np.abs(xd) @ np.abs(m).T) for m in (wg, wu))
    a, slope = act_of(act, g)
    oa, os_ = 1.13 * og + np.abs(g) * 2.0 ** -20, og + 2.0 ** -17
    dg, du = dd * u * slope, dd * a
    odg = np.abs(dd) * ((np.abs(u) + ou) * os_ + 1.2 * ou) + np.abs(dg) * 2.0 ** -23
    odu = np.abs(dd) * oa + np.abs(du) * 2.0 ** -23
    dx = dg @ wg + du @ wu
    S = (np.abs(dg) + odg) @ np.abs(wg) + (np.abs(du) + odu) @ np.abs(wu)
    off = odg @ np.abs(wg) + odu @ np.abs(wu) + 12 * 2 * U * S
    most = max(np.abs(wg).max(), np.abs(wu).max())
    off += 4 * 2.0 ** -30 * np.maximum(np.abs(dg).max(1), np.abs(du).max(1))[:, None] * most
    between(got, dx, off)


def uneven(fmt, rows, nb, seed, row, block, by):
    """Block scales of about 0.004, that of one block `by` times as large."""
    d = 0.004 * np.exp(0.3 * inputs.rng(seed).standard_normal((rows, nb)))
    d[row, block] *= by
    return payload(fmt, rows, nb, seed, d16=d.astype(np.float16).view(np.uint16))


# how much larger one block's scale is than the others', and one activation than the token's others, in columns whose
# weights are zeros; a batch, and tokens enough for tiles
@pytest.mark.parametrize("T", [20, 600])
@pytest.mark.parametrize("scale,activation", [(1, 0), (16, 0), (1, 1000), (16, 1000), (100, 1000), (1000, 100)])
def test_float32_glu_backward_with_outliers(api, orc, T, scale, activation):
    fmt, inter, nb = "IQ1_S", 400, 20
    print("[case] glu backward outliers", T, scale, activation, flush=True)
    g = inputs.rng(31)
    grid = inputs.grid_for(fmt, 41)
    gate, up = uneven(fmt, inter, nb, 3, 17, 5, scale), uneven(fmt, inter, nb, 4, 30, 6, 1)
    if activation:
        for p in (gate, up):
            p[:, 2] = 0
    wg, wu = decoded(orc, fmt, gate, grid), decoded(orc, fmt, up, grid)
    x = g.standard_normal((T, nb * 256)).astype(np.float32)
    dh = (1e-3 * g.standard_normal((T, inter))).astype(np.float32)
    if activation:
        x[:, 2 * 256 + 7] = activation
    got = f64(api.glu_backward(fmt, dev(gate), dev(up), dev(grid), dev(x), dev(dh)))
    xd, dd = x.astype(np.float64), dh.astype(np.float64)
    a, slope = act_of("silu", xd @ wg.T)
    want = (dd * (xd @ wu.T) * slope) @ wg + (dd * a) @ wu
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    print("off by", off, flush=True)
    assert off <= 2.0 ** -20


@pytest.mark.parametrize("scale,gradient", [(1, 1), (1000, 1), (1, 1000), (100, 100)])
def test_float32_linear_backward_with_outliers(api, orc, scale, gradient):
    fmt, rows, nb, T = "IQ2_S", 500, 6, 50
    print("[case] linear backward outliers", scale, gradient, flush=True)
    g = inputs.rng(32)
    grid, p = inputs.grid_for(fmt, 41), uneven(fmt, rows, nb, 5, 11, 3, scale)
    w = decoded(orc, fmt, p, grid)
    dy = g.standard_normal((T, rows)).astype(np.float32)
    dy[:, 12] *= gradient
    got, want = f64(api.linear_backward(fmt, dev(p), dev(grid), dev(dy))), dy.astype(np.float64) @ w
    for at in (slice(0, 768), slice(768, 1024), slice(1024, None)):  # the large scale's columns, and those beside them
        off = np.linalg.norm((got - want)[:, at]) / np.linalg.norm(want[:, at])
        print("off by", off, flush=True)
        assert off <= 2.0 ** -20


@pytest.mark.parametrize("act", ACTS)
def test_gradients_past_float32_on_the_way(api, act):
    """dh * u past float32 where the slope is zero, and gradients of 2^-100 and of 2^60 beside those of one."""
    print("[case] far gradients", act, flush=True)
    fmt, T = "IQ2_XS", 20
    grid, gate = dev(inputs.grid_for(fmt, 5)), dev(payload(fmt, 48, 1, 6))
    up = dev(payload(fmt, 48, 1, 7, d16=1))
    x = dev(np.abs(inputs.activations(T, 256, 7, 8)).astype(np.float32)) * 1e15
    wg, wu = (api.dequantize(fmt, p, grid, torch.float32).double() for p in (gate, up))
    g, u = x.double() @ wg.T, x.double() @ wu.T
    off_state = g < -200  # activation and slope are zeros there
    assert bool(off_state.any())
    dh = torch.where(off_state, 1e35, 0.0).float()
    assert bool((dh.double() * u)[off_state].abs().max() > 1e39)
    assert bool((api.glu_backward(fmt, gate, up, grid, x, dh, activation=act) == 0).all())

    x = x * 1e-15
    dh = torch.ones((T, 48), device="cuda")
    near = api.glu_backward(fmt, gate, up, grid, x, dh, activation=act)
    for n in (-60, -100, 60):
        far = api.glu_backward(fmt, gate, up, grid, x, dh * 2.0 ** n, activation=act)
        scaled = torch.linalg.norm(far.double() * 2.0 ** -n - near.double())
        assert bool(scaled <= 2.0 ** -22 * torch.linalg.norm(near.double()))


@pytest.mark.parametrize("fmt,inter,nb,T", [("IQ2_XS", 33, 2, 9), ("IQ2_S", 130, 3, 40), ("IQ1_M", 300, 4, 150),
                                            ("IQ1_S", 1500, 8, 4100), ("IQ2_XXS", 1500, 20, 4100)])
def test_float32_glu_backward_sums_a_checkpoint_as_its_values(api, fmt, inter, nb, T):
    """A checkpoint's values have seven bits, so that a call's sums are those of the float32 tokens it stands for, bit
    for bit, in any kernel: few tokens, batches, tiles."""
    print("[case] float32 checkpoint", fmt, inter, nb, T, flush=True)
    grid = dev(inputs.grid_for(fmt, 5))
    gate, up = dev(payload(fmt, inter, nb, 6)), dev(payload(fmt, inter, nb, 7))
    x = dev(inputs.activations(T, nb * 256, 1, 2, bf16=False))
    dh = dev((1e-3 * inputs.rng(3).standard_normal((T, inter))).astype(np.float32))
    kept = api.checkpoint(x)
    assert torch.equal(api.glu_backward(fmt, gate, up, grid, kept, dh),
                       api.glu_backward(fmt, gate, up, grid, api.restore(*kept), dh))
