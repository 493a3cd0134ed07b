"""iq_linear and iq_moe on the GPU against plain 64-bit arithmetic on the oracle's decoded weights.

Exact cases: tokens, adapters and block scales are small integers or powers of two, so every product and every sum
in any order is a float32 number and the result must be equal bit for bit.  Random cases: the tolerances below are
sums of the roundings that the method makes (u = 2^-24 a half step of float32):
  product of K columns   each fp32 addition, in any order, is off by at most 2u (truncation allowed) of a partial sum
                         that is at most S = sum |x w|; no output passes through more than 256 additions in a block
                         and one per block: (260 + K / 256 + waves <= 16) 2u S; float32 tokens are held to 2^-22 each
  output                 bf16 eps / 2 = 2^-8 of the value, float32 2^-24
  h                      1 / (1 + exp(-g)) to 2^-20 with h's own products; held to 2^-11 (bf16) or 2^-21 (float32)"""
import numpy as np
import pytest

from ggml_iq_codebook_imatrix_amd import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FORMATS = ["IQ2_XXS", "IQ2_XS", "IQ2_S", "IQ1_S", "IQ1_M"]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ggml_iq_codebook_imatrix_amd import api as a
    a.lib()
    return a


def payload(fmt, rows, nb, seed, d16=None):
    """Random fields; block scales d16 (fp16 bits; default about 0.004)."""
    g = inputs.rng(seed)
    size = {"IQ2_XXS": 66, "IQ2_XS": 74, "IQ2_S": 82, "IQ1_S": 50, "IQ1_M": 56}[fmt]
    p = g.integers(0, 256, (rows, nb, size), dtype=np.uint8)
    if d16 is None:
        d16 = (0.004 * np.exp(0.3 * g.standard_normal((rows, nb)))).astype(np.float16).view(np.uint16)
    d16 = np.broadcast_to(np.asarray(d16, dtype=np.uint16), (rows, nb))
    if fmt == "IQ1_M":
        for w in range(4):
            p[..., 49 + 2 * w] = (p[..., 49 + 2 * w] & 15) | (((d16 >> (4 * w)) & 15) << 4).astype(np.uint8)
    else:
        p[..., 0], p[..., 1] = d16 & 255, d16 >> 8
    return p


def decoded(orc, fmt, p, grid):
    return orc.dequantize(fmt, p, p.shape[0], p.shape[1] * 256, grid).astype(np.float64)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def round_to(v, dtype):
    return torch.from_numpy(v).to(torch.float32).to(dtype).double().numpy()


def shifted(t, by):
    """The same values, `by` elements into a buffer of their own."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    buf[by:] = t.reshape(-1)
    return buf[by:].view(t.shape)


def odd(t):
    return shifted(t, 1)


# --------------------------------------------------------------------------
# iq_linear
# --------------------------------------------------------------------------
# rows, blocks, tokens, adapters, rank: one row and token, ends inside every tile size, odd ranks, long batches
SHAPES = [(1, 1, 1, 0, 0), (16, 2, 1, 2, 1), (15, 1, 2, 1, 3), (17, 3, 16, 3, 8), (33, 2, 17, 5, 5), (100, 5, 33, 2, 16),
          (257, 8, 63, 7, 7), (64, 9, 65, 4, 32), (1001, 3, 130, 3, 4), (300, 2, 300, 40, 2), (70, 20, 40, 3, 64),
          (513, 1, 515, 2, 17)]


def exact_linear(orc, fmt, rows, nb, T, N, r, seed):
    g = inputs.rng(seed)
    grid = inputs.grid_for(fmt, 300 + seed)
    p = payload(fmt, rows, nb, seed, d16=g.choice([0x2000, 0x2400, 0x1c00], (rows, nb)))  # 2^-7, 2^-6, 2^-8
    x = g.integers(-8, 9, (T, nb * 256)).astype(np.float32)
    a = g.integers(-1, 2, (N, r, nb * 256)).astype(np.float32)
    b = g.integers(-2, 3, (N, rows, r)).astype(np.float32)
    scale = 2.0 ** g.integers(-2, 3, N).astype(np.float32)
    ids = g.integers(-1, max(N, 1), T).astype(np.int32)
    w = decoded(orc, fmt, p, grid)
    y, size = x.astype(np.float64) @ w.T, np.abs(x).astype(np.float64) @ np.abs(w).T
    for n in range(N):
        at = ids == n
        v = x[at].astype(np.float64) @ a[n].T
        y[at] += scale[n] * (v @ b[n].T)
        size[at] += scale[n] * (np.abs(v) @ np.abs(b[n]).T)
    return grid, p, x, a, b, scale.astype(np.float32), ids, y, size


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_exact(api, orc, fmt, dtype):
    for i, (rows, nb, T, N, r) in enumerate(SHAPES):
        print("[case] linear exact", fmt, dtype, rows, nb, T, N, r, flush=True)
        grid, p, x, a, b, scale, ids, y, size = exact_linear(orc, fmt, rows, nb, T, N, r, 20 + i)
        # Weights are multiples of 2^-11, adapters' products of 2^-2.  `size`, the sum of |x w| and of scale |v b| over
        # the ranks, bounds every partial sum in any order: below 2^13 a float32 holds each exactly.  Above it (adapters
        # of large rank) no output takes more than 8 + 64 / 16 + 2 additions of sums that are themselves exact (blocks
        # alone stay below 2^13), each off by 2^-24 of at most `size`.
        lora = dict(lora_a=dev(a, dtype), lora_b=dev(b, dtype), lora_scale=dev(scale), lora_ids=dev(ids)) if N else {}
        st = api.new_status()
        got = api.linear(fmt, dev(p), dev(grid), dev(x, dtype), status=st, **lora)
        assert got.dtype == dtype and got.shape == (T, rows)
        sure = size < 2.0 ** 13
        assert sure.mean() > (0.5 if r < 64 else 0.1)
        assert np.array_equal(f64(got)[sure], round_to(y, dtype)[sure]), (rows, nb, T, N, r)
        near = np.abs(f64(got) - y) <= 14 * U * size + np.abs(y) * (2.0 ** -8 if dtype == torch.bfloat16 else U)
        assert near.all(), (rows, nb, T, N, r)
        assert api.read_status(st) == 0


def linear_tolerance(x, w, dtype, y):
    S = np.abs(x) @ np.abs(w).T
    K = x.shape[1]
    return ((276 + K / 256) * 2 * U + (2.0 ** -22 if dtype == torch.float32 else 0)) * S + \
        np.abs(y) * (2.0 ** -8 if dtype == torch.bfloat16 else U) * 1.01


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_random(api, orc, fmt, dtype):
    for rows, nb, T, N, r in ((129, 8, 5, 2, 16), (200, 3, 45, 4, 9), (96, 20, 200, 3, 24)):
        print("[case] linear random", fmt, dtype, rows, nb, T, flush=True)
        g = inputs.rng(rows)
        grid = inputs.grid_for(fmt, 41)
        p = payload(fmt, rows, nb, rows + 1)
        x = dev(inputs.activations(T, nb * 256, 42, 43, bf16=False), dtype)
        a = dev(g.standard_normal((N, r, nb * 256), dtype=np.float32) * 0.02, dtype)
        b = dev(g.standard_normal((N, rows, r), dtype=np.float32) * 0.02, dtype)
        ids = g.integers(-1, N, T).astype(np.int32)
        got = f64(api.linear(fmt, dev(p), dev(grid), x, lora_a=a, lora_b=b, lora_ids=dev(ids)))
        xd, w = f64(x), decoded(orc, fmt, p, grid)
        y, more = xd @ w.T, np.zeros((T, rows))
        for n in range(N):
            at = ids == n
            y[at] += (xd[at] @ f64(a)[n].T) @ f64(b)[n].T
            # K additions for v, r more for its product with B
            more[at] += (nb * 256 + r + 8) * 2 * U * ((np.abs(xd[at]) @ np.abs(f64(a)[n]).T) @ np.abs(f64(b)[n]).T)
        assert np.all(np.abs(got - y) <= linear_tolerance(xd, w, dtype, y) + more)
        # the errors do not add up in one direction: over all outputs they stay near one rounding
        rel = np.linalg.norm(got - y) / np.linalg.norm(y)
        assert rel < (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20)


@pytest.mark.parametrize("T", [3, 40, 150])
def test_linear_scales_with_the_tokens(api, T):
    """Blocks are scaled by powers of two: a token times 2^n gives its outputs times 2^n, bit for bit, down to
    subnormal tokens and up to where outputs still fit; every token has its own scale."""
    print("[case] linear powers of two", T, flush=True)
    fmt, rows, nb = "IQ2_XS", 80, 3
    grid, p = dev(inputs.grid_for(fmt, 5)), dev(payload(fmt, rows, nb, 6))
    x = dev(inputs.activations(T, nb * 256, 7, 8))
    base = api.linear(fmt, p, grid, x)
    n = torch.arange(T, device="cuda") * (190 // max(T - 1, 1)) - 100  # 2^-100 .. 2^90
    f = dev(np.ldexp(np.float32(1), n.cpu().numpy()))[:, None]  # torch.ldexp on the GPU is an ulp off from 2^90 on
    got = api.linear(fmt, p, grid, x * f)
    assert torch.equal(got, base * f)
    small = torch.full((T, nb * 256), 2.0 ** -133, device="cuda").to(torch.bfloat16)  # the smallest bf16
    ones = api.linear(fmt, p, grid, torch.ones_like(small).float())
    got = api.linear(fmt, p, grid, small.float())
    # each of the nb blocks' sums is rounded once to the subnormal step 2^-149 (half a step: 2^-150); sums of
    # multiples of that step are exact
    assert bool(((got.double() - ones.double() * 2.0 ** -133).abs() <= nb * 2.0 ** -150).all())
    zeros = api.linear(fmt, p, grid, torch.zeros_like(x))
    assert bool((zeros == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [6, 50, 140])
def test_linear_infinities_stay_in_their_token(api, T, dtype):
    print("[case] linear inf nan", T, dtype, flush=True)
    fmt, rows, nb = "IQ2_S", 100, 4
    grid, p = dev(inputs.grid_for(fmt, 5)), dev(payload(fmt, rows, nb, 6))
    x = dev(inputs.activations(T, nb * 256, 7, 8)).to(dtype)
    clean = api.linear(fmt, p, grid, x)
    w = api.dequantize(fmt, p, grid)
    bad = x.clone()
    bad[1, 300], bad[T - 2, 17], bad[T - 1, 5] = float("inf"), float("-inf"), float("nan")
    got = api.linear(fmt, p, grid, bad)
    keep = [t for t in range(T) if t not in (1, T - 2, T - 1)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.equal(got[1].float(), torch.sign(w[:, 300]) * float("inf"))
    assert torch.equal(got[T - 2].float(), torch.sign(w[:, 17]) * -float("inf"))
    assert bool(got[T - 1].isnan().all())


def test_linear_adapter_ids(api):
    """-1 adds nothing and raises nothing; other ids outside the range add nothing and raise the bit."""
    fmt, rows, nb, T, N, r = "IQ1_S", 50, 2, 20, 3, 6
    for T in (20, 150):
        print("[case] linear ids", T, flush=True)
        g = torch.Generator(device="cuda").manual_seed(1)
        grid, p = dev(inputs.grid_for(fmt, 5)), dev(payload(fmt, rows, nb, 6))
        x = dev(inputs.activations(T, nb * 256, 7, 8)).bfloat16()
        a = torch.randn((N, r, nb * 256), device="cuda", generator=g).bfloat16()
        b = torch.randn((N, rows, r), device="cuda", generator=g).bfloat16()
        none = api.linear(fmt, p, grid, x)
        ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        st = api.new_status()
        assert torch.equal(api.linear(fmt, p, grid, x, a, b, None, ids, status=st), none)
        assert api.read_status(st) == 0
        ids[3], ids[7], ids[T - 1], ids[5] = N, -2, 2 ** 31 - 1, 1
        got = api.linear(fmt, p, grid, x, a, b, None, ids, status=st)
        assert api.read_status(st) == api.STATUS_BADID
        keep = [t for t in range(T) if t != 5]
        assert torch.equal(got[keep], none[keep]) and not torch.equal(got[5], none[5])
        # an adapter's infinities reach its own tokens only
        a2 = a.clone()
        a2[0] = float("inf")
        assert torch.equal(api.linear(fmt, p, grid, x, a2, b, None, ids), got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows, T", [(70, 5), (70, 40), (1100, 500), (2000, 1100)])
def test_linear_infinities_through_the_adapters(api, rows, T, dtype):
    """An infinity in a token passes through its adapter as plain arithmetic has it: inf, or NaN against an opposite one."""
    print("[case] linear inf adapters", rows, T, dtype, flush=True)
    fmt, nb = "IQ2_XS", 2
    grid, p = dev(inputs.grid_for(fmt, 5)), dev(payload(fmt, rows, nb, 6))
    x = dev(inputs.activations(T, nb * 256, 7, 8)).to(dtype)
    x[1, 300], x[T - 2, 17] = float("inf"), float("-inf")
    sign = torch.sign(api.dequantize(fmt, p, grid)).double()
    for r in (1, 8, 9, 40):
        g = torch.Generator(device="cuda").manual_seed(r)
        a = (torch.rand((2, r, nb * 256), device="cuda", generator=g) + 0.5).to(dtype)
        b = (torch.rand((2, rows, r), device="cuda", generator=g) + 0.5).to(dtype)
        ids = (torch.arange(T, device="cuda") % 2).int()
        got = api.linear(fmt, p, grid, x, a, b, None, ids).double()
        # A and B are positive: the adapter gives the infinity's own sign in every row
        inf = float("inf")
        assert torch.equal(got[1].nan_to_num(7, inf, -inf), (sign[:, 300] * inf + inf).nan_to_num(7, inf, -inf)), r
        assert torch.equal(got[T - 2].nan_to_num(7, inf, -inf), (sign[:, 17] * -inf - inf).nan_to_num(7, inf, -inf)), r
        keep = [t for t in range(T) if t not in (1, T - 2)]
        assert bool(got[keep].isfinite().all())


def test_linear_codebook_rounding_is_reported(api, orc):
    """A codebook that fp16 does not hold is rounded (2^-11 twice per weight) and reported."""
    for fmt in FORMATS:
        print("[case] linear codebook", fmt, flush=True)
        g = inputs.rng(9)
        grid = inputs.grid_for(fmt, 5) * np.float32(0.97)
        p, x = payload(fmt, 40, 2, 6), inputs.activations(9, 512, 7, 8)
        st = api.new_status()
        got = f64(api.linear(fmt, dev(p), dev(grid), dev(x), status=st))
        assert api.read_status(st) == api.STATUS_ROUNDED
        w = decoded(orc, fmt, p, grid)
        # IQ1 adds 1/8 to the rounded value: the value's rounding is 2^-11 of at most 0.97, in units of the weight's step
        step = np.abs(w) * 2.0 ** -10 if fmt.startswith("IQ2") else np.abs(w) * 2.0 ** -11 + \
            2.0 ** -11 * np.abs(w).max(1, keepdims=True)
        tol = np.abs(x).astype(np.float64) @ (step * 1.01).T + linear_tolerance(x.astype(np.float64), w, torch.float32, got)
        assert np.all(np.abs(got - x.astype(np.float64) @ w.T) <= tol)
        # values of six significant bits in IQ2 (25/8 = 11.001b) need no rounding
        if fmt.startswith("IQ2"):
            st = api.new_status()
            lattice = np.where(inputs.grid_for(fmt, 5) == 3, np.float32(3.125), inputs.grid_for(fmt, 5))
            api.linear(fmt, dev(p), dev(lattice), dev(x), status=st)
            assert api.read_status(st) == 0


@pytest.mark.parametrize("T", [1, 20, 200])
def test_linear_views_guards_and_empty(api, T):
    """Every even address of the payload, odd ones of the rest, caller buffers, memory behind every output, empty calls."""
    print("[case] linear views", T, flush=True)
    rows, nb, N, r = 37, 3, 2, 3
    for fmt in FORMATS:
        grid, pay = dev(inputs.grid_for(fmt, 5)), dev(payload(fmt, rows, nb, 6))
        x = dev(inputs.activations(T, nb * 256, 7, 8)).bfloat16()
        want = api.linear(fmt, pay, grid, x)
        for by in (2, 4, 6, 14):
            assert torch.equal(api.linear(fmt, shifted(pay, by), grid, x), want), (fmt, by)
        with pytest.raises(api.IQError):
            api.linear(fmt, odd(pay), grid, x)
    fmt = "IQ2_XXS"
    grid, pay = dev(inputs.grid_for(fmt, 5)), dev(payload(fmt, rows, nb, 6))
    x = dev(inputs.activations(T, nb * 256, 7, 8)).bfloat16()
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn((N, r, nb * 256), device="cuda", generator=g).bfloat16()
    b = torch.randn((N, rows, r), device="cuda", generator=g).bfloat16()
    ids = (torch.arange(T, device="cuda") % N).int()
    want = api.linear(fmt, pay, grid, x, a, b, None, ids)

    need = api.linear_workspace_size(fmt, rows, nb * 256, x.dtype, T, r)
    ws = torch.full((need + 100,), 7, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 2, rows), 7.0, dtype=x.dtype, device="cuda")
    got = api.linear(fmt, shifted(pay, 2), odd(grid), odd(x), odd(a), odd(b), None, ids, out=out[1:T + 1],
                     workspace=ws[1:need + 1])
    assert got.data_ptr() == out[1].data_ptr() and torch.equal(got, want)
    assert bool((out[0] == 7).all()) and bool((out[T + 1] == 7).all())
    assert int(ws[0]) == 7 and bool((ws[need + 1:] == 7).all())
    assert api.linear(fmt, pay, grid, x[:0]).shape == (0, rows)
    assert api.linear(fmt, pay[:0], grid, x).shape == (T, 0)
    with pytest.raises(api.IQError):
        api.linear(fmt, pay, grid, x, a, b, None, ids, workspace=ws[:need - 1])
    with pytest.raises(api.IQError):
        api.linear(fmt, pay, grid, torch.stack((x, x), -1)[..., 0])  # not contiguous
    with pytest.raises(api.IQError):
        api.linear(fmt, pay, grid.cpu(), x)


# Row tiles times token tiles decide the kernel: rows, blocks, tokens, adapters, rank for each of those of many.
MANY = {torch.bfloat16: [(1100, 3, 500, 3, 5), (1500, 2, 1000, 5, 24), (2000, 5, 1000, 0, 0), (2000, 3, 1100, 30, 17),
                         (4000, 1, 1100, 2, 3), (8000, 2, 1100, 4, 16), (30000, 1, 33, 20, 8), (13000, 2, 9, 4, 6)],
        torch.float32: [(300, 2, 1000, 3, 5), (1100, 3, 1000, 3, 5), (4000, 1, 600, 20, 17), (13000, 2, 9, 4, 6)]}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_many_exact(api, orc, fmt, dtype):
    for i, (rows, nb, T, N, r) in enumerate(MANY[dtype]):
        print("[case] linear many", fmt, dtype, rows, nb, T, N, r, flush=True)
        grid, p, x, a, b, scale, ids, y, size = exact_linear(orc, fmt, rows, nb, T, N, r, 120 + i)
        lora = dict(lora_a=dev(a, dtype), lora_b=dev(b, dtype), lora_scale=dev(scale), lora_ids=dev(ids)) if N else {}
        st = api.new_status()
        got = f64(api.linear(fmt, dev(p), dev(grid), dev(x, dtype), status=st, **lora))
        # exact below 2^13, as above; adapters' sums beyond: 14 additions of exact terms
        sure = size < 2.0 ** 13
        assert sure.mean() > 0.5
        assert np.array_equal(got[sure], round_to(y, dtype)[sure]), (rows, nb, T, N, r)
        near = np.abs(got - y) <= 14 * U * size + np.abs(y) * (2.0 ** -8 if dtype == torch.bfloat16 else U)
        assert near.all(), (rows, nb, T, N, r)
        assert api.read_status(st) == 0


@pytest.mark.parametrize("rows, T", [(60, 100), (1100, 500), (1500, 1000), (2000, 1000), (2000, 1100), (4000, 1100),
                                     (8000, 1100)])
def test_linear_block_scales(api, orc, rows, T):
    """Scales of either sign from the smallest subnormal up to 2^6, blocks and whole rows of zero scale, and a token
    with an infinity in a block that some rows scale by zero (0 * inf: NaN there)."""
    print("[case] linear block scales", rows, T, flush=True)
    for fmt in ("IQ2_S", "IQ1_M"):
        nb = 4
        g = inputs.rng(rows)
        d = np.ldexp(1 + g.random((rows, nb)), g.integers(-24, 6, (rows, nb))).astype(np.float16)
        d = np.where(g.random((rows, nb)) < 0.5, -d, d)
        d[g.random((rows, nb)) < 0.3] = 0
        d[rows // 2:rows // 2 + 3] = 0
        d[0], d[-1, :2] = (0, 0, 0, 1), 0
        grid, p = inputs.grid_for(fmt, 5), payload(fmt, rows, nb, 6, d16=d.astype(np.float16).view(np.uint16))
        x = dev(inputs.activations(T, nb * 256, 7, 8)).bfloat16()
        got = api.linear(fmt, dev(p), dev(grid), x)
        xd, w = f64(x), decoded(orc, fmt, p, grid)
        y, S = xd @ w.T, np.abs(xd) @ np.abs(w).T
        # accumulated over the whole of K: K additions and a rescaling per block; sums in units of another block's
        # scale stay between 2^-60 and 2^80, far from where float32 loses bits or overflows
        tol = ((nb * 258 + 16) * 2 * U) * S + np.abs(y) * 2.0 ** -8 * 1.01
        assert np.all(np.abs(f64(got) - y) <= tol), fmt
        assert bool((got[:, rows // 2:rows // 2 + 3] == 0).all())
        bad = x.clone()
        bad[T // 2, 256 + 5] = float("inf")
        out = api.linear(fmt, dev(p), dev(grid), bad)
        keep = [t for t in range(T) if t != T // 2]
        assert torch.equal(out[keep], got[keep])
        row, zero = out[T // 2].float(), torch.from_numpy(d[:, 1] == 0).cuda()
        assert bool(row[zero].isnan().all())
        at = torch.from_numpy(w[:, 256 + 5]).cuda()
        assert torch.equal(row[~zero], (torch.sign(at) * float("inf")).float()[~zero])


@pytest.mark.parametrize("rows, T", [(1100, 500), (1500, 1000), (2000, 1000), (2000, 1100), (4000, 1100), (8000, 1100)])
def test_linear_many_random(api, orc, rows, T):
    print("[case] linear many random", rows, T, flush=True)
    for fmt, dtype, nb in (("IQ2_XXS", torch.bfloat16, 5), ("IQ1_S", torch.bfloat16, 3), ("IQ2_XS", torch.float32, 3)):
        grid, p = inputs.grid_for(fmt, 41), payload(fmt, rows, nb, rows + 1)
        x = dev(inputs.activations(T, nb * 256, 42, 43, bf16=False), dtype)
        base = api.linear(fmt, dev(p), dev(grid), x)
        got, xd, w = f64(base), f64(x), decoded(orc, fmt, p, grid)
        y, S = xd @ w.T, np.abs(xd) @ np.abs(w).T
        # bf16 sums run through the whole of K, with a rescaling per block
        assert np.all(np.abs(got - y) <= linear_tolerance(xd, w, dtype, y) + nb * 258 * 2 * U * S)
        rel = np.linalg.norm(got - y) / np.linalg.norm(y)
        assert rel < (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20)
        # every token has a scale of its own
        n = torch.arange(T, device="cuda") % 150 - 90
        f = dev(np.ldexp(np.float32(1), n.cpu().numpy()))[:, None]
        assert torch.equal(api.linear(fmt, dev(p), dev(grid), (x.float() * f).to(dtype)).float(), base.float() * f)


# --------------------------------------------------------------------------
# iq_moe
# --------------------------------------------------------------------------
def moe_inputs(fmt, down_fmt, E, H, I, T, dtype, seed, rdtype=None):
    g = inputs.rng(seed)
    grid, dgrid = inputs.grid_for(fmt, 50), inputs.grid_for(down_fmt, 50 if fmt == down_fmt else 51)
    gate, up, down = payload(fmt, E * I, H // 256, seed), payload(fmt, E * I, H // 256, seed + 1), \
        payload(down_fmt, E * H, I // 256, seed + 2)
    x = dev(inputs.activations(T, H, seed + 3, seed + 4, bf16=False), dtype)
    router = dev(g.standard_normal((E, H), dtype=np.float32) / np.float32(np.sqrt(H)), rdtype or dtype)
    return grid, dgrid, gate, up, down, x, router


def moe_reference(orc, fmt, down_fmt, E, H, I, grid, dgrid, gate, up, down, x, ids, weights, dtype):
    """(y, tolerance) in 64 bits."""
    T = x.shape[0]
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    step = 2.0 ** -22 if dtype == torch.float32 else 0.0
    for e in np.unique(ids):
        if not 0 <= e < E:
            continue
        wg = decoded(orc, fmt, gate[e * I:(e + 1) * I], grid)
        wu = decoded(orc, fmt, up[e * I:(e + 1) * I], grid)
        wd = decoded(orc, down_fmt, down[e * H:(e + 1) * H], dgrid)
        for t, s in zip(*np.nonzero(ids == e)):
            g, u, p = x[t] @ wg.T, x[t] @ wu.T, float(weights[t, s])
            c = (276 + H / 256) * 2 * U + step
            dg, du = c * (np.abs(x[t]) @ np.abs(wg).T), c * (np.abs(x[t]) @ np.abs(wu).T)
            silu = g / (1 + np.exp(-g))
            h = silu * u * p
            # silu' <= 1.1
            dh = p * (1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du)
            dh += np.abs(h) * (2.0 ** -20 + (2.0 ** -21 if dtype == torch.float32 else 2.0 ** -11))
            # fp16 below the block's normal range: 2^-39 of the block's largest value
            dh += 2.0 ** -39 * np.abs(h).max()
            y[t] += h @ wd.T
            tol[t] += dh @ np.abs(wd).T + (276 + I / 256 + 128) * 2 * U * (np.abs(h) @ np.abs(wd).T)
    return y, tol + np.abs(y) * (2.0 ** -8 if dtype == torch.bfloat16 else U) * 1.01


MOE_SHAPES = [(4, 1, 256, 256, 1), (8, 2, 512, 256, 5), (5, 3, 768, 512, 17), (16, 8, 256, 768, 33), (3, 3, 512, 256, 70),
              (40, 6, 256, 256, 150)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
def test_moe_random(api, orc, fmt, dtype):
    for i, (E, k, H, I, T) in enumerate(MOE_SHAPES):
        dfmt = FORMATS[(FORMATS.index(fmt) + i) % 5]
        print("[case] moe", fmt, dfmt, dtype, E, k, H, I, T, flush=True)
        grid, dgrid, gate, up, down, x, router = moe_inputs(fmt, dfmt, E, H, I, T, dtype, 70 + 10 * i,
                                                            torch.float32 if i % 2 else None)
        st = api.new_status()
        y, ids, weights = api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), x, E, router=router, top_k=k,
                                  renormalize=i % 3 != 1, down_fmt=dfmt, down_grid=dev(dgrid), status=st)
        assert api.read_status(st) == 0
        logits = f64(x) @ f64(router).T
        want = np.argsort(-logits, axis=1, kind="stable")[:, :k]
        assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), want)
        p = np.exp(logits - logits.max(1, keepdims=True))
        full = p.sum(1, keepdims=True)
        p = np.take_along_axis(p, want, 1)
        p = p / (p.sum(1, keepdims=True) if i % 3 != 1 else full)
        # exp of a float32 difference (relative 2^-24 of at most 40) and a few roundings
        assert np.allclose(f64(weights), p, rtol=2.0 ** -17, atol=0)
        ref, tol = moe_reference(orc, fmt, dfmt, E, H, I, grid, dgrid, gate, up, down, f64(x), want, f64(weights), dtype)
        assert np.all(np.abs(f64(y) - ref) <= tol), (E, k, H, I, T)
        rel = np.linalg.norm(f64(y) - ref) / np.linalg.norm(ref)
        assert rel < (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20)
        # the caller's own routing gives the same layer
        y2, i2, w2 = api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), x, E, ids=ids, weights=weights,
                             down_fmt=dfmt, down_grid=dev(dgrid))
        assert torch.equal(y, y2) and i2 is ids and w2 is weights


# K of the router over four workgroups, each number of experts a lane holds, more than 256 of them, top_k of 64,
# whole rows of few tokens, few tokens with the choice in a launch of its own
MORE_MOE = [("IQ2_XS", 6, 2, 1024, 256, 6), ("IQ1_S", 5, 2, 1280, 256, 20), ("IQ2_S", 200, 9, 256, 256, 7),
            ("IQ1_M", 200, 9, 256, 256, 13), ("IQ2_XXS", 300, 64, 256, 256, 3), ("IQ2_XS", 64, 64, 256, 256, 16),
            ("IQ1_S", 64, 8, 512, 256, 8), ("IQ2_S", 30, 4, 256, 1024, 16), ("IQ2_XXS", 5, 2, 1536, 768, 2),
            ("IQ2_S", 16, 3, 512, 256, 16), ("IQ1_M", 257, 1, 256, 256, 1), ("IQ1_S", 1, 1, 256, 256, 300),
            ("IQ1_M", 1100, 3, 256, 256, 40)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt, E, k, H, I, T", MORE_MOE)
def test_moe_more_shapes(api, orc, fmt, E, k, H, I, T, dtype):
    print("[case] moe more", fmt, dtype, E, k, H, I, T, flush=True)
    grid, _, gate, up, down, x, router = moe_inputs(fmt, fmt, E, H, I, T, dtype, 1000 + E)
    st = api.new_status()
    y, ids, weights = api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), x, E, router=router, top_k=k, status=st)
    assert api.read_status(st) == 0
    logits = f64(x) @ f64(router).T
    want = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids.cpu().numpy(), want)
    p = np.take_along_axis(np.exp(logits - logits.max(1, keepdims=True)), want, 1)
    assert np.allclose(f64(weights), p / p.sum(1, keepdims=True), rtol=2.0 ** -17, atol=0)
    ref, tol = moe_reference(orc, fmt, fmt, E, H, I, grid, grid, gate, up, down, f64(x), want, f64(weights), dtype)
    assert np.all(np.abs(f64(y) - ref) <= tol)
    rel = np.linalg.norm(f64(y) - ref) / np.linalg.norm(ref)
    assert rel < (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20)


def test_moe_most_experts(api):
    """4,096 experts, the most there can be: ids, and the output against the same experts gathered into a small layer."""
    print("[case] moe 4096 experts", flush=True)
    fmt, E, k, H, I, T = "IQ1_S", 4096, 3, 256, 256, 20
    grid, _, gate, up, down, x, router = moe_inputs(fmt, fmt, E, H, I, T, torch.bfloat16, 1300)
    gate, up, down, grid = dev(gate), dev(up), dev(down), dev(grid)
    y, ids, weights = api.moe(fmt, gate, up, down, grid, x, E, router=router, top_k=k)
    want = np.argsort(-(f64(x) @ f64(router).T), axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids.cpu().numpy(), want)
    some = ids.unique()
    pick = lambda p, rows: p.view(E, rows, -1)[some.long()].reshape(-1, 1, p.shape[-1]).contiguous()
    small = torch.searchsorted(some, ids).int()
    y2, _, _ = api.moe(fmt, pick(gate, I), pick(up, I), pick(down, H), grid, x, len(some), ids=small, weights=weights)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("T", [4, 40, 130])
def test_moe_callers_routing(api, orc, T):
    """Ids outside the range, ids repeated in a token, zero weights, a token with no expert at all, experts that
    every token names and experts that none does."""
    print("[case] moe routing", T, flush=True)
    fmt, E, k, H, I, dtype = "IQ2_XS", 7, 4, 512, 256, torch.float32
    grid, dgrid, gate, up, down, x, _ = moe_inputs(fmt, fmt, E, H, I, T, dtype, 500)
    g = inputs.rng(501)
    ids = g.integers(0, 5, (T, k)).astype(np.int32)  # experts 5 and 6 idle; repeats are common
    weights = g.random((T, k)).astype(np.float32)
    ids[:, 0] = 2
    ids[1] = (-1, E, 2 ** 31 - 1, -2 ** 31)
    ids[2] = 3
    weights[3] = 0.0
    st = api.new_status()
    y, _, _ = api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), x, E, ids=dev(ids), weights=dev(weights), status=st)
    assert api.read_status(st) == api.STATUS_BADID
    ref, tol = moe_reference(orc, fmt, fmt, E, H, I, grid, dgrid, gate, up, down, f64(x), ids, weights, dtype)
    assert np.all(np.abs(f64(y) - ref) <= tol)
    assert bool((y[1] == 0).all()) and bool((y[3] == 0).all())


@pytest.mark.parametrize("T", [4, 40])
def test_moe_ties_infinities_and_empty(api, T):
    print("[case] moe ties", T, flush=True)
    fmt, E, k, H, I = "IQ1_M", 70, 5, 256, 256
    grid, _, gate, up, down, x, router = moe_inputs(fmt, fmt, E, H, I, T, torch.bfloat16, 600)
    args = (fmt, dev(gate), dev(up), dev(down), dev(grid))
    router[3:50] = router[2]  # 48 equal logits
    router[50:] = 0
    clean, ids, w = api.moe(*args, x, E, router=router, top_k=k)
    l = x.double() @ router.double().T
    want = l.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    same, ids, w = api.moe(*args, torch.zeros_like(x), E, router=router, top_k=k)
    assert torch.equal(ids.long(), torch.arange(k, device="cuda").expand(T, k)) and bool((same == 0).all())
    assert bool((w == w[0, 0]).all()) and abs(float(w[0, 0]) - 1 / k) < 1e-7
    bad = x.clone()
    bad[1, 7], bad[2, 9] = float("nan"), float("inf")
    y, ids, w = api.moe(*args, bad, E, router=router, top_k=k)
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.equal(ids[1].long(), torch.arange(k, device="cuda")) and bool(y[1].isnan().all())
    assert bool(((ids >= 0) & (ids < E)).all()) and bool((~y[2].isfinite()).all())
    y, ids, w = api.moe(*args, x[:0], E, router=router, top_k=k)
    assert y.shape == (0, H) and ids.shape == (0, k) and w.shape == (0, k)


@pytest.mark.parametrize("T", [3, 50])
def test_moe_views_and_guards(api, T):
    print("[case] moe views", T, flush=True)
    fmt, dfmt, E, k, H, I = "IQ2_S", "IQ1_S", 9, 3, 512, 256
    grid, dgrid, gate, up, down, x, router = moe_inputs(fmt, dfmt, E, H, I, T, torch.bfloat16, 700)
    kw = dict(down_fmt=dfmt, down_grid=dev(dgrid), top_k=k)
    want, wi, ww = api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), x, E, router=router, **kw)

    need = api.moe_workspace_size(fmt, H, I, E, x.dtype, T, k, dfmt)
    ws = torch.full((need + 100,), 7, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 2, H), 7.0, dtype=x.dtype, device="cuda")
    ids = torch.full((T + 2, k), 7, dtype=torch.int32, device="cuda")
    weights = torch.full((T + 2, k), 7.0, device="cuda")
    api.moe(fmt, shifted(dev(gate), 2), shifted(dev(up), 6), shifted(dev(down), 2), odd(dev(grid)), odd(x), E,
            router=odd(router), **kw,
            ids=ids[1:T + 1], weights=weights[1:T + 1], out=out[1:T + 1], workspace=ws[1:need + 1])
    assert torch.equal(out[1:T + 1], want) and torch.equal(ids[1:T + 1], wi) and torch.equal(weights[1:T + 1], ww)
    for t in (out, ids, weights):
        assert bool((t[0] == 7).all()) and bool((t[T + 1] == 7).all())
    assert int(ws[0]) == 7 and bool((ws[need + 1:] == 7).all())
    with pytest.raises(api.IQError):
        api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), x, E, router=router, workspace=ws[:need - 1], **kw)


# --------------------------------------------------------------------------
# Streams, graphs, and a run of the calls together
# --------------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 24, 140, 1100])
def test_streams_graphs_and_repeats(api, T):
    """The same bits on every call, on another stream, and from a captured graph on new inputs after each replay;
    two graphs with a workspace each, replayed in turn."""
    print("[case] streams graphs", T, flush=True)
    fmt, E, k, H, I, N, r = "IQ2_XXS", 10, 4, 512, 256, 3, 8
    grid, _, gate, up, down, x, router = moe_inputs(fmt, fmt, E, H, I, T, torch.bfloat16, 800)
    grid, gate, up, down = dev(grid), dev(gate), dev(up), dev(down)
    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randn((N, r, H), device="cuda", generator=g).bfloat16()
    b = torch.randn((N, E * I, r), device="cuda", generator=g).bfloat16()
    ids = torch.randint(-1, N, (T,), device="cuda", generator=g, dtype=torch.int32)

    def both(x, **kw):
        return (api.linear(fmt, gate, grid, x, a, b, None, ids, workspace=kw.get("w1"), out=kw.get("o1")),
                *api.moe(fmt, gate, up, down, grid, x, E, router=router, top_k=k, workspace=kw.get("w2"),
                         out=kw.get("o2"), ids=kw.get("i2"), weights=kw.get("p2")))
    want = both(x)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(both(x), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both(x)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(other, want))

    graphs = []
    for n in range(2):
        xs = x.clone()
        w1 = torch.empty(api.linear_workspace_size(fmt, E * I, H, x.dtype, T, r), dtype=torch.uint8, device="cuda")
        w2 = torch.empty(api.moe_workspace_size(fmt, H, I, E, x.dtype, T, k), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = both(xs, w1=w1, w2=w2)
        graphs.append((graph, xs, outs, w1, w2))
    for n in range(4):
        new = (x.float() * (0.5 + n)).roll(n, 1).bfloat16()
        fresh = both(new)
        for graph, xs, outs, w1, w2 in graphs:
            xs.copy_(new)
            w1.fill_(255)
            w2.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(outs, fresh))


def test_encode_then_run_then_collect(api, orc):
    """As they are used together: experts encoded with their importance, tokens through the layer, and the layer's
    ids fed to the collector; a projection encoded and run against its own decode."""
    print("[case] encode, run, collect", flush=True)
    fmt, E, k, H, I, T = "IQ2_XS", 5, 2, 512, 256, 60
    grid = inputs.grid_for(fmt, 202)
    gd = dev(grid)
    x = dev(inputs.activations(T, H, 900, 901)).bfloat16()
    router = dev(inputs.weight(E, H, 902)).bfloat16()
    sums, counts = api.imatrix_collect(x)
    imp = api.imatrix_importance(sums, counts)
    enc = {}
    for n, (rows, cols, s) in {"gate": (I, H, 903), "up": (I, H, 904), "down": (H, I, 905)}.items():
        w = dev(inputs.weight(E * rows, cols, s))
        enc[n] = api.quantize(fmt, w, gd, imp.expand(E, H).contiguous() if cols == H else None, rows_per_expert=rows,
                              check=True)
    y, ids, weights = api.moe(fmt, enc["gate"], enc["up"], enc["down"], gd, x, E, router=router, top_k=k)
    host = {n: p.cpu().numpy() for n, p in enc.items()}
    ref, tol = moe_reference(orc, fmt, fmt, E, H, I, grid, grid, host["gate"], host["up"], host["down"], f64(x),
                             ids.cpu().numpy(), f64(weights), torch.bfloat16)
    assert np.all(np.abs(f64(y) - ref) <= tol)
    s2, c2 = api.imatrix_collect(x, ids, num_experts=E)
    so, co, _ = orc.collect(x.float().cpu().numpy(), ids.cpu().numpy(), E)
    assert np.array_equal(c2.cpu().numpy(), co) and np.allclose(f64(s2), so, rtol=1e-5)
    got = f64(api.linear(fmt, enc["gate"], gd, x.float()))
    w = f64(api.dequantize(fmt, enc["gate"], gd))
    want = f64(x) @ w.T
    assert np.all(np.abs(got - want) <= linear_tolerance(f64(x), w, torch.float32, want))


def test_large_offsets(api, orc):
    """Payloads beyond 2^31 bytes: the rows behind that offset are read, and outputs behind 2^31 bytes written."""
    print("[case] large offsets", flush=True)
    fmt, rows, nb = "IQ1_S", 1 << 22, 11  # 2.3 GB of payload
    grid = inputs.grid_for(fmt, 5)
    tail = payload(fmt, 64, nb, 6)
    p = torch.zeros((rows, nb, 50), dtype=torch.uint8, device="cuda")
    p[-64:] = dev(tail)
    x = inputs.activations(140, nb * 256, 7, 8)
    w = decoded(orc, fmt, tail, grid)
    for T in (1, 20, 140):  # 140 x 2^22 float32 outputs: 2.3 GB
        y = api.linear(fmt, p, dev(grid), dev(x[:T]))
        got, want = f64(y[:, -64:]), x[:T].astype(np.float64) @ w.T
        assert np.all(np.abs(got - want) <= linear_tolerance(x[:T].astype(np.float64), w, torch.float32, want))
        assert bool((y[:, :-64] == 0).all())
        del y


@pytest.mark.parametrize("T", [2, 16, 48, 400])
def test_two_calls_at_once(api, T):
    """Calls in flight on two streams, each with memory of its own, are the calls one after the other."""
    print("[case] two calls at once", T, flush=True)
    fmt, E, k, H, I = "IQ2_S", 16, 4, 512, 512
    grid, _, gate, up, down, x, router = moe_inputs(fmt, fmt, E, H, I, T, torch.bfloat16, 1400)
    grid, gate, up, down = dev(grid), dev(gate), dev(up), dev(down)
    xs = [x, (x.float() * 0.5).roll(1, 0).bfloat16()]

    def both(x):
        return (api.linear(fmt, gate, grid, x), *api.moe(fmt, gate, up, down, grid, x, E, router=router, top_k=k))
    want = [both(v) for v in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [[], []]
    for _ in range(8):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(both(xs[n]))
    torch.cuda.synchronize()
    for n in range(2):
        for g in got[n]:
            assert all(torch.equal(p, q) for p, q in zip(g, want[n]))


def test_large_offsets_in_prompts(api, orc):
    """bf16 tokens over a payload of more than 2^31 bytes: the rows behind that offset, in the kernels for prompts."""
    print("[case] large offsets, prompts", flush=True)
    fmt, rows, nb = "IQ1_S", 1 << 22, 11
    grid = inputs.grid_for(fmt, 5)
    tail = payload(fmt, 64, nb, 6)
    p = torch.zeros((rows, nb, 50), dtype=torch.uint8, device="cuda")
    p[-64:] = dev(tail)
    x = dev(inputs.activations(300, nb * 256, 7, 8)).bfloat16()
    w = decoded(orc, fmt, tail, grid)
    for T in (1, 20, 40, 300):  # 300 x 2^22 bf16 outputs: 2.5 GB
        y = api.linear(fmt, p, dev(grid), x[:T])
        got, xd = f64(y[:, -64:]), f64(x[:T])
        want, S = xd @ w.T, np.abs(xd) @ np.abs(w).T
        assert np.all(np.abs(got - want) <= linear_tolerance(xd, w, torch.bfloat16, want) + nb * 258 * 2 * U * S)
        assert bool((y[:, :-64] == 0).all())
        del y


# (experts, top_k, hidden, inter, tokens): the waves that share an expert's blocks, whole rows of few tokens, and one,
# two and four tiles of pairs; more blocks than a stage of h holds
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("down_fmt", ["IQ2_XXS", "IQ2_S", "IQ1_S"])
@pytest.mark.parametrize("E, k, H, I, T", [(4, 2, 512, 256, 1), (4, 2, 512, 768, 5), (4, 2, 512, 768, 12),
                                           (6, 2, 512, 768, 24), (4, 2, 256, 768, 40), (3, 1, 512, 1280, 120)])
def test_moe_keeps_the_bits_of_h(api, orc, E, k, H, I, T, down_fmt, dtype):
    """h of 12 and 13 bits beside sums that float32 holds exactly: the layer rounds nothing but its output."""
    print("[case] moe bits of h", E, k, H, I, T, down_fmt, dtype, flush=True)
    g = inputs.rng(1500 + T)
    fmt = "IQ2_XXS"
    grid = inputs.grid_for(fmt, 5)
    grid[0] = 1

    def rows_of(m, signs):
        """Rows whose weights at columns 0 and 32 are +-m[:, 0] and +-m[:, 1] (odd, 1 to 31)."""
        p = np.zeros((len(m), H // 256, 66), dtype=np.uint8)
        p[..., 0], p[..., 1] = 0x00, 0x48  # d = 8, and a weight is d / 8 times its integers
        for n in range(2):
            p[:, 0, 2 + 8 * n + 7] = (m[:, n] // 2) << 4
            p[:, 0, 2 + 8 * n + 4] = signs[n] & 127  # the eighth sign is the seven's parity, of a column that is zero
        return p

    # x = 2^n at column 0 and 2^n 32 at column 32: g = 2^n (m0 + 32 m1) >= 33, where silu(g) = g in float32, and
    # u = 2^n (m0 - 32) with m0 of 27 to 31
    gate = rows_of(2 * g.integers(0, 16, (E * I, 2)) + 1, (0, 0))
    up = rows_of(np.stack((2 * g.integers(13, 16, E * I) + 1, np.ones(E * I, dtype=np.int64)), 1), (0, 1))
    dgrid = grid if down_fmt == fmt else inputs.grid_for(down_fmt, 51)
    down = payload(down_fmt, E * H, I // 256, 1501 + T, d16=0x4800)
    if down_fmt == fmt:
        down.reshape(-1, I // 256, 66)[..., 9::8] &= 15  # multipliers of one: weights of +-1, 3, 5
    elif down_fmt == "IQ2_S":
        down[..., 74:] = 0
    else:
        down[..., 35::2] &= 0x8f  # and here eighths: 1, 7 and 9 of them
    x = np.zeros((T, H), dtype=np.float32)
    x[:, 0] = 2.0 ** g.integers(0, 3, T)
    x[:, 32] = 32 * x[:, 0]
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    weights = g.choice([-1.0, 1.0], (T, k)).astype(np.float32)
    wg, wu, wd = decoded(orc, fmt, gate, grid), decoded(orc, fmt, up, grid), decoded(orc, down_fmt, down, dgrid)
    y, size = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, s = np.nonzero(ids == e)
        if not len(t):
            continue
        a, b = x[t] @ wg[e * I:(e + 1) * I].T, x[t] @ wu[e * I:(e + 1) * I].T
        assert a.min() >= 33 and np.array_equal(a, a.astype(np.int64)) and np.abs(b).max() <= 4 * 5
        h = a * b * weights[t, s, None]
        np.add.at(y, t, h @ wd[e * H:(e + 1) * H].T)
        np.add.at(size, t, np.abs(h) @ np.abs(wd[e * H:(e + 1) * H]).T / x[t, :1] ** 2)
    assert size.max() < 2.0 ** 24  # in units of the token's own step: every partial sum, in any order, is exact
    assert np.array_equal(y, y.astype(np.float32))
    got, _, _ = api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), dev(x, dtype), E, ids=dev(ids),
                        weights=dev(weights), down_fmt=down_fmt, down_grid=dev(dgrid))
    assert np.array_equal(f64(got), round_to(y, dtype))


@pytest.mark.parametrize("T", [1, 20, 40, 300])
def test_linear_wide_tokens(api, orc, T):
    """bf16 tokens of more than 6,144 columns (float32: 2,048), which the conversion reads twice; the largest value in
    each part of a row in turn."""
    print("[case] linear wide", T, flush=True)
    for fmt, dtype, nb in (("IQ2_XXS", torch.bfloat16, 25), ("IQ1_M", torch.bfloat16, 49), ("IQ2_S", torch.float32, 25)):
        grid, p = inputs.grid_for(fmt, 41), payload(fmt, 40, nb, 1600 + nb)
        x = dev(inputs.activations(T, nb * 256, 42, 43, bf16=False), dtype)
        at = torch.arange(T, device="cuda") * 911 % (nb * 256)
        at[0] = nb * 256 - 1
        x[torch.arange(T, device="cuda"), at] = 1000.0
        got, xd, w = f64(api.linear(fmt, dev(p), dev(grid), x)), f64(x), decoded(orc, fmt, p, grid)
        y = xd @ w.T
        assert np.all(np.abs(got - y) <= linear_tolerance(xd, w, dtype, y)), (fmt, dtype)
        rel = np.linalg.norm(got - y) / np.linalg.norm(y)
        assert rel < (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20)


# Blocks of K as real layers have them.  Gate and up with K split over eight waves, some with a second block (1 and 16
# tokens), whole rows of few tokens; down in more than one stage of h with one, two and four tiles of pairs
DEEP_MOE = [("IQ2_XXS", 4, 2, 2304, 256, 1), ("IQ2_S", 4, 2, 4096, 512, 1), ("IQ1_M", 3, 2, 2304, 1280, 16),
            ("IQ2_XS", 8, 2, 2304, 1280, 16), ("IQ1_S", 4, 1, 512, 2304, 20), ("IQ2_XS", 3, 2, 512, 1280, 25),
            ("IQ2_XXS", 2, 2, 512, 2304, 60), ("IQ1_M", 2, 1, 4096, 512, 70)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt, E, k, H, I, T", DEEP_MOE)
def test_moe_deep(api, orc, fmt, E, k, H, I, T, dtype):
    test_moe_more_shapes(api, orc, fmt, E, k, H, I, T, dtype)


@pytest.mark.parametrize("T", [1, 12, 40])
def test_moe_large_offsets(api, T):
    """256 experts in payloads of more than 2^31 bytes each: the last one, against the same expert in a small layer."""
    print("[case] moe large offsets", T, flush=True)
    fmt, E, H, I = "IQ1_S", 256, 16384, 4096  # 3.4 GB each of gate, up and down
    grid = dev(inputs.grid_for(fmt, 5))
    one = [dev(payload(fmt, rows, nb, 1700 + n)) for n, (rows, nb) in enumerate([(I, H // 256), (I, H // 256), (H, I // 256)])]

    def layer(experts):
        out = []
        for p in one:
            full = torch.zeros((experts * p.shape[0], *p.shape[1:]), dtype=torch.uint8, device="cuda")
            full[-p.shape[0]:] = p
            out.append(full)
        return out
    big, small = layer(E), layer(5)
    assert min(p.numel() for p in big) > 2 ** 31
    x = dev(inputs.activations(T, H, 7, 8)).bfloat16()
    ids = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
    if T > 2:
        ids[1] = 3  # an expert of zeros
    weights = torch.full((T, 1), 0.5, device="cuda")
    y, _, _ = api.moe(fmt, *big, grid, x, E, ids=ids, weights=weights)
    want, _, _ = api.moe(fmt, *small, grid, x, 5, ids=torch.where(ids == E - 1, 4, ids), weights=weights)
    assert torch.equal(y, want) and bool(y[0].isfinite().all()) and bool((y[0] != 0).any())
    if T > 2:
        assert bool((y[1] == 0).all())


@pytest.mark.parametrize("rows, T", [(1100, 500), (2000, 1000), (4000, 1100), (8000, 1100)])
def test_linear_wide_prompts(api, orc, rows, T):
    """The kernels for prompts over 25 blocks of K."""
    print("[case] linear wide prompts", rows, T, flush=True)
    fmt, nb = "IQ2_XS", 25
    grid, p = inputs.grid_for(fmt, 41), payload(fmt, rows, nb, 1800 + rows)
    x = dev(inputs.activations(T, nb * 256, 42, 43, bf16=False), torch.bfloat16)
    got, xd, w = f64(api.linear(fmt, dev(p), dev(grid), x)), f64(x), decoded(orc, fmt, p, grid)
    y, S = xd @ w.T, np.abs(xd) @ np.abs(w).T
    # sums that run through the whole of K, with a rescaling per block
    assert np.all(np.abs(got - y) <= linear_tolerance(xd, w, torch.bfloat16, y) + nb * 258 * 2 * U * S)
    assert np.linalg.norm(got - y) / np.linalg.norm(y) < 2.0 ** -8


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r", [100, 513, 1024])
def test_linear_large_ranks(api, orc, r, dtype):
    fmt, nb, N = "IQ2_XXS", 3, 2
    for rows, T in ((40, 1), (70, 45), (1100, 500)):
        print("[case] linear large ranks", r, dtype, rows, T, flush=True)
        g = inputs.rng(r + T)
        grid, p = inputs.grid_for(fmt, 41), payload(fmt, rows, nb, 1900 + r)
        x = dev(inputs.activations(T, nb * 256, 42, 43, bf16=False), dtype)
        a = dev(g.standard_normal((N, r, nb * 256), dtype=np.float32) * 0.02, dtype)
        b = dev(g.standard_normal((N, rows, r), dtype=np.float32) * 0.02, dtype)
        ids = g.integers(-1, N, T).astype(np.int32)
        ids[0] = 1
        got = f64(api.linear(fmt, dev(p), dev(grid), x, lora_a=a, lora_b=b, lora_ids=dev(ids)))
        xd, w = f64(x), decoded(orc, fmt, p, grid)
        y, more = xd @ w.T, nb * 258 * 2 * U * (np.abs(xd) @ np.abs(w).T)
        for n in range(N):
            at = ids == n
            y[at] += (xd[at] @ f64(a)[n].T) @ f64(b)[n].T
            # K additions for v; r more for its product with B, each of three parts
            more[at] += (nb * 256 + 3 * r + 8) * 2 * U * ((np.abs(xd[at]) @ np.abs(f64(a)[n]).T) @ np.abs(f64(b)[n]).T)
        assert np.all(np.abs(got - y) <= linear_tolerance(xd, w, dtype, y) + more), (rows, T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows, T", [(50, 3), (50, 40), (1100, 500), (2000, 1000), (4000, 1100)])
def test_linear_small_values_beside_a_large_one(api, orc, rows, T, dtype):
    """A token's largest value meets a block of zero scale; the rest, 2^-30 and 2^-38 of it, are integers whose sums
    float32 holds exactly: multiples of 2^-24 in fp16 under the token's power of two, subnormal ones included."""
    print("[case] linear small beside large", rows, T, dtype, flush=True)
    for fmt in ("IQ2_XS", "IQ1_M"):
        nb = 3
        g = inputs.rng(rows + T)
        grid = inputs.grid_for(fmt, 5)
        d = np.full((rows, nb), 0x2000)  # 2^-7
        d[:, 0] = 0
        p = payload(fmt, rows, nb, 2000 + rows, d16=d)
        x = g.integers(-8, 9, (T, nb * 256)).astype(np.float32)
        x[:, 17] = np.where(np.arange(T) % 2, np.float32(2.0 ** 30), np.float32(2.0 ** 38))
        w = decoded(orc, fmt, p, grid)
        y, size = x.astype(np.float64) @ w.T, np.abs(x[:, 256:]).astype(np.float64) @ np.abs(w[:, 256:]).T
        assert size.max() < 2.0 ** 13  # in steps of 2^-10: every partial sum is exact
        got = api.linear(fmt, dev(p), dev(grid), dev(x, dtype))
        assert np.array_equal(f64(got), round_to(y, dtype)), fmt


@pytest.mark.parametrize("T", [7, 16, 40])
def test_moe_more_choices_than_experts(api, orc, T):
    """The caller's routing may name 64 experts a token of a layer of two."""
    print("[case] moe repeats", T, flush=True)
    for fmt, dtype in (("IQ2_S", torch.bfloat16), ("IQ1_S", torch.float32)):
        E, k, H, I = 2, 64, 512, 256
        grid, _, gate, up, down, x, _ = moe_inputs(fmt, fmt, E, H, I, T, dtype, 2100)
        g = inputs.rng(2101)
        ids = g.integers(0, E, (T, k)).astype(np.int32)
        ids[0] = 1
        weights = (g.random((T, k)) / k).astype(np.float32)
        y, _, _ = api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), x, E, ids=dev(ids), weights=dev(weights))
        ref, tol = moe_reference(orc, fmt, fmt, E, H, I, grid, grid, gate, up, down, f64(x), ids, weights, dtype)
        assert np.all(np.abs(f64(y) - ref) <= tol)


@pytest.mark.parametrize("T", [3, 20])
def test_moe_router_of_another_type(api, T):
    """float32 tokens with a bf16 router: the choice and its weights as 64 bits have them."""
    print("[case] moe router type", T, flush=True)
    fmt, E, k, H, I = "IQ2_XXS", 30, 4, 1024, 256
    grid, _, gate, up, down, x, router = moe_inputs(fmt, fmt, E, H, I, T, torch.float32, 2200, torch.bfloat16)
    y, ids, weights = api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), x, E, router=router, top_k=k)
    logits = f64(x) @ f64(router).T
    want = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids.cpu().numpy(), want)
    p = np.take_along_axis(np.exp(logits - logits.max(1, keepdims=True)), want, 1)
    assert np.allclose(f64(weights), p / p.sum(1, keepdims=True), rtol=2.0 ** -17, atol=0)
    y2, _, _ = api.moe(fmt, dev(gate), dev(up), dev(down), dev(grid), x, E, ids=ids, weights=weights)
    assert torch.equal(y, y2)
