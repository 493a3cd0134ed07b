"""Adapting a model whose weights stay encoded, as it is measured: a gated feed-forward block's two
projections, activation and product on IQ payloads with its backward pass, the backward pass of an
encoded projection with the low-rank adapters beside it, and the activations that wait for a
backward pass, kept in 8 bits.

Each case runs either in its plain form (elementary torch operations in 32 bits, one rounding at
the end) or, where `own` is true, through the framework's entry points.  `exact` gives the same
results in 64 bits, written apart from the plain form.
"""
import math

import torch

own = False

GRID_SIZE = {"IQ2_XXS": 256, "IQ2_XS": 512, "IQ2_S": 1024, "IQ1_S": 2048, "IQ1_M": 2048}
BLOCK_BYTES = {"IQ2_XXS": 66, "IQ2_XS": 74, "IQ2_S": 82, "IQ1_S": 50, "IQ1_M": 56}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTIVATIONS = ("silu", "gelu", "gelu_tanh")
LARGEST = 2.8e12  # operations of the largest listed case, rounded down


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _checkpoint(name, tokens, cols, dtype="bf16"):
    return {"name": name, "op": "checkpoint", "tokens": tokens, "cols": cols, "dtype": dtype}


def _glu(name, fmt, inter, hidden, tokens, activation="silu", dtype="bf16"):
    return {"name": name, "op": "glu", "fmt": fmt, "inter": inter, "hidden": hidden, "tokens": tokens,
            "activation": activation, "dtype": dtype}


def _glu_backward(name, fmt, inter, hidden, tokens, kept, activation="silu", dtype="bf16"):
    # kept: x waits for the backward pass as a checkpoint in 8 bits, not as it was
    return {"name": name, "op": "glu_backward", "fmt": fmt, "inter": inter, "hidden": hidden, "tokens": tokens,
            "kept": kept, "activation": activation, "dtype": dtype}


def _linear_backward(name, fmt, rows, cols, tokens, adapters, rank, kept, dtype="bf16"):
    return {"name": name, "op": "linear_backward", "fmt": fmt, "rows": rows, "cols": cols, "tokens": tokens,
            "adapters": adapters, "rank": rank, "kept": kept, "dtype": dtype}


def listed():
    return [
        # float32 activations of a short sequence, whose last block of 32 is not full
        _checkpoint("checkpoint small", 37, 1001, "f32"),
        # a wide layer's inputs for a batch of sequences
        _checkpoint("checkpoint 8192 tokens", 8192, 17408),
        # one user generating: every step reads both projections for one token
        _glu("glu one token", "IQ2_XS", 5632, 2048, 1),
        # a serving batch
        _glu("glu 48 requests", "IQ1_M", 17408, 5120, 48),
        # odd sizes in float32: rows that end inside a tile, a ragged batch, another activation
        _glu("glu ragged", "IQ2_S", 1001, 768, 37, "gelu_tanh", "f32"),
        # a long prompt, or a training batch's forward pass
        _glu("glu 4096 tokens", "IQ1_S", 17408, 5120, 4096),
        # a small layer in float32, its input as it was
        _glu_backward("glu backward ragged", "IQ2_XXS", 777, 512, 19, False, "gelu", "f32"),
        # a training batch through a small model's layer
        _glu_backward("glu backward 2048 tokens", "IQ2_XS", 5632, 2048, 2048, True),
        # and through a wide one's
        _glu_backward("glu backward 4096 tokens", "IQ1_M", 17408, 5120, 4096, True),
        # float32 throughout, two small adapters of an odd rank in one small batch
        _linear_backward("linear backward ragged", "IQ2_S", 333, 768, 21, 2, 5, False, "f32"),
        # one adapter in training on a small model's down projection
        _linear_backward("linear backward 2048 tokens", "IQ2_XXS", 2048, 5632, 2048, 1, 16, True),
        # four adapters trained side by side on a wide one's
        _linear_backward("linear backward 4096 tokens", "IQ1_S", 5120, 17408, 4096, 4, 32, True),
    ]


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    while True:
        dtype = "f32" if rng.random() < 0.25 else "bf16"
        fmt = rng.choice(sorted(GRID_SIZE))
        activation = rng.choice(ACTIVATIONS)
        rows, cols, tokens = _log(rng, 32, 17408), 256 * _log(rng, 1, 20), _log(rng, 1, 4096)
        kept = rng.random() < 0.6
        op = rng.choice(("checkpoint", "glu", "glu_backward", "linear_backward"))
        if op == "checkpoint":
            c = _checkpoint("", _log(rng, 1, 8192), _log(rng, 32, 17408), dtype)
        elif op == "glu":
            c = _glu("", fmt, rows, cols, tokens, activation, dtype)
        elif op == "glu_backward":
            c = _glu_backward("", fmt, rows, cols, tokens, kept, activation, dtype)
        else:
            rank = _log(rng, 1, 64)
            adapters = 0 if rng.random() < 0.2 else min(_log(rng, 1, 16), max(1, 256 // rank))
            c = _linear_backward("", fmt, rows, cols, tokens, adapters, rank if adapters else 0,
                                 kept and adapters > 0, dtype)
        if work(c)["flops"] <= LARGEST:
            del c["name"]
            return c


def work(case):
    T, size = case["tokens"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "checkpoint":  # x read, codes and exponents written; both read, the values written
        n, blocks = T * case["cols"], T * -(-case["cols"] // 32)
        return {"bytes": 2 * (n * size + n + blocks), "flops": 4 * n}
    if case["op"] == "linear_backward":
        rows, cols, N, r = case["rows"], case["cols"], case["adapters"], case["rank"]
        nbytes = rows * (cols // 256) * BLOCK_BYTES[case["fmt"]] + GRID_SIZE[case["fmt"]] * 32
        nbytes += T * (rows + cols) * size
        if N:  # x for the gradients, the adapters in and their gradients out
            nbytes += T * cols * (33 / 32 if case["kept"] else size) + 2 * N * r * (rows + cols) * size + T * 4
        return {"bytes": nbytes, "flops": 2 * T * rows * cols + (6 * T * r * (rows + cols) if N else 0)}
    I, H = case["inter"], case["hidden"]
    nbytes = 2 * I * (H // 256) * BLOCK_BYTES[case["fmt"]] + GRID_SIZE[case["fmt"]] * 32
    if case["op"] == "glu":
        return {"bytes": nbytes + T * (H + I) * size, "flops": 4 * T * I * H}
    return {"bytes": nbytes + T * (H + I) * size + T * H * (33 / 32 if case["kept"] else size), "flops": 8 * T * I * H}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _grid(fmt, gen):
    """Distinct 8-tuples over the layout's three values, ascending by code, as the encoder's seeded codebooks."""
    codes = torch.randperm(3 ** 8, generator=gen, device="cuda")[:GRID_SIZE[fmt]].sort().values
    digits = (codes[:, None] // (3 ** torch.arange(8, device="cuda"))) % 3
    values = torch.tensor([-1.0, 0.0, 1.0] if fmt.startswith("IQ1") else [1.0, 3.0, 5.0], device="cuda")
    return values[digits].contiguous()


def _payload(fmt, rows, cols, gen):
    """Encoded blocks of a weight whose values spread by about 0.02: free index, sign and scale fields,
    block scales as the encoder anchors them, and a block in 500 that is all zeros."""
    nb, size = cols // 256, BLOCK_BYTES[fmt]
    p = torch.randint(0, 256, (rows, nb, size), dtype=torch.uint8, device="cuda", generator=gen)
    d = 0.0035 * torch.exp(0.25 * torch.randn((rows, nb), device="cuda", generator=gen))
    d16 = d.to(torch.float16).view(torch.int16).to(torch.int32) & 0xFFFF
    if fmt == "IQ1_M":  # one nibble of the scale in the top of each of the last four words
        for w in range(4):
            p[..., 49 + 2 * w] = (p[..., 49 + 2 * w] & 15) | (((d16 >> (4 * w)) & 15) << 4).to(torch.uint8)
    else:
        p[..., 0], p[..., 1] = (d16 & 255).to(torch.uint8), (d16 >> 8).to(torch.uint8)
    p[torch.rand((rows, nb), device="cuda", generator=gen) < 0.002] = 0
    return p


def _tokens(T, cols, dtype, gen):
    sigma = torch.exp(torch.randn(cols, device="cuda", generator=gen))
    return (torch.randn((T, cols), device="cuda", generator=gen) * sigma).to(dtype)


def _upstream(T, cols, dtype, gen):
    """A gradient that arrives from the layers above: small, of another size for every token, and zero for a
    token in 20 (masked out of the loss)."""
    size = 1e-4 * torch.exp(torch.randn((T, 1), device="cuda", generator=gen))
    size = size * (torch.rand((T, 1), device="cuda", generator=gen) >= 0.05)
    return (torch.randn((T, cols), device="cuda", generator=gen) * size).to(dtype)


def _keep(x):
    """A checkpoint of x: int8 codes, and a power of two (its exponent in a byte) for each block of 32 columns."""
    T, cols = x.shape
    blocks = torch.nn.functional.pad(x.float(), (0, -cols % 32)).unflatten(1, (-1, 32))
    most = blocks.abs().amax(-1, keepdim=True)
    e = ((most.view(torch.int32) >> 23) & 255).clamp(min=1)
    unit = torch.pow(2.0, (133 - e).double())  # values in units of 2^(e - 133): the largest lies in 64 .. 128
    e = e + ((most.double() * unit).round() > 127).to(e.dtype) * (e < 254).to(e.dtype)
    codes = (blocks.double() * torch.pow(2.0, (133 - e).double())).round().clamp(-127, 127)
    return codes.flatten(1)[:, :cols].to(torch.int8).contiguous(), e[..., 0].to(torch.uint8).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, T = DTYPE[case["dtype"]], case["tokens"]
    s = {"op": case["op"], "dtype": dtype}
    if case["op"] == "checkpoint":
        s["x"] = _tokens(T, case["cols"], dtype, gen)
        return s
    s["fmt"] = fmt = case["fmt"]
    s["grid"] = _grid(fmt, gen)
    if case["op"] == "linear_backward":
        rows, cols, N, r = case["rows"], case["cols"], case["adapters"], case["rank"]
        s["packed"] = _payload(fmt, rows, cols, gen)
        s["dy"] = _upstream(T, rows, dtype, gen)
        if N:
            x = _tokens(T, cols, dtype, gen)
            s["x"] = _keep(x) if case["kept"] else x
            s["a"] = (torch.randn((N, r, cols), device="cuda", generator=gen) / math.sqrt(cols)).to(dtype)
            s["b"] = (torch.randn((N, rows, r), device="cuda", generator=gen) * 0.02).to(dtype)
            s["scale"] = 2.0 ** torch.randint(-1, 2, (N,), device="cuda", generator=gen).float()
            # the sequences of a batch lie one after the other, each with its adapter; -1: none
            s["ids"] = torch.randint(-1 if N > 1 else 0, N, (T,), device="cuda", generator=gen,
                                     dtype=torch.int32).sort().values
        return s
    I, H = case["inter"], case["hidden"]
    s["activation"] = case["activation"]
    s["gate"], s["up"] = _payload(fmt, I, H, gen), _payload(fmt, I, H, gen)
    x = _tokens(T, H, dtype, gen)
    if case["op"] == "glu_backward":
        s["dh"] = _upstream(T, I, dtype, gen)
    s["x"] = _keep(x) if case.get("kept") else x
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _decode(fmt, packed, grid):
    """The weight's values in 32 bits: uint8 [..., blocks, bytes] -> [..., blocks * 256]."""
    p = packed.to(torch.int32)
    u16 = p[..., 0::2] | (p[..., 1::2] << 8)
    sub = torch.arange(4, device=p.device, dtype=torch.int32)
    shape = p.shape[:-1]
    mask = h = None
    if fmt == "IQ2_XXS":
        w = u16[..., 1:].unflatten(-1, (8, 4))
        k = torch.stack((w[..., 0] & 255, w[..., 0] >> 8, w[..., 1] & 255, w[..., 1] >> 8), -1)
        word = w[..., 2].to(torch.int64) | (w[..., 3].to(torch.int64) << 16)
        mask = (word[..., None] >> (7 * sub)).to(torch.int32) & 127
        ls = (word >> 28).to(torch.int32)[..., None].expand(mask.shape)
    elif fmt == "IQ2_XS":
        v = u16[..., 1:33]
        k, mask = v & 511, v >> 9
        ls = torch.stack((p[..., 66:74] & 15, p[..., 66:74] >> 4), -1).repeat_interleave(2, -1)
    elif fmt == "IQ2_S":
        k = p[..., 2:34] | (((p[..., 66:74, None] >> (2 * sub)) & 3) << 8).reshape(*shape, 32)
        mask = p[..., 34:66]
        ls = torch.stack((p[..., 74:82] & 15, p[..., 74:82] >> 4), -1).repeat_interleave(2, -1)
    elif fmt == "IQ1_S":
        w = u16[..., 17:25, None]
        k = p[..., 2:34].unflatten(-1, (8, 4)) | (((w >> (3 * sub)) & 7) << 8)
        ls, h = ((w >> 12) & 7).expand(k.shape), (w >> 15).expand(k.shape)
    else:
        nib = torch.stack((p[..., 32:48] & 15, p[..., 32:48] >> 4), -1).reshape(*shape, 32)
        k, h = p[..., 0:32] | ((nib & 7) << 8), nib >> 3
        w = u16[..., 24:28]
        ls = ((w[..., None] >> (3 * sub)) & 7).reshape(*shape, 16).repeat_interleave(2, -1)
    if fmt == "IQ1_M":
        d16 = ((u16[..., 24:28] >> 12) << (4 * sub)).sum(-1)
    else:
        d16 = u16[..., 0]
    d = d16.to(torch.int16).view(torch.float16).float()
    k, ls = k.reshape(*shape, 32), ls.reshape(*shape, 32).float()
    values = grid[k.long()]
    if fmt.startswith("IQ1"):
        values = values + (0.125 - 0.25 * h.reshape(*shape, 32).float())[..., None]
        scale = d[..., None] * (2 * ls + 1)
    else:
        mask = mask.reshape(*shape, 32)
        if fmt != "IQ2_S":  # the eighth sign is the parity of the seven
            odd = mask ^ (mask >> 4)
            odd = odd ^ (odd >> 2)
            mask = mask | (((odd ^ (odd >> 1)) & 1) << 7)
        j = torch.arange(8, device=p.device, dtype=torch.int32)
        values = values * (1 - 2 * ((mask[..., None] >> j) & 1)).float()
        scale = d[..., None] * ((2 * ls + 1) / 8)
    return (values * scale[..., None]).reshape(*shape[:-1], shape[-1] * 256)


def _kept(x):
    """The values in 32 bits of a tensor or of a checkpoint (codes, exponents)."""
    if isinstance(x, torch.Tensor):
        return x.float()
    codes, e = x
    unit = torch.pow(2.0, (e.double() - 133)).float().repeat_interleave(32, 1)[:, :codes.shape[1]]
    return codes.float() * unit


def _activation(name, g):
    """The activation and its derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    z = math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)
    t = 1 - 2 / (torch.exp(2 * z) + 1)
    dz = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * dz


def _plain_checkpoint(s):
    return _kept(_keep(s["x"])).to(s["dtype"])


def _plain_glu(s):
    x = s["x"].float()
    g, u = x @ _decode(s["fmt"], s["gate"], s["grid"]).T, x @ _decode(s["fmt"], s["up"], s["grid"]).T
    return (_activation(s["activation"], g)[0] * u).to(s["dtype"])


def _plain_glu_backward(s):
    x, dh = _kept(s["x"]), s["dh"].float()
    gate, up = _decode(s["fmt"], s["gate"], s["grid"]), _decode(s["fmt"], s["up"], s["grid"])
    g, u = x @ gate.T, x @ up.T
    a, da = _activation(s["activation"], g)
    return ((dh * u * da) @ gate + (dh * a) @ up).to(s["dtype"])


def _plain_linear_backward(s):
    dy = s["dy"].float()
    dx = dy @ _decode(s["fmt"], s["packed"], s["grid"])
    if "a" not in s:
        return {"dx": dx.to(s["dtype"])}
    x, a, b = _kept(s["x"]), s["a"].float(), s["b"].float()
    (N, r), T = a.shape[:2], len(x)
    # s_n of the token's adapter, zero for the others: [T, N, 1]
    mine = ((s["ids"][:, None] == torch.arange(N, device=x.device)).float() * s["scale"])[..., None]
    v = ((x @ a.reshape(N * r, -1).T).reshape(T, N, r) * mine).reshape(T, N * r)
    p = ((dy @ b.permute(1, 0, 2).reshape(-1, N * r)).reshape(T, N, r) * mine).reshape(T, N * r)
    dx = dx + p @ a.reshape(N * r, -1)
    da = (p.T @ x).reshape(N, r, -1)
    db = (dy.T @ v).reshape(-1, N, r).permute(1, 0, 2).contiguous()
    return {"dx": dx.to(s["dtype"]), "da": da.to(s["dtype"]), "db": db.to(s["dtype"])}


def run(s):
    if own:
        from ggml_iq_codebook_imatrix_amd import api
        if s["op"] == "checkpoint":
            codes, exponents = api.checkpoint(s["x"])
            return api.restore(codes, exponents, s["dtype"])
        if s["op"] == "glu":
            return api.glu(s["fmt"], s["gate"], s["up"], s["grid"], s["x"], activation=s["activation"])
        if s["op"] == "glu_backward":
            return api.glu_backward(s["fmt"], s["gate"], s["up"], s["grid"], s["x"], s["dh"],
                                    activation=s["activation"])
        if "a" not in s:
            return {"dx": api.linear_backward(s["fmt"], s["packed"], s["grid"], s["dy"])}
        dx, da, db = api.linear_backward(s["fmt"], s["packed"], s["grid"], s["dy"], x=s["x"], lora_a=s["a"],
                                         lora_b=s["b"], lora_scale=s["scale"], lora_ids=s["ids"])
        return {"dx": dx, "da": da, "db": db}
    return {"checkpoint": _plain_checkpoint, "glu": _plain_glu, "glu_backward": _plain_glu_backward,
            "linear_backward": _plain_linear_backward}[s["op"]](s)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _bits(packed, start, width):
    """Whole numbers read from a block as from one string of bits, least significant first."""
    total = 0
    for i in range(width):
        at = start + i
        total = total + (((packed[..., at // 8].long() >> (at % 8)) & 1) << i)
    return total


def _weights64(fmt, packed, grid):
    g = torch.arange(32, device=packed.device)
    sub, pair = g // 4, g // 2
    if fmt == "IQ2_XXS":
        word = 8 * (6 + 8 * sub)
        k, sign, ls = (_bits(packed, 8 * (2 + 8 * sub + g % 4), 8), _bits(packed, word + 7 * (g % 4), 7),
                       _bits(packed, word + 28, 4))
    elif fmt == "IQ2_XS":
        k, sign, ls = _bits(packed, 16 + 16 * g, 9), _bits(packed, 25 + 16 * g, 7), _bits(packed, 528 + 4 * pair, 4)
    elif fmt == "IQ2_S":
        k = _bits(packed, 16 + 8 * g, 8) + 256 * _bits(packed, 528 + 2 * g, 2)
        sign, ls = _bits(packed, 272 + 8 * g, 8), _bits(packed, 592 + 4 * pair, 4)
    elif fmt == "IQ1_S":
        k = _bits(packed, 16 + 8 * g, 8) + 256 * _bits(packed, 272 + 16 * sub + 3 * (g % 4), 3)
        ls, shift = _bits(packed, 272 + 16 * sub + 12, 3), _bits(packed, 272 + 16 * sub + 15, 1)
    else:
        k = _bits(packed, 8 * g, 8) + 256 * _bits(packed, 256 + 4 * g, 3)
        ls, shift = _bits(packed, 384 + 16 * (pair // 4) + 3 * (pair % 4), 3), _bits(packed, 259 + 4 * g, 1)
    if fmt == "IQ1_M":
        at = torch.arange(4, device=packed.device)
        code = (_bits(packed, 396 + 16 * at, 4) * 16 ** at).sum(-1)
    else:
        code = _bits(packed, torch.zeros(1, dtype=torch.long, device=packed.device), 16)[..., 0]
    # a half-precision number from its code: sign, exponent, fraction
    e, f = (code >> 10) & 31, (code & 1023).double()
    d = torch.where(e > 0, (1 + f / 1024) * torch.pow(2.0, (e - 15).double()), f * 2.0 ** -24)
    d = torch.where(code >= 32768, -d, d)
    entry = grid.double()[k]
    if fmt.startswith("IQ1"):
        w = (entry + torch.where(shift == 1, -0.125, 0.125).double()[..., None]) * (2 * ls + 1).double()[..., None]
    else:
        signs = [(sign >> i) & 1 for i in range(8 if fmt == "IQ2_S" else 7)]
        if fmt != "IQ2_S":
            signs.append(sum(signs) % 2)
        w = entry * (1 - 2 * torch.stack(signs, -1)).double() * ((2 * ls + 1).double() / 8)[..., None]
    return (w * d[..., None, None]).flatten(-3)


def _whole64(fmt, packed, grid):
    step = max(1, 2 ** 25 // (packed.shape[1] * 256))
    return torch.cat([_weights64(fmt, packed[i:i + step], grid) for i in range(0, len(packed), step)])


def _values64(x):
    if isinstance(x, torch.Tensor):
        return x.double()
    codes, e = x
    column = torch.arange(codes.shape[1], device=codes.device) // 32
    return torch.ldexp(codes.double(), (e.long() - 133)[:, column])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        x = s["x"].double()
        kept = torch.empty_like(x)
        for i in range(0, x.shape[1], 32):
            block = x[:, i:i + 32]
            most = block.abs().amax(1)
            # the smallest power of two in whose units the largest value rounds to 127 at most
            e = torch.frexp(most).exponent - 7
            e = torch.where(torch.round(torch.ldexp(most, -e)) > 127, e + 1, e)[:, None]
            kept[:, i:i + 32] = torch.ldexp(torch.round(torch.ldexp(block, -e)), e)
        return kept
    if case["op"] == "linear_backward":
        dy = s["dy"].double()
        dx = dy @ _whole64(s["fmt"], s["packed"], s["grid"])
        if not case["adapters"]:
            return {"dx": dx}
        x, a, b = _values64(s["x"]), s["a"].double(), s["b"].double()
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        for n in range(case["adapters"]):
            at, scale = (s["ids"] == n).nonzero()[:, 0], s["scale"][n].double()
            back = scale * (dy[at] @ b[n])
            dx[at] += back @ a[n]
            da[n] = back.T @ x[at]
            db[n] = scale * (dy[at].T @ (x[at] @ a[n].T))
        return {"dx": dx, "da": da, "db": db}
    x = _values64(s["x"])
    gate, up = _whole64(s["fmt"], s["gate"], s["grid"]), _whole64(s["fmt"], s["up"], s["grid"])
    g, u = x @ gate.T, x @ up.T
    if case["activation"] == "silu":
        sig = torch.sigmoid(g)
        act, slope = g * sig, sig + g * sig * (1 - sig)
    elif case["activation"] == "gelu":
        phi = torch.special.ndtr(g)
        act, slope = g * phi, phi + g * torch.exp(-g ** 2 / 2) / (2 * math.pi) ** 0.5
    else:
        k = (2 / math.pi) ** 0.5
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        act = g / 2 * (1 + t)
        slope = (1 + t) / 2 + g / 2 * (1 - t ** 2) * k * (1 + 0.134145 * g ** 2)
    if case["op"] == "glu":
        return act * u
    dh = s["dh"].double()
    return (dh * u * slope) @ gate + (dh * act) @ up
