"""Cases of the quantised-weight operators: microscaled 4-bit floating point
(quantise, dequantise, product) and the product with the packed b-bit codes
that the layer solve returns.

Formats.  An MX matrix [rows][K] holds e2m1 codes, two to a byte (element 2i in
the low nibble), and one 8-bit scale per block of a row: "mxfp4" 32 elements and
a power of two (e8m0, value 2^(byte - 127)), "nvfp4" 16 elements and an e4m3
scale on top of one fp32 scale of the whole tensor.  Scales lie in tiles of 128
rows x 4 blocks of 512 bytes, [ceil(rows / 128)][ceil(K / (4 block))][32][4][4]:
row r, block c of a tile at byte 16 (r % 32) + 4 (r // 32) + c; bytes without a
block are zero.  Packed codes are b-bit little-endian rows of 32-bit words
(code k of a row at bits [b k, b k + b)), with fp32 scale and zero point per
group of a row: weight = scale (code - zero).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = {"mxfp4": 32, "nvfp4": 16}


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # one decoded token's activations on their way into a 4-bit layer: latency
        dict(name="quantize token mxfp4", op="quantize", rows=1, k=4096, fmt="mxfp4", dtype="bf16"),
        # the stacked gate/up weights of a decoder layer, quantised once
        dict(name="quantize weights mxfp4", op="quantize", rows=24576, k=4096, fmt="mxfp4",
             dtype="bf16"),
        # a ragged prompt's activations in front of the down projection
        dict(name="quantize activations nvfp4", op="quantize", rows=2047, k=12288, fmt="nvfp4",
             dtype="bf16"),
        # a large layer's stored weights, back to 16 bits (for a layer that is to run unquantised)
        dict(name="dequantize weights nvfp4", op="dequantize", rows=25600, k=5120, fmt="nvfp4",
             dtype="bf16"),
        # a small odd matrix in fp32, for comparing a layer with its weights
        dict(name="dequantize odd mxfp4", op="dequantize", rows=777, k=416, fmt="mxfp4",
             dtype="fp32"),
        # decoding: one token through the output projection
        dict(name="mx token", op="mx", tokens=1, k=4096, n=4096, fmt="mxfp4", dtype="bf16",
             quantised=False),
        # decoding in a batch: the down projection of 48 sequences
        dict(name="mx batch", op="mx", tokens=48, k=12288, n=4096, fmt="nvfp4", dtype="bf16",
             quantised=False),
        # prefill: two prompts of 2048 tokens through gate/up
        dict(name="mx prefill", op="mx", tokens=4096, k=4096, n=24576, fmt="mxfp4", dtype="bf16",
             quantised=False),
        # a ragged chunk whose activations are quantised already (they feed several products)
        dict(name="mx ragged", op="mx", tokens=1000, k=5120, n=25600, fmt="nvfp4", dtype="fp16",
             quantised=True),
        # decoding: one token through q/k/v solved at 3 bits
        dict(name="packed token", op="packed", tokens=1, k=4096, n=6144, bits=3, group=128,
             dtype="bf16"),
        # decoding in a batch: 33 sequences through the down projection solved at 2 bits
        dict(name="packed batch", op="packed", tokens=33, k=12288, n=4096, bits=2, group=128,
             dtype="bf16"),
        # prefill: two prompts of 2048 tokens through gate/up solved at 4 bits
        dict(name="packed prefill", op="packed", tokens=4096, k=4096, n=24576, bits=4, group=128,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "mx", "mx", "packed", "packed"])
    if op in ("quantize", "dequantize"):
        k = 32 * _log(rng, 1, 384)
        rows = _log(rng, 1, min(25600, 100_000_000 // k))
        return dict(op=op, rows=rows, k=k, fmt=rng.choice(["mxfp4", "nvfp4"]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    tokens, n = _log(rng, 1, 4096), _log(rng, 16, 25600)
    if op == "mx":
        k = 32 * _log(rng, 2, min(384, 410_000_000_000 // (32 * tokens * n)))
        return dict(op=op, tokens=tokens, k=k, n=n, fmt=rng.choice(["mxfp4", "nvfp4"]),
                    dtype=rng.choice(["bf16", "fp16"]), quantised=rng.random() < 0.5)
    group = rng.choice([32, 64, 128, 128])
    k = group * _log(rng, 1, min(12288 // group, 410_000_000_000 // (group * tokens * n)))
    return dict(op=op, tokens=tokens, k=k, n=n, bits=rng.choice([1, 2, 3, 3, 4, 4, 5, 6, 7, 8]),
                group=group, dtype=rng.choice(["bf16", "fp16"]))


# ------------------------------------------------------------------ the inputs


def _activations(rows, k, dtype, gen):
    """Heavy-tailed activations with outlier channels and a few padding rows."""
    x = torch.randn((rows, k), generator=gen, device="cuda")
    chi2 = torch.zeros_like(x)
    for _ in range(4):
        chi2 += torch.randn((rows, k), generator=gen, device="cuda").square_()
    x *= (chi2 / 4).rsqrt_()
    x[:, torch.randperm(k, generator=gen, device="cuda")[: max(1, k // 100)]] *= 30
    x[rows - rows // 16:] = 0          # padding behind the last sequence
    return x.clamp_(-3e4, 3e4).to(dtype)


def _weights(n, k, dtype, gen):
    return (torch.randn((n, k), generator=gen, device="cuda") * 0.02).to(dtype)


def _scale_tiles(s):
    """u8 [rows][blocks] -> the tiles of 128 rows x 4 blocks."""
    rows, blocks = s.shape
    full = s.new_zeros((-(-rows // 128) * 128, -(-blocks // 4) * 4))
    full[:rows, :blocks] = s
    t = full.view(full.shape[0] // 128, 4, 32, full.shape[1] // 4, 4)
    return t.permute(0, 3, 2, 1, 4).contiguous()


def _mx_operand(x, fmt):
    """What a program keeps of a quantised matrix: codes, scale tiles, tensor scale."""
    g = _tensor_scale(x) if fmt == "nvfp4" else None
    index, scale = _plain_quantize(x, fmt, g)
    codes = (index[:, 0::2] + 16 * index[:, 1::2]).to(torch.uint8)
    if fmt == "mxfp4":
        byte = torch.frexp(scale)[1] + 126
    else:
        e = (torch.frexp(scale)[1] - 1).clamp(min=-6)
        frac = torch.ldexp(scale, -e)                   # in [1, 2), below 1 when subnormal
        byte = ((e + 6) * 8 + (frac * 8).round()).to(torch.int32)
    return codes, _scale_tiles(byte.to(torch.uint8)), g


def _tensor_scale(x):
    """nvfp4: the largest value lands on the largest code under the largest scale."""
    return (x.float().abs().amax().clamp(min=1e-30) / (448 * 6)).reshape(1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "quantize":
        x = (_weights if case["rows"] > 4096 else _activations)(case["rows"], case["k"], dt, gen)
        s.update(x=x, g=_tensor_scale(x) if case["fmt"] == "nvfp4" else None)
    elif case["op"] == "dequantize":
        x = _weights(case["rows"], case["k"], torch.bfloat16, gen)
        s.update(zip(("codes", "scale", "g"), _mx_operand(x, case["fmt"])))
    elif case["op"] == "mx":
        w = _weights(case["n"], case["k"], torch.bfloat16, gen)
        s.update(zip(("codes", "scale", "g"), _mx_operand(w, case["fmt"])))
        x = _activations(case["tokens"], case["k"], dt, gen)
        if case["quantised"]:
            s.update(zip(("x_codes", "x_scale", "x_g"), _mx_operand(x, case["fmt"])))
        else:
            s.update(x=x, x_g=_tensor_scale(x) if case["fmt"] == "nvfp4" else None)
    else:
        n, k, bits, group = case["n"], case["k"], case["bits"], case["group"]
        w = _weights(n, k, torch.float32, gen).view(n, k // group, group)
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        top = 2 ** bits - 1
        scale = (hi - lo) / top
        zero = (-lo / scale).round()
        codes = ((w / scale[:, :, None]).round() + zero[:, :, None]).clamp(0, top)
        codes = codes.view(n, k // 32, 32).to(torch.int64)
        words = codes.new_zeros((n, k // 32, bits + 1))
        for i in range(32):
            at, shift = bits * i // 32, bits * i % 32
            words[:, :, at] |= (codes[:, :, i] << shift) & 0xFFFFFFFF
            words[:, :, at + 1] |= codes[:, :, i] >> (32 - shift)
        words = words[:, :, :bits].reshape(n, k // 32 * bits)
        packed = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
        s.update(x=_activations(case["tokens"], k, dt, gen), packed=packed, scale=scale, zero=zero)
    return s


# ------------------------------------------------------------- the plain forms


def _e2m1_index(a):
    """Nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 to a >= 0, ties to the even code."""
    return ((a > 0.25).to(torch.int32) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5))


def _e2m1_value(code):
    half = code & 1
    e = (code & 7) >> 1
    v = torch.where(e == 0, half * 0.5, (1 + half * 0.5) * torch.exp2((e - 1).float()))
    return torch.where(code >= 8, -v, v)


def _plain_quantize(x, fmt, g):
    """Code of each element (sign in bit 3) and scale of each block."""
    rows, k = x.shape
    xb = x.float().view(rows, -1, BLOCK[fmt])
    amax = xb.abs().amax(2)
    if fmt == "mxfp4":                  # 2^(floor(log2 amax) - 2): every step is exact in 32 bits
        e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
        scale = torch.ldexp(torch.ones_like(amax, dtype=torch.float64), e)
        a = xb.abs().double() / scale[:, :, None]
    else:                               # decisions next to a border: 64 bits
        q = amax.double() / (6 * g.double())
        step = torch.exp2((torch.frexp(q)[1] - 1).clamp(min=-6).double() - 3)
        scale = ((q / step).round() * step).clamp(max=448)
        t = (scale * g.double()).float().double()       # a block's step is an fp32 number
        a = xb.abs().double() / torch.where(t > 0, t, 1)[:, :, None] * (t > 0)[:, :, None]
    index = _e2m1_index(a) + 8 * (xb < 0)
    return index.view(rows, k), scale


def _plain_step(scale, fmt, g):
    return (scale if fmt == "mxfp4" else scale * g.double()).float()


def _plain_values(index, scale, fmt, g):
    """e2m1 value times its block's step, fp32."""
    rows, k = index.shape
    v = _e2m1_value(index).view(rows, -1, BLOCK[fmt]) * _plain_step(scale, fmt, g)[:, :, None]
    return v.view(rows, k)


def _plain_unpack(codes, tiles, fmt):
    """Stored codes and scale tiles -> code and scale as _plain_quantize gives them."""
    rows, k = codes.shape[0], codes.shape[1] * 2
    index = torch.stack([codes & 15, codes >> 4], 2).view(rows, k).to(torch.int32)
    s = tiles.permute(0, 3, 2, 1, 4).reshape(tiles.shape[0] * 128, -1)
    s = s[:rows, : k // BLOCK[fmt]].to(torch.int32)
    if fmt == "mxfp4":
        return index, torch.exp2((s - 127).double())
    e, m = s >> 3, s & 7
    normal = (8 + m).double() * torch.exp2((e - 10).double())
    return index, torch.where(e == 0, m.double() * 2.0 ** -9, normal)


def _plain(s):
    fmt, dt = s.get("fmt"), DTYPES[s["dtype"]]
    if s["op"] == "quantize":
        return _plain_values(*_plain_quantize(s["x"], fmt, s["g"]), fmt, s["g"]).to(dt)
    if s["op"] == "dequantize":
        return _plain_values(*_plain_unpack(s["codes"], s["scale"], fmt), fmt, s["g"]).to(dt)
    if s["op"] == "mx":
        w = _plain_values(*_plain_unpack(s["codes"], s["scale"], fmt), fmt, s["g"])
        if s["quantised"]:
            x = _plain_unpack(s["x_codes"], s["x_scale"], fmt)
        else:
            x = _plain_quantize(s["x"], fmt, s["x_g"])
        return (_plain_values(*x, fmt, s["x_g"]) @ w.T).to(dt)
    bits, n, k = s["bits"], s["n"], s["k"]
    at = bits * torch.arange(32, device="cuda")
    words = s["packed"].view(n, k // 32, bits).to(torch.int64) & 0xFFFFFFFF
    both = words | (torch.roll(words, -1, 2) << 32)
    codes = (both[:, :, at // 32] >> (at % 32)) & (2 ** bits - 1)
    w = (codes.view(n, -1, s["group"]) - s["zero"][:, :, None]) * s["scale"][:, :, None]
    return (s["x"].float() @ w.view(n, k).T).to(dt)


def _own(s):
    from post_weight_quantization_10_b200 import admmq
    dt = DTYPES[s["dtype"]]
    if s["op"] == "quantize":
        q = admmq.mx_quantize(s["x"], s["fmt"], tensor_scale=s["g"])
        return admmq.mx_dequantize(q, dt)
    if s["op"] == "packed":
        return admmq.packed_matmul(s["x"], s["packed"], s["scale"], s["zero"], s["bits"], dt)
    q = admmq.MxTensor(s["codes"], s["scale"], s["fmt"], s["g"])
    if s["op"] == "dequantize":
        return admmq.mx_dequantize(q, dt)
    if s["quantised"]:
        x = admmq.MxTensor(s["x_codes"], s["x_scale"], s["fmt"], s["x_g"])
        return admmq.mx_matmul(x, q, dt)
    return admmq.mx_linear(s["x"], q, dt, tensor_scale=s["x_g"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------ work


def _bytes_of(dtype):
    return 4 if dtype == "fp32" else 2


def work(case):
    size = _bytes_of(case["dtype"])
    if case["op"] in ("quantize", "dequantize"):
        e = case["rows"] * case["k"]
        mx = e // 2 + e // BLOCK[case["fmt"]]
        return {"bytes": e * size + (e * size if case["op"] == "quantize" else mx), "flops": 2 * e}
    m, n, k = case["tokens"], case["n"], case["k"]
    out, flops = m * n * size, 2 * m * n * k
    if case["op"] == "mx":
        per = 0.5 + 1 / BLOCK[case["fmt"]]
        return {"bytes": n * k * per + m * k * (per if case["quantised"] else size) + out,
                "flops": flops}
    return {"bytes": n * k * case["bits"] / 8 + n * k // case["group"] * 8 + m * k * size + out,
            "flops": flops}


# ----------------------------------------------------------------------- exact


def _exact_round(x, fmt, g):
    """The quantised values of a matrix in 64 bits, from the definition: the nearest
    level of each block's grid, ties to the level with the even code."""
    rows, k = x.shape
    x = x.double().view(rows, -1, BLOCK[fmt])
    top = x.abs().amax(2, keepdim=True)
    if fmt == "mxfp4":
        _, e = torch.frexp(top)
        t = torch.where(top > 0, torch.exp2((e - 3).clamp(min=-127).double()), 2.0 ** -127)
    else:
        codes = torch.arange(127, device=x.device)
        table = torch.where(codes < 8, codes * 2.0 ** -9,
                            (1 + codes % 8 / 8) * torch.exp2((codes // 8 - 7).double()))
        t = (_nearest(top / (6 * g.double()), table) * g.double()).float().double()
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    u = x.abs() / torch.where(t > 0, t, 1)
    v = torch.where(t > 0, _nearest(u, levels), 0) * t
    return (v * x.sign()).view(rows, k)


def _nearest(u, levels):
    """The nearest of sorted levels (index parity breaks ties), the last one above them."""
    hi = torch.searchsorted(levels, u.contiguous()).clamp(1, len(levels) - 1)
    below, above = u - levels[hi - 1], levels[hi] - u
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return levels[torch.where(up, hi, hi - 1)]


def _exact_stored(codes, tiles, fmt, g):
    rows, k = codes.shape[0], 2 * codes.shape[1]
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    levels = torch.cat([levels, -levels])
    v = torch.empty((rows, k), dtype=torch.float64, device=codes.device)
    v[:, 0::2], v[:, 1::2] = levels[(codes % 16).long()], levels[(codes // 16).long()]
    r = torch.arange(rows, device=codes.device)[:, None]
    c = torch.arange(k // BLOCK[fmt], device=codes.device)[None, :]
    s = tiles[r // 128, c // 4, r % 32, r % 128 // 32, c % 4].double()
    if fmt == "mxfp4":
        t = torch.exp2(s - 127)
    else:
        e, m = torch.div(s, 8, rounding_mode="floor"), s % 8
        t = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e - 7))
        t = (t * g.double()).float().double()
    return (v.view(rows, -1, BLOCK[fmt]) * t[:, :, None]).view(rows, k)


def exact(case, seed):
    s = prepare(case, seed)
    fmt = case.get("fmt")
    if case["op"] == "quantize":
        return _exact_round(s["x"], fmt, s["g"])
    if case["op"] == "dequantize":
        return _exact_stored(s["codes"], s["scale"], fmt, s["g"])
    if case["op"] == "mx":
        x = (_exact_stored(s["x_codes"], s["x_scale"], fmt, s["x_g"]) if case["quantised"]
             else _exact_round(s["x"], fmt, s["x_g"]))
        return x @ _exact_stored(s["codes"], s["scale"], fmt, s["g"]).T
    n, k, bits, group = case["n"], case["k"], case["bits"], case["group"]
    bit = torch.arange(32, device="cuda")
    w = torch.zeros((n, k), dtype=torch.float64, device="cuda")
    for j in range(bits):               # bit j of every code, from the row's bit stream
        pos = bits * torch.arange(k, device="cuda") + j
        w += ((s["packed"][:, pos // 32] >> bit[pos % 32]) & 1).double() * 2 ** j
    scale = s["scale"].double().repeat_interleave(group, 1)
    w = scale * (w - s["zero"].double().repeat_interleave(group, 1))
    return s["x"].double() @ w.T
