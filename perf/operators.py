"""The microscaled 4-bit floating-point operators: cases, plain forms and exact values.

Operators
    roundtrip   ck_quant_fp4 then ck_dequant_fp4: activations to blocks of 4-bit values that share
                a scale, and back to the values that they stand for
    linear      ck_fp4_linear: activations quantised per block, times quantised weights, plus bias
    experts     ck_fp4_expert_linear: the same product with the rows sorted by expert, each
                expert's rows (any number, none among them) times that expert's weights

Formats.  Elements are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the
even k in the low nibble.
    "mx"  blocks of 32 with a power-of-two scale, 2^(floor(log2(amax)) - 2) (E8M0 byte)
    "nv"  blocks of 16 with an E4M3 scale, e4m3(amax / (6 t)), under a per-tensor fp32 scale t
Block scales are laid out in tiles of 128 rows x 4 blocks, 512 bytes each: the scale of row r,
block c of a tile is byte (r % 32) * 16 + (r // 32) * 4 + c, tiles in row-major order.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"mx": 32, "nv": 16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# the most that a drawn case may cost: that of the largest listed one
MOST_FLOPS = 2.0 * 4096 * 16384 * 6144
MOST_VALUES = 4096 * 16384


def listed():
    return [
        # a denoising step's activations, as every quantised layer of the model takes them
        dict(name="roundtrip mx bf16 8192x3840", op="roundtrip", fmt="mx", dtype="bf16", M=8192,
             K=3840, layout="rows", tensor_scale=False),
        # fp32 activations held column-major, with a calibrated tensor scale
        dict(name="roundtrip nv f32 4096x16384", op="roundtrip", fmt="nv", dtype="f32", M=4096,
             K=16384, layout="cols", tensor_scale=True),
        # a few rows: a call whose launches are most of its time
        dict(name="roundtrip nv bf16 32x3840", op="roundtrip", fmt="nv", dtype="bf16", M=32,
             K=3840, layout="rows", tensor_scale=True),
        # one token: a read of the weights
        dict(name="linear nv bf16 1x3840x3840", op="linear", fmt="nv", dtype="bf16", M=1, K=3840,
             N=3840, layout="rows", tensor_scale=True, bias=True),
        # a small batch through the same layer
        dict(name="linear mx bf16 32x3840x3840", op="linear", fmt="mx", dtype="bf16", M=32, K=3840,
             N=3840, layout="rows", tensor_scale=False, bias=True),
        # ragged sizes everywhere: no tile is full, K ends inside a tile
        dict(name="linear nv bf16 413x2064x1111", op="linear", fmt="nv", dtype="bf16", M=413,
             K=2064, N=1111, layout="pitch", tensor_scale=True, bias=True),
        # the benchmark's layer
        dict(name="linear nv bf16 8192x3840x3840", op="linear", fmt="nv", dtype="bf16", M=8192,
             K=3840, N=3840, layout="rows", tensor_scale=True, bias=True),
        # the feed-forward's second layer, in fp16, without bias
        dict(name="linear mx f16 8192x10240x3840", op="linear", fmt="mx", dtype="f16", M=8192,
             K=10240, N=3840, layout="rows", tensor_scale=False, bias=False),
        # the largest layer: fp32 in and out
        dict(name="linear nv f32 4096x16384x6144", op="linear", fmt="nv", dtype="f32", M=4096,
             K=16384, N=6144, layout="rows", tensor_scale=True, bias=True),
        # decoding: two experts for each of 32 tokens, most experts with a row or two
        dict(name="experts mx bf16 64 rows, 32", op="experts", fmt="mx", dtype="bf16", M=64,
             rows=64, K=3840, N=3840, E=32, tensor_scale=False, bias=False),
        # ragged: a buffer with room behind the last row, experts without rows, odd channels
        dict(name="experts nv f16 1500 rows, 8", op="experts", fmt="nv", dtype="f16", M=2000,
             rows=1500, K=1040, N=1111, E=8, tensor_scale=True, bias=True),
        # a long prompt: two experts for each of 8192 tokens
        dict(name="experts nv bf16 16384 rows, 16", op="experts", fmt="nv", dtype="bf16", M=16384,
             rows=16384, K=3840, N=3840, E=16, tensor_scale=True, bias=False),
    ]


def _log(rng, low, high):
    """A size between low and high, spread over its logarithm."""
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["roundtrip", "linear", "linear", "experts"])
    fmt = rng.choice(["mx", "nv"])
    b = BLOCK[fmt]
    case = dict(op=op, fmt=fmt, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                K=b * _log(rng, 64 // b, 16384 // b), M=_log(rng, 1, 16384))
    case["tensor_scale"] = fmt == "nv" and rng.random() < 0.7
    if op == "roundtrip":
        case["layout"] = rng.choice(["rows", "rows", "pitch", "cols"])
        case["M"] = max(1, min(case["M"], MOST_VALUES // case["K"]))
        return case
    case["N"] = _log(rng, 64, 6144)
    case["bias"] = rng.random() < 0.6
    if op == "linear":
        case["layout"] = rng.choice(["rows", "rows", "pitch"])
        case["M"] = max(1, min(case["M"], int(MOST_FLOPS / (2 * case["K"] * case["N"]))))
        return case
    # the experts' weights together are no larger than the listed prompt's
    case["E"] = max(1, min(_log(rng, 2, 64), 16 * 3840 * 3840 // (case["K"] * case["N"])))
    case["M"] = max(1, min(case["M"], MOST_VALUES // case["K"],
                           int(MOST_FLOPS / (2 * case["K"] * case["N"]))))
    case["rows"] = case["M"] if rng.random() < 0.5 else rng.randint(0, case["M"])
    return case


# ------------------------------------------------------------------------------ the plain form

def _grid(q, low, bits, top):
    """q (float64) rounded half to even to `bits` bits of precision, down to steps of the
    exponent `low`, and clamped to +-top."""
    e = (torch.frexp(q).exponent - 1).clamp(min=low)
    step = torch.ldexp(torch.ones_like(q), e - (bits - 1))
    return ((q / step).round() * step).clamp(-top, top)


def _quantise(x, fmt, tensor_scale):
    """(values on the E2M1 grid (M, K), block scales (M, K / block)), both fp32.  The quotients
    are taken in 64 bits: many lie next to the border between two values."""
    M, K = x.shape
    v = x.float().reshape(M, K // BLOCK[fmt], BLOCK[fmt])
    amax = v.abs().amax(-1)
    if fmt == "mx":
        e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
        e = torch.where(amax == 0, torch.full_like(e, -127), e)
        scale = torch.ldexp(torch.ones_like(amax, dtype=torch.float64), e)
        unit = scale
    else:
        t = tensor_scale if tensor_scale is not None else torch.ones((), device=x.device)
        scale = _grid(amax.double() / (6.0 * t).double(), -6, 4, 448.0)
        unit = (scale.float() * t).double()
    unit = unit[..., None]
    q = torch.where(unit == 0, torch.zeros_like(unit), v.double() / unit)
    bad = ~torch.isfinite(amax)
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    q = torch.where(bad[..., None], torch.zeros_like(q), q)
    return _grid(q, 0, 2, 6.0).reshape(M, K).float(), scale.float()


def _tile(s):
    """Block scales (R, C) as bytes -> the tiled layout, with zeros past R and C."""
    R, C = s.shape
    rb, cb = -(-R // 128), -(-C // 4)
    p = torch.zeros(rb * 128, cb * 4, dtype=torch.uint8, device=s.device)
    p[:R, :C] = s
    return p.view(rb, 4, 32, cb, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile(b, R, C):
    rb, cb = -(-R // 128), -(-C // 4)
    return b.view(rb, cb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, cb * 4)[:R, :C]


def _scale_bytes(s, fmt):
    if fmt == "nv":
        return s.to(torch.float8_e4m3fn).view(torch.uint8)
    return (torch.frexp(s).exponent + 126).to(torch.uint8)


def _scale_values(b, fmt):
    if fmt == "nv":
        return b.contiguous().view(torch.float8_e4m3fn).float()
    return torch.ldexp(torch.ones(b.shape, device=b.device), b.int() - 127)


def _pack(v):
    """Values on the E2M1 grid -> codes, two to a byte."""
    half = (v.abs() * 2).long()
    code = torch.tensor([0, 1, 2, 3, 4, 4, 5, 5, 6, 6, 6, 6, 7], device=v.device)[half]
    code = (code + 8 * torch.signbit(v)).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(c):
    grid = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=c.device)
    return torch.stack([grid[(c & 15).long()], grid[(c >> 4).long()]], -1).flatten(-2)


def _spread(values, scales, fmt):
    """Grid values times their block's scale, (..., K)."""
    return (values.unflatten(-1, (-1, BLOCK[fmt])) * scales[..., None]).flatten(-2)


def _weights(state, rows):
    """The stored weights' values without the tensor scale, (E, N, K) in fp32."""
    c, fmt = state["w_codes"], state["fmt"]
    E, N, half = c.shape
    C = 2 * half // BLOCK[fmt]
    b = torch.stack([_untile(t, N, C) for t in state["w_scales"]])
    return _spread(_unpack(c), _scale_values(b, fmt), fmt)


# ------------------------------------------------------------------------------ inputs

def _activations(gen, M, K, dtype, dev):
    """Normal values with one channel in a hundred twenty times as large, one row in a hundred zero."""
    x = torch.randn(M, K, generator=gen, device=dev)
    x *= torch.where(torch.rand(K, generator=gen, device=dev) < 0.01, 20.0, 1.0)
    if M > 1:
        x[torch.rand(M, generator=gen, device=dev) < 0.01] = 0.0
    return x.to(dtype)


def _placed(x, layout):
    if layout == "cols":
        return x.t().contiguous().t()
    if layout == "pitch":
        buf = torch.zeros(x.shape[0], 2 * x.shape[1], dtype=x.dtype, device=x.device)
        buf[:, : x.shape[1]] = x
        return buf[:, : x.shape[1]]
    return x


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    fmt, M, K, dtype = case["fmt"], case["M"], case["K"], DTYPES[case["dtype"]]
    x = _activations(gen, M, K, dtype, dev)
    state = dict(case, x=_placed(x, case.get("layout", "rows")), x_tensor_scale=None,
                 w_tensor_scale=None, bias_values=None)
    if case["tensor_scale"]:   # calibrated so that the largest block scale is the largest E4M3
        state["x_tensor_scale"] = x.abs().amax().float().clamp(min=1e-6).reshape(1) / (6.0 * 448.0)
    if case["op"] == "roundtrip":
        return state
    E, N = case.get("E", 1), case["N"]
    codes, scales = [], []
    t = torch.rand(E, generator=gen, device=dev) * 5e-5 + 5e-5 if case["tensor_scale"] else None
    for e in range(E):
        w = torch.randn(N, K, generator=gen, device=dev) * 0.03
        v, s = _quantise(w, fmt, t[e] if t is not None else None)
        codes.append(_pack(v))
        scales.append(_tile(_scale_bytes(s, fmt)))
    # rows of packed codes at a pitch of 16 bytes
    half = K // 2
    buf = torch.zeros(E, N, -(-half // 16) * 16, dtype=torch.uint8, device=dev)
    buf[:, :, :half] = torch.stack(codes)
    state["w_codes"] = buf[:, :, :half]
    state["w_scales"] = torch.stack(scales)
    state["w_tensor_scale"] = t
    if case["bias"]:
        state["bias_values"] = (torch.randn(E, N, generator=gen, device=dev) * 0.1).to(dtype)
    if case["op"] == "experts":
        # a router's choice: some experts far more in demand than others, some without a row
        p = torch.randn(E, generator=gen, device=dev).exp()
        pick = torch.multinomial(p, max(1, case["rows"]), replacement=True, generator=gen)
        count = torch.bincount(pick[: case["rows"]], minlength=E)
        state["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
        state["most"] = int(count.max())
        state["out"] = torch.zeros(M, N, dtype=dtype, device=dev)
    return state


# ------------------------------------------------------------------------------ one pass

def _scaled(y, x_scale, w_scale, bias, dtype):
    if x_scale is not None:
        y = y * (x_scale * w_scale)
    if bias is not None:
        y = y + bias.float()
    return y.to(dtype)


def run(state):
    op, fmt, x, ts = state["op"], state["fmt"], state["x"], state["x_tensor_scale"]
    if own:
        from rotated_w4a4_quantized_group_b200 import ck

        kind = ck.CK_MXFP4 if fmt == "mx" else ck.CK_NVFP4
        if op == "roundtrip":
            codes, scales = ck.ck_quant_fp4(x, kind, tensor_scale=ts)
            return ck.ck_dequant_fp4(codes, scales, kind, tensor_scale=ts, out_dtype=x.dtype)
        if op == "linear":
            bias = state["bias_values"]
            return ck.ck_fp4_linear(x, state["w_codes"][0], state["w_scales"][0], kind,
                                    None if bias is None else bias[0], x_tensor_scale=ts,
                                    w_tensor_scale=state["w_tensor_scale"])
        return ck.ck_fp4_expert_linear(x, state["offsets"], state["w_codes"], state["w_scales"],
                                       kind, state["bias_values"], x_tensor_scale=ts,
                                       w_tensor_scale=state["w_tensor_scale"], out=state["out"])

    values, scales = _quantise(x, fmt, ts)
    y = _spread(values, scales, fmt)
    if op == "roundtrip":
        return (y if ts is None else y * ts).to(x.dtype)
    w = _weights(state, state["N"])
    bias, wt = state["bias_values"], state["w_tensor_scale"]
    if op == "linear":
        return _scaled(y @ w[0].t(), ts, wt, None if bias is None else bias[0], x.dtype)
    # each expert's rows, padded to the most that one has; row i of expert e is offsets[e] + i
    first, count = state["offsets"][:-1].long(), state["offsets"].diff().long()
    i = torch.arange(state["most"], device=x.device)
    row = (first[:, None] + i).clamp(max=x.shape[0] - 1)
    z = torch.bmm(y[row], w.transpose(1, 2))
    z = _scaled(z, ts, None if wt is None else wt[:, None, None],
                None if bias is None else bias[:, None, :], x.dtype)
    there = i < count[:, None]
    out = state["out"]
    out[row[there]] = z[there]
    return out


def work(case):
    """Activations, weights with their scales, and bias in; outputs out.  The round trip also
    writes and reads the codes and scales, the products do not have to."""
    size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
    M, K, b = case["M"], case["K"], BLOCK[case["fmt"]]
    if case["op"] == "roundtrip":
        return {"bytes": 2 * M * K * size + 2 * M * (K // 2 + K // b), "flops": 3 * M * K}
    N, E = case["N"], case.get("E", 1)
    rows = case.get("rows", M)
    used = min(E, rows) if case["op"] == "experts" else 1
    weights = used * (N * (K // 2 + K // b) + (N * size if case["bias"] else 0))
    return {"bytes": rows * K * size + weights + rows * N * size, "flops": 2 * rows * K * N}


# ------------------------------------------------------------------------------ exact values

def exact(case, seed):
    """The definition in 64 bits: scales from the bits of amax or from the table of E4M3 values,
    elements by comparing the quotient with the borders between neighbours, products in fp64."""
    state = prepare(case, seed)
    fmt, b, dev = state["fmt"], BLOCK[state["fmt"]], state["x"].device
    x = state["x"].float()
    M, K = x.shape
    v = x.reshape(M, K // b, b)
    amax = v.abs().max(-1).values
    ts = state["x_tensor_scale"]
    if fmt == "mx":
        byte = ((amax.view(torch.int32) >> 23) - 2).clamp(0, 254)
        s = torch.pow(2.0, (byte - 127).double())
        unit = s
    else:
        t32 = ts if ts is not None else torch.ones(1, device=dev)
        code = torch.arange(127, device=dev)
        e, m = code // 8, (code % 8).double()
        table = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.pow(2.0, (e - 10).double()))
        mid = (table[1:] + table[:-1]) / 2
        q = amax.double() / (t32 * 6.0).double()
        # a quotient on a border goes to the even code: up from an odd one, not from an even one
        n = torch.bucketize(q, mid[0::2].contiguous()) + torch.bucketize(
            q, mid[1::2].contiguous(), right=True)
        s = table[n]
        unit = (s.float() * t32).double()
    a = v.double().abs() / torch.where(unit == 0, torch.ones_like(unit), unit)[..., None]
    a = torch.where((unit == 0)[..., None], torch.zeros_like(a), a)
    even = torch.tensor([0.25, 1.25, 2.5, 5.0], device=dev, dtype=torch.float64)
    odd = torch.tensor([0.75, 1.75, 3.5], device=dev, dtype=torch.float64)
    n = torch.bucketize(a, even) + torch.bucketize(a, odd, right=True)
    grid = torch.tensor(MAGNITUDES, device=dev, dtype=torch.float64)
    y = (torch.copysign(grid[n], v.double()) * s[..., None]).reshape(M, K)
    if ts is not None:
        y = y * ts.double()
    if case["op"] == "roundtrip":
        return y
    bias, wt = state["bias_values"], state["w_tensor_scale"]
    E, N = state["w_codes"].shape[:2]
    offsets = state["offsets"].tolist() if case["op"] == "experts" else [0, M]
    out = torch.zeros(M, N, device=dev, dtype=torch.float64)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        c = state["w_codes"][e]
        w = torch.empty(N, K, device=dev, dtype=torch.float64)
        for h in (0, 1):
            nib = ((c >> (4 * h)) & 15).long()
            w[:, h::2] = grid[nib & 7] * (1.0 - 2.0 * (nib >> 3).double())
        r = torch.arange(N, device=dev)[:, None]
        k = torch.arange(K // b, device=dev)[None, :]
        tiles = -(-(K // b) // 4)
        byte = state["w_scales"][e][((r // 128) * tiles + k // 4) * 512 + (r % 32) * 16
                                    + (r % 128) // 32 * 4 + k % 4].long()
        ws = table[byte] if fmt == "nv" else torch.pow(2.0, (byte - 127).double())
        w *= ws.repeat_interleave(b, 1)
        z = y[lo:hi] @ w.t()
        if wt is not None:
            z = z * wt[e].double()
        out[lo:hi] = z if bias is None else z + bias[e].double()
    return out
