"""The operators between a stack's residual stream and its mixers' projections, as cases to be timed and compared.

Every mixer or attention block of a stack starts with the sum of the residual stream and a norm, and its projections
read weights that are the larger part of a decoded token's bytes.  One rank runs there
  rms_norm        the block's output added to the residual stream and its root-mean-square norm, in the io
                  dtype or in 8 bits with a scale per token
  q4_quantize     a projection's weight in 4 bits (e2m1), with a power of two for each 32 of its values
  q4_dequantize   such a weight back in the io dtype
  q4_linear       products of tokens (bf16, fp32, or 8 bits with scales) with such a weight
Where `own` is false, run() computes a case in elementary torch operations in fp32; where it is true, it calls the
package."""
import math

import torch

own = False

F32 = torch.float32
E4M3 = torch.float8_e4m3fn
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
TOP = 448.0
TINY = 2.0 ** -100  # a row or group whose largest magnitude is below this is stored as zeros
EPS = 1e-5
GROUP = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token of a 7B-class stack: its block's output into the residual stream, and the norm
        dict(name="norm_token", op="norm", T=1, D=4096, io="bf16", res="bf16", out="io"),
        # a decode batch, residual stream in fp32, 8-bit tokens for the projection
        dict(name="norm_batch", op="norm", T=64, D=2560, io="bf16", res="f32", out="e4m3"),
        # a 32768-token prompt, 8-bit tokens
        dict(name="norm_prompt", op="norm", T=32768, D=4096, io="bf16", res="bf16", out="e4m3"),
        # the stack's last norm (nothing to add), fp32, odd width
        dict(name="norm_f32", op="norm", T=1000, D=1544, io="f32", res="none", out="io"),
        # one decoded token through the whole in_proj of a 7B-class mixer
        dict(name="linear_token", op="linear", T=1, M=16384, K=4096, x="bf16"),
        # a decode batch of 64 through its out_proj, 8-bit tokens
        dict(name="linear_batch", op="linear", T=64, M=4096, K=8192, x="e4m3"),
        # five tokens, fp32, odd sizes
        dict(name="linear_f32", op="linear", T=5, M=1000, K=1552, x="f32"),
        # a short prompt's in_proj, a 2.8B-class mixer's slice
        dict(name="linear_chunk", op="linear", T=300, M=5120, K=2560, x="bf16"),
        # a 4096-token prompt through the whole in_proj of a 7B-class mixer
        dict(name="linear_prompt", op="linear", T=4096, M=16384, K=4096, x="bf16"),
        # a decode batch's way into a block: norm in 8 bits, then a rank's in_proj
        dict(name="norm_linear", op="norm_linear", T=17, M=4096, K=4096, io="bf16", res="f32"),
        # the in_proj of a 7B-class mixer in 4 bits, and back
        dict(name="quantize_in_proj", op="quantize", M=16384, K=4096, io="bf16"),
        # the x_proj rows of a slice, fp32, odd sizes
        dict(name="quantize_x_proj", op="quantize", M=288, K=2064, io="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "linear", "norm_linear", "quantize"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "norm":
        D = 8 * _log(rng, 8, 1024)
        return dict(op=op, T=_log(rng, 1, min(32768, (1 << 25) // D)), D=D, io=io,
                    res=rng.choice(["none", io, io, "f32"]), out=rng.choice(["io", "e4m3"]))
    if op == "linear":
        M, K = _log(rng, 1, 16384), 16 * _log(rng, 1, 512)
        return dict(op=op, T=_log(rng, 1, min(8192, (1 << 37) // (M * K))), M=M, K=K,
                    x=rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"]))
    if op == "norm_linear":
        M, K = _log(rng, 16, 16384), 16 * _log(rng, 4, 512)
        return dict(op=op, T=_log(rng, 1, min(2048, (1 << 37) // (M * K))), M=M, K=K, io="bf16",
                    res=rng.choice(["bf16", "f32"]))
    M = _log(rng, 1, 16384)
    return dict(op=op, M=M, K=16 * _log(rng, 1, 512 if M <= 8192 else 256), io=io)


# ---------------------------------------------------------------- weights in 4 bits

def _pow2(e):
    """2^(e - 127) exactly, for exponents 1 .. 254 of any whole type (exp2 and pow need not give it on a GPU)."""
    return (e.int() << 23).view(F32)


def _packed(c, s):
    """Codes [M, K] and group exponents [M, ceil(K / 32)] (uint8) as the package holds them: tiles of 16 rows by 128
    columns, in a tile 16 bytes for each column group of 32 and row; exponents of four tiles side by side."""
    (M, K), dev = c.shape, c.device
    mt, kt, k4 = -(-M // 16), -(-K // 128), -(-K // 512)
    full = torch.zeros(mt * 16, kt * 128, dtype=torch.uint8, device=dev)
    full[:M, :K] = c
    full = full[:, 0::2] | full[:, 1::2] << 4
    codes = full.view(mt, 16, kt, 4, 16).permute(0, 2, 3, 1, 4).reshape(mt, kt, 64, 16).contiguous()
    exps = torch.full((mt * 16, k4 * 16), 127, dtype=torch.uint8, device=dev)
    exps[:M, :s.shape[1]] = s
    exps = exps.view(mt, 16, k4, 4, 4).permute(0, 2, 4, 1, 3).reshape(mt, k4, 64, 4).contiguous()
    return codes, exps


def _values(codes, exps, M, K):
    """The fp32 weight [M, K] that they stand for."""
    mt, kt = codes.shape[:2]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    v = v.view(mt, kt, 4, 16, 32).permute(0, 3, 1, 2, 4)
    e = exps.view(mt, -1, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(mt, 16, -1, 4)[:, :, :kt]
    return (v * _pow2(e).unsqueeze(-1)).reshape(mt * 16, kt * 128)[:M, :K]


def _to_codes(w):
    """Codes and group exponents of a weight: the exponent that brings a group's largest magnitude, rounded to e2m1's
    three significant bits, to 4 .. 6; codes rounded to nearest, ties to the even code."""
    M, K = w.shape
    x = torch.nn.functional.pad(w.float(), (0, -K % GROUP)).view(M, -1, GROUP)
    amax = x.abs().amax(-1)
    e = (((amax.view(torch.int32) + 0x200000) >> 23) - 2).clamp(max=252)
    e = torch.where(amax >= TINY, e, torch.full_like(e, 127))
    mag = x.abs() * _pow2(254 - e).unsqueeze(-1)
    mag = torch.where((amax >= TINY).unsqueeze(-1), mag, torch.zeros_like(mag))
    c = torch.zeros(x.shape, dtype=torch.uint8, device=w.device)
    c += mag > 0.25
    c += mag >= 0.75
    c += mag > 1.25
    c += mag >= 1.75
    c += mag > 2.5
    c += mag >= 3.5
    c += mag > 5.0
    c += 8 * (torch.signbit(x) & (amax >= TINY).unsqueeze(-1)).to(torch.uint8)
    return c.view(M, -1)[:, :K], e.to(torch.uint8)


# ---------------------------------------------------------------- what a program has before the call

def _weight(M, K, g, dev, io=F32):
    w = torch.randn(M, K, generator=g, device=dev) * (torch.rand(M, 1, generator=g, device=dev) + 0.2) / math.sqrt(K)
    return w.to(io)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("norm", "norm_linear"):
        T, D, io = case["T"], case["D"] if op == "norm" else case["K"], IO[case["io"]]
        s["x"] = torch.randn(T, D, generator=g, device=dev).to(io)
        s["w"] = 1 + 0.2 * torch.randn(D, generator=g, device=dev)
        s["res"] = s["sum"] = None
        if case["res"] != "none":  # a residual stream grows over a stack, some channels more than others
            res = torch.randn(T, D, generator=g, device=dev) * (1 + 8 * torch.rand(D, generator=g, device=dev) ** 4)
            s["res"] = res.to(IO[case["res"]])
            s["sum"] = torch.empty_like(s["res"])
    if op in ("linear", "norm_linear"):
        s["codes"], s["exps"] = _packed(*_to_codes(_weight(case["M"], case["K"], g, dev)))
    if op == "linear":
        x = torch.randn(case["T"], case["K"], generator=g, device=dev)
        s["x_scale"] = None
        if case["x"] == "e4m3":
            s["x"], s["x_scale"] = _row_codes(x)
        else:
            s["x"] = x.to(IO[case["x"]])
    if op == "quantize":
        s["x"] = _weight(case["M"], case["K"], g, dev, IO[case["io"]])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    if op == "norm":
        y, total = _norm(s, case)
        if case["out"] == "io":
            return [y.to(IO[case["io"]]), total]
        return [*_row_codes(y), total]
    if op == "linear":
        x = s["x"].float()
        y = torch.matmul(x, _values(s["codes"], s["exps"], case["M"], case["K"]).t())
        if s["x_scale"] is not None:
            y *= s["x_scale"].unsqueeze(1)
        return y.to(F32 if case["x"] == "f32" else torch.bfloat16)
    if op == "norm_linear":
        y, total = _norm(s, case)
        codes, scale = _row_codes(y)
        y = torch.matmul(codes.float(), _values(s["codes"], s["exps"], case["M"], case["K"]).t())
        return [(y * scale.unsqueeze(1)).to(torch.bfloat16), total]
    c, e = _to_codes(s["x"])
    codes, exps = _packed(c, e)
    return [_values(codes, exps, case["M"], case["K"]).to(s["x"].dtype), exps]


def _own(s, case, op):
    import selective_state_space_causal_amd as ssm
    if op == "norm":
        y = ssm.rms_norm(s["x"], s["w"], residual=s["res"], residual_out=s["sum"], eps=EPS,
                         out_dtype=None if case["out"] == "io" else E4M3)
        return [y, s["sum"]] if case["out"] == "io" else [*y, s["sum"]]
    if op == "linear":
        return ssm.q4_linear(s["x"], ssm.Q4Weight(s["codes"], s["exps"], case["M"], case["K"]), x_scale=s["x_scale"])
    if op == "norm_linear":
        x, scale = ssm.rms_norm(s["x"], s["w"], residual=s["res"], residual_out=s["sum"], eps=EPS, out_dtype=E4M3)
        return [ssm.q4_linear(x, ssm.Q4Weight(s["codes"], s["exps"], case["M"], case["K"]), x_scale=scale), s["sum"]]
    w = ssm.q4_quantize(s["x"])
    return [ssm.q4_dequantize(w, dtype=s["x"].dtype), w.scales]


# ---------------------------------------------------------------- plain forms

def _norm(s, case):
    """(the norm in fp32, the new residual stream or None)."""
    x, total = s["x"].float(), None
    if s["res"] is not None:
        total = (x + s["res"].float()).to(s["res"].dtype)
        x = total.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"], total


def _row_codes(y):
    """Rows in e4m3 and their scales."""
    amax = y.abs().amax(-1)
    live = amax >= TINY
    scale = torch.where(live, amax * (1 / TOP), torch.zeros_like(amax))
    mult = torch.where(live, (1 / amax) * TOP, torch.zeros_like(amax))
    return (y * mult.unsqueeze(-1)).clamp(-TOP, TOP).to(E4M3), scale


# ---------------------------------------------------------------- work

def _size(t):
    return {"bf16": 2, "f32": 4, "e4m3": 1, "none": 0}[t]


def work(case):
    """Each input read once, each output written once, and the products of the formulas."""
    op = case["op"]
    q4 = 0 if op == "norm" else case["M"] * (case["K"] / 2 + -(-case["K"] // GROUP))
    if op in ("norm", "norm_linear"):
        n = case["T"] * (case["D"] if op == "norm" else case["K"])
        b = n * (_size(case["io"]) + 2 * _size(case["res"])) + 4 * n / case["T"]
        if op == "norm":
            b += n * _size(case["io"]) if case["out"] == "io" else n + 4 * case["T"]
            return {"bytes": b, "flops": 4 * n}
        return {"bytes": b + q4 + 2 * case["T"] * case["M"], "flops": 4 * n + 2 * n * case["M"]}
    if op == "linear":
        T, M, K = case["T"], case["M"], case["K"]
        out = 4 if case["x"] == "f32" else 2
        return {"bytes": q4 + T * K * _size(case["x"]) + T * M * out + (4 * T if case["x"] == "e4m3" else 0), "flops": 2 * T * M * K}
    n = case["M"] * case["K"]
    return {"bytes": 2 * n * _size(case["io"]) + 2 * q4, "flops": 4 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s, f = prepare(case, seed), torch.float64
    op = case["op"]

    def two_to(n):
        """2^n as a double with that exponent and no mantissa."""
        return ((n.long() + 1023) << 52).view(f)

    def weight():
        """w[m, k] = sign * magnitude * 2^(exponent - 127), code by code from its place in the tiles."""
        M, K, dev = case["M"], case["K"], s["codes"].device
        m, k = torch.arange(M, device=dev)[:, None], torch.arange(K, device=dev)[None, :]
        lane = (k % 128) // 32 * 16 + m % 16
        byte = s["codes"][m // 16, k // 128, lane, (k % 32) // 2].int()
        code = torch.where(k % 2 == 0, byte % 16, byte // 16)
        e, man = code % 8 // 2, code % 2  # two bits of exponent (bias 1), one of mantissa
        mag = torch.where(e == 0, man.to(f) / 2, (1 + man.to(f) / 2) * two_to(e - 1))
        scale = s["exps"][m // 16, k // 512, lane, k // 128 % 4].int()
        return torch.where(code >= 8, -mag, mag) * two_to(scale - 127)

    def normed():
        x, total = s["x"].to(f), None
        if s["res"] is not None:
            total = x + s["res"].to(f)
            x = total.to(s["res"].dtype).to(f)  # the stream is stored in its own type, and the norm is of what is stored
        return s["w"].to(f) * x / (x.square().mean(-1, keepdim=True) + EPS).sqrt(), total

    def coded(y):
        big = y.abs().max(-1, keepdim=True).values
        return (y * (TOP / big)).to(E4M3).to(f), big / TOP

    if op == "norm":
        y, total = normed()
        if case["out"] == "io":
            return [y, total]
        c, scale = coded(y)
        return [c, scale[:, 0], total]
    if op == "linear":
        y = s["x"].to(f) @ weight().t()
        return y if s["x_scale"] is None else y * s["x_scale"].to(f)[:, None]
    if op == "norm_linear":
        y, total = normed()
        c, scale = coded(y)
        return [(c * scale) @ weight().t(), total]
    x = s["x"].to(f)
    M, K = x.shape
    groups = torch.cat((x, x.new_zeros(M, -K % GROUP)), 1).unflatten(1, (-1, GROUP))
    big = groups.abs().max(-1, keepdim=True).values
    n = torch.frexp(big).exponent - 1
    n = n + (big >= 1.75 * two_to(n))
    grid = torch.tensor(E2M1, dtype=f, device=x.device)
    z = groups.abs() / two_to(n - 2)
    low = (torch.searchsorted(grid, z, right=True) - 1).clamp(max=6)
    below, above = z - grid[low], grid[low + 1] - z
    up = (above < below) | ((above == below) & (low % 2 == 1))
    v = torch.where(up, grid[low + 1], grid[low]) * two_to(n - 2) * groups.sign()
    return [v.flatten(1)[:, :K], None]
