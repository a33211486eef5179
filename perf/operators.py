"""The attention operators beside the selective-SSM mixer, as cases to be timed and compared.

A hybrid stack puts attention blocks between selective-SSM mixers.  One rank's attention block runs
  rope               rotary positions of q and k
  kv_write           a prompt's or a token's keys and values into the paged cache, quantised
  kv_read            cached keys and values back in the io dtype
  attn_prefill       attention over packed prompts
  attn_decode_step   one token per sequence against the paged cache
Where `own` is false, run() computes a case in elementary torch operations in fp32; where it is true,
it calls the package."""
import math

import torch

own = False

F32 = torch.float32
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}
TINY = 2.0 ** -100  # a cache row whose largest magnitude is below this is stored as zeros


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one rank's 8 + 2 heads of a 32768-token prompt, long-context (YaRN) scaled, interleaved pairs in
        # the first half of each head
        dict(name="rope_prompt", op="rope", T=32768, Hq=8, Hkv=2, D=128, rot=64, layout="interleaved", scaling="yarn",
             factor=8.0, io="bf16", far=0),
        # a whole head count's 1000 tokens at far positions, fp32, odd head size
        dict(name="rope_far_f32", op="rope", T=1000, Hq=12, Hkv=12, D=80, rot=80, layout="half", scaling="linear",
             factor=4.0, io="f32", far=1000000),
        # a decode batch's 64 new tokens: q and k rotated, k and v into the 8-bit cache
        dict(name="write_tokens", op="kv_write", T=64, Hkv=8, D=128, page=64, codes="e4m3", Hq=32, rot=128,
             io="bf16"),
        # a 32768-token prompt's keys and values into an int8 cache
        dict(name="write_prompt", op="kv_write", T=32768, Hkv=8, D=128, page=64, codes="int8", Hq=0, rot=0, io="bf16"),
        # a short prefix read back in fp32, odd head size
        dict(name="read_prefix_f32", op="kv_read", T=777, Hkv=4, D=72, page=16, codes="e4m3", io="f32"),
        # a 65536-token context read back to be attended to by a prompt's next chunk
        dict(name="read_context", op="kv_read", T=65536, Hkv=8, D=128, page=64, codes="int8", io="bf16"),
        # a ragged batch of prompts, packed (lengths from 1 to 2048)
        dict(name="prefill_ragged", op="attn_prefill", B=17, L=2048, ragged=True, past=0, Hq=32, Hkv=8, D=128,
             causal=True, io="bf16"),
        # one rank's heads of a 32768-token prompt
        dict(name="prefill_long", op="attn_prefill", B=1, L=32768, ragged=False, past=0, Hq=8, Hkv=2, D=128,
             causal=True, io="bf16"),
        # fp32, odd head size, next chunk of prompts that already have up to 300 keys
        dict(name="prefill_chunk_f32", op="attn_prefill", B=3, L=500, ragged=True, past=300, Hq=6, Hkv=2, D=80,
             causal=True, io="f32"),
        # a decode batch of 64 sequences of up to 8192 tokens, int8 cache
        dict(name="decode_batch", op="attn_decode", B=64, L=8192, Hq=32, Hkv=8, D=128, page=64, codes="int8",
             io="bf16"),
        # one sequence of 65536 tokens, one rank's heads, 8-bit floating point cache
        dict(name="decode_long", op="attn_decode", B=1, L=65536, Hq=8, Hkv=2, D=128, page=64, codes="e4m3", io="bf16"),
        # a few short sequences, unquantised cache, three query heads to a key head
        dict(name="decode_short", op="attn_decode", B=5, L=300, Hq=12, Hkv=4, D=64, page=16, codes="io", io="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "kv_write", "kv_read", "attn_prefill", "attn_decode"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 72, 80, 96, 112, 128, 128, 128, 192, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        Hkv = min(Hkv, 4)
        return dict(op=op, T=_log(rng, 1, 8192), Hq=Hkv * rng.choice([1, 2, 3]), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 16.0]), io=io,
                    far=rng.choice([0, 0, 100000, 1000000]))
    if op == "kv_write":
        codes = rng.choice(["e4m3", "int8", "io"])
        rotate = codes != "int8" and rng.random() < 0.6
        Hq = Hkv * rng.choice([1, 3, 4]) if rotate else 0
        return dict(op=op, T=_log(rng, 1, 16384 if Hq <= 8 else 4096), Hkv=Hkv, D=min(D, 128), page=page, codes=codes,
                    Hq=Hq, rot=min(D, 128) if rotate else 0, io=io)
    if op == "kv_read":
        return dict(op=op, T=_log(rng, 1, 32768), Hkv=min(Hkv, 4), D=D, page=page,
                    codes=rng.choice(["e4m3", "int8", "io"]), io=io)
    G = rng.choice([1, 2, 3, 4, 8])
    if op == "attn_prefill":
        L = _log(rng, 1, 8192)
        return dict(op=op, B=max(1, min(_log(rng, 1, 24), 16384 // L)), L=L, ragged=rng.random() < 0.7,
                    past=rng.choice([0, 0, 1, 100, 1000]), Hq=Hkv * G, Hkv=Hkv, D=D, causal=rng.random() < 0.8,
                    io=io if L <= 2048 else "bf16")
    L = _log(rng, 1, 32768)
    return dict(op=op, B=max(1, min(_log(rng, 1, 64), 65536 // L)), L=L, Hq=Hkv * G, Hkv=Hkv, D=D, page=page,
                codes=rng.choice(["e4m3", "int8", "io"]), io=io)


# ---------------------------------------------------------------- what a program has before the call

def _lengths(case):
    """New tokens of each sequence: all L, or spread over 1 .. L with the ends among them."""
    B, L = case["B"], case["L"]
    if B == 1 or not case.get("ragged", True):
        return [L] * B
    return [max(1, L * (1 + (7 * i + 3) % B) // B - (i % 3)) if i else 1 for i in range(B - 1)] + [L]


def _past(case):
    """Keys of each sequence before its new tokens."""
    return [case["past"] * (i % 3) // 2 for i in range(case["B"])]


def _frequencies(rot, scaling, factor, dev, base=10000.0, orig=4096):
    """Radians per position of each rotated pair, fp64, and the factor on cos and sin."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    m = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        at = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        m = 0.1 * math.log(factor) + 1.0
    return f.to(dev), m


def _codes_of(x, codes):
    """The cache's form of rows x [..., D]: (codes, scales) or (x, None)."""
    if codes == "io":
        return x, None
    dtype, top = CODES[codes]
    x = x.float()
    amax = x.abs().amax(-1)
    live = amax >= TINY
    scale = torch.where(live, amax / top, torch.zeros_like(amax))
    mult = torch.where(live, top / amax, torch.zeros_like(amax))
    q = (x * mult.unsqueeze(-1)).clamp(-top, top)
    return (q.round() if codes == "int8" else q).to(dtype), scale


def _cache(case, pages, dev, io):
    dtype = io if case["codes"] == "io" else CODES[case["codes"]][0]
    shape = (pages, case["Hkv"], case["page"], case["D"])
    c = {n: torch.zeros(shape, dtype=F32, device=dev).to(dtype) for n in ("k", "v")}
    for n in ("k", "v"):
        c[n + "_scale"] = None if case["codes"] == "io" else torch.zeros(shape[:3], device=dev)
    return c


def _fill(c, case, g, dev, io):
    for n in ("k", "v"):
        x = torch.randn(c[n].shape, generator=g, device=dev)
        if n == "k":
            x *= torch.rand(c[n].shape[-1], generator=g, device=dev) * 2 + 0.2  # channels of different weight
        q, s = _codes_of(x.to(io), case["codes"])
        c[n], c[n + "_scale"] = q, s


def _handle(c):
    """The package's view of the same cache buffers."""
    import selective_state_space_causal_amd as ssm
    return ssm.KVCache(c["k"], c["v"], c["k_scale"], c["v_scale"])


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    io = IO[case["io"]]
    D, op = case["D"], case["op"]
    randn = lambda *s: torch.randn(*s, generator=g, device=dev).to(io)  # noqa: E731
    s = {"case": case}
    if op == "rope":
        T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
        s["qkv"] = randn(T, Hq + 2 * Hkv, D)  # a projection's packed output: q, k, v heads of a token side by side
        s["freq"], s["m"] = _frequencies(case["rot"], case["scaling"], case["factor"], dev)
        s["pos"] = torch.arange(T, device=dev) + case["far"]
    elif op == "kv_write":
        T, Hq, Hkv, page = case["T"], case["Hq"], case["Hkv"], case["page"]
        pages = -(-T // page) + 3
        s["qkv"] = randn(T, Hq + 2 * Hkv, D)
        s["cache"] = _cache(case, pages, dev, io)
        order = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        s["slots"] = order[t // page] * page + t % page
        if Hq:
            s["freq"], s["m"] = _frequencies(case["rot"], "none", 1.0, dev)
            s["pos"] = torch.randint(0, 32768, (T,), generator=g, device=dev)
    elif op == "kv_read":
        T, page = case["T"], case["page"]
        pages = -(-T // page) + 3
        s["cache"] = _cache(case, pages, dev, io)
        _fill(s["cache"], case, g, dev, io)
        order = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        s["slots"] = order[t // page] * page + t % page
    elif op == "attn_prefill":
        lq, past = _lengths(case), _past(case)
        lk = [a + b for a, b in zip(lq, past)]
        Tq, Tk, Hq, Hkv = sum(lq), sum(lk), case["Hq"], case["Hkv"]
        if Tq == Tk:
            qkv = randn(Tq, Hq + 2 * Hkv, D)
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = randn(Tq, Hq, D), randn(Tk, Hkv, D), randn(Tk, Hkv, D)
        s["lq"], s["lk"] = lq, lk
        ends = lambda n: torch.tensor([0] + n).cumsum(0).to(device=dev, dtype=torch.int32)  # noqa: E731
        s["cu_q"] = ends(lq)
        s["cu_k"] = ends(lk)
    else:
        B, page = case["B"], case["page"]
        lens = _lengths(case)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        s["cache"] = _cache(case, pages, dev, io)
        _fill(s["cache"], case, g, dev, io)
        order = torch.randperm(pages, generator=g, device=dev)[:sum(need)].to(torch.int32).split(need)
        table = torch.full((B, max(need)), -1, dtype=torch.int32, device=dev)
        for b, o in enumerate(order):
            table[b, :len(o)] = o
        s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q"] = randn(B, case["Hq"], D)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    io = IO[case["io"]]
    if op == "rope":
        Hq, Hkv = case["Hq"], case["Hkv"]
        rotate = lambda x: _rotate(x, s["pos"], s["freq"], s["m"], case["layout"] == "interleaved").to(io)  # noqa: E731
        return rotate(s["qkv"][:, :Hq]), rotate(s["qkv"][:, Hq:Hq + Hkv])
    if op == "kv_write":
        Hq, Hkv, c = case["Hq"], case["Hkv"], s["cache"]
        q, k, v = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
        if Hq:
            q, k = (_rotate(x, s["pos"], s["freq"], s["m"], False).to(io) for x in (q, k))
        page, off = s["slots"] // case["page"], s["slots"] % case["page"]
        for n, x in (("k", k), ("v", v)):
            codes, scale = _codes_of(x, case["codes"])
            as_bytes = (lambda t: t.view(torch.uint8)) if codes.element_size() == 1 else (lambda t: t)
            as_bytes(c[n])[page, :, off] = as_bytes(codes)
            if scale is not None:
                c[n + "_scale"][page, :, off] = scale
        return [q if Hq else None] + list(c.values())
    if op == "kv_read":
        c = s["cache"]
        return [_gather(c, n, s["slots"], case["page"]).to(io) for n in ("k", "v")]
    if op == "attn_prefill":
        return _plain_prefill(s, case, F32).to(io)
    return _plain_decode(s, case, F32).to(io)


def _own(s, case, op):
    import selective_state_space_causal_amd as ssm
    if op == "rope":
        Hq, Hkv = case["Hq"], case["Hkv"]
        return ssm.rope(s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["pos"], s["freq"], mscale=s["m"],
                        interleaved=case["layout"] == "interleaved")
    if op == "kv_write":
        Hq, Hkv = case["Hq"], case["Hkv"]
        q, k, v = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
        out = None
        if Hq:
            out = ssm.kv_write(k, v, _handle(s["cache"]), s["slots"], q=q, positions=s["pos"], freq=s["freq"],
                               mscale=s["m"])
        else:
            ssm.kv_write(k, v, _handle(s["cache"]), s["slots"])
        return [out] + list(s["cache"].values())
    if op == "kv_read":
        return list(ssm.kv_read(_handle(s["cache"]), s["slots"], dtype=IO[case["io"]]))
    if op == "attn_prefill":
        return ssm.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"])
    return ssm.attn_decode_step(s["q"], _handle(s["cache"]), s["table"], s["lens"])


# ---------------------------------------------------------------- plain forms

def _rotate(x, pos, freq, m, interleaved):
    """x [T, H, D] in fp32, its first 2 * len(freq) values rotated (angles in fp64: positions are far)."""
    angle = pos.double().unsqueeze(1) * freq
    cos, sin = (angle.cos() * m).float().unsqueeze(1), (angle.sin() * m).float().unsqueeze(1)
    rot = 2 * freq.numel()
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((p, q), -1).flatten(-2) if interleaved else torch.cat((p, q), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _gather(c, n, slots, page):
    at, off = slots // page, slots % page
    x = c[n].view(torch.uint8) if c[n].element_size() == 1 else c[n]
    x = x[at, :, off]
    x = (x.view(c[n].dtype) if c[n].element_size() == 1 else x).float()
    return x if c[n + "_scale"] is None else x * c[n + "_scale"][at, :, off].unsqueeze(-1)


def _plain_prefill(s, case, t, rows=2048):
    """Softmax attention of each sequence, `rows` queries at a time, in dtype t."""
    G, D, Hkv = case["Hq"] // case["Hkv"], case["D"], case["Hkv"]
    out = []
    q0 = k0 = 0
    for lq, lk in zip(s["lq"], s["lk"]):
        k = s["k"][k0:k0 + lk].to(t).permute(1, 2, 0).contiguous()  # [Hkv, D, lk]
        v = s["v"][k0:k0 + lk].to(t).transpose(0, 1).contiguous()
        for r in range(0, lq, rows):
            n = min(rows, lq - r)
            seen = lk if not case["causal"] else min(lk, r + n + lk - lq)
            q = s["q"][q0 + r:q0 + r + n].to(t).view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
            a = torch.matmul(q, k[:, :, :seen].contiguous()) * D ** -0.5
            if case["causal"]:
                i = torch.arange(r, r + n, device=q.device).repeat(G) + (lk - lq)
                a.masked_fill_(torch.arange(seen, device=q.device) > i.unsqueeze(1), -math.inf)
            a = (a - a.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(a, v[:, :seen].contiguous()) / a.sum(-1, keepdim=True)
            out.append(o.view(Hkv, G, n, D).permute(2, 0, 1, 3).reshape(n, Hkv * G, D))
        q0, k0 = q0 + lq, k0 + lk
    return torch.cat(out)


def _plain_decode(s, case, t):
    """All sequences at once, padded to the longest."""
    c, page, G = s["cache"], case["page"], case["Hq"] // case["Hkv"]
    B, W = s["table"].shape
    at = s["table"].clamp(min=0).long().view(-1)

    def rows(n):
        x = c[n][at].to(t) if c[n].element_size() > 1 else c[n].view(torch.uint8)[at].view(c[n].dtype).to(t)
        if c[n + "_scale"] is not None:
            x *= c[n + "_scale"][at].to(t).unsqueeze(-1)
        return x.view(B, W, case["Hkv"], page, case["D"]).permute(0, 2, 1, 3, 4).reshape(B, case["Hkv"], W * page, -1)

    k = rows("k")
    q = s["q"].to(t).view(B, case["Hkv"], G, case["D"])
    a = torch.matmul(k, q.transpose(2, 3).contiguous()).transpose(2, 3).contiguous() * case["D"] ** -0.5
    del k
    a.masked_fill_(torch.arange(W * page, device=q.device) >= s["lens"].view(B, 1, 1, 1), -math.inf)
    a = (a - a.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(a, rows("v")) / a.sum(-1, keepdim=True)
    return o.view(B, case["Hq"], case["D"])


# ---------------------------------------------------------------- work

def _size(t):
    return {"bf16": 2, "f32": 4, "io": None, "int8": 1, "e4m3": 1}[t]


def work(case):
    """Each input read once, each output written once, and the products (and rotations) of the formulas."""
    op, D, e = case["op"], case["D"], _size(case["io"])
    row = 0 if "codes" not in case else D * (_size(case["codes"]) or e) + (0 if case["codes"] == "io" else 4)
    if op == "rope":
        n = case["T"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 2 * n * D * e + 8 * case["T"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    if op == "kv_write":
        n = case["T"] * case["Hkv"]
        return {"bytes": 2 * n * (D * e + row) + case["T"] * (8 + (8 + 2 * case["Hq"] * D * e if case["Hq"] else 0)),
                "flops": 4 * n * D + 3 * case["T"] * (case["Hq"] + case["Hkv"]) * case["rot"]}
    if op == "kv_read":
        n = case["T"] * case["Hkv"]
        return {"bytes": 2 * n * (D * e + row) + 8 * case["T"], "flops": 2 * n * D}
    lens = _lengths(case)
    if op == "attn_prefill":
        past = _past(case)
        pairs = sum(n * p + (n * (n + 1) // 2 if case["causal"] else n * n) for n, p in zip(lens, past))
        new, keys = sum(lens), sum(lens) + sum(past)
        return {"bytes": e * D * (2 * new * case["Hq"] + 2 * keys * case["Hkv"]), "flops": 4 * D * case["Hq"] * pairs}
    keys = sum(lens)
    return {"bytes": 2 * keys * case["Hkv"] * row + 2 * case["B"] * case["Hq"] * D * e + 4 * keys // case["page"],
            "flops": 4 * D * case["Hq"] * keys}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, f = case["op"], torch.float64

    def turned(x, interleaved):
        """Each pair as a complex number times m * exp(i * position * frequency)."""
        x, h = x.to(f), s["freq"].numel()
        head = x[..., :2 * h].unflatten(-1, (h, 2) if interleaved else (2, h))
        z = torch.complex(*(head.unbind(-1) if interleaved else head.unbind(-2)))
        z = z * torch.polar(torch.full_like(s["freq"], s["m"]).expand(len(s["pos"]), h),
                            s["pos"].to(f)[:, None] * s["freq"][None, :])[:, None, :]
        y = torch.stack((z.real, z.imag), -1 if interleaved else -2).flatten(-2)
        return torch.cat((y, x[..., 2 * h:]), -1)

    if op == "rope":
        Hq, Hkv = case["Hq"], case["Hkv"]
        mode = case["layout"] == "interleaved"
        return turned(s["qkv"][:, :Hq], mode), turned(s["qkv"][:, Hq:Hq + Hkv], mode)
    if op == "kv_write":
        Hq, Hkv, c = case["Hq"], case["Hkv"], s["cache"]
        q = turned(s["qkv"][:, :Hq], False) if Hq else None
        k, v = s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
        k = (turned(k, False).to(IO[case["io"]]) if Hq else k).to(f)  # the cache is made of keys in the io dtype
        out = [q]
        for x in (k, v.to(f)):
            full = torch.zeros(c["k"].shape, dtype=f, device=x.device)
            sc = torch.zeros(c["k"].shape[:3], dtype=f, device=x.device)
            at, off = s["slots"].div(case["page"], rounding_mode="floor"), s["slots"].remainder(case["page"])
            if case["codes"] == "io":
                full[at, :, off] = x
                out += [full, None]
                continue
            top = CODES[case["codes"]][1]
            big = x.abs().max(-1).values
            sc[at, :, off] = big / top
            full[at, :, off] = x * (top / big)[..., None]
            # int8 codes are whole numbers, equal or not, and have no nearness
            out += [None if case["codes"] == "int8" else full.to(torch.float8_e4m3fn).to(f), sc]
        # run() gives q, k, v, k_scale, v_scale
        return [out[0], out[1], out[3], out[2], out[4]]
    if op == "kv_read":
        c, out = s["cache"], []
        for n in ("k", "v"):
            x = c[n].to(f).transpose(1, 2).flatten(0, 1)[s["slots"]]
            if c[n + "_scale"] is not None:
                x = x * c[n + "_scale"].to(f).transpose(1, 2).flatten(0, 1)[s["slots"]][..., None]
            out.append(x)
        return out
    G, D = case["Hq"] // case["Hkv"], case["D"]
    if op == "attn_prefill":
        out = torch.zeros(s["q"].shape, dtype=f, device="cuda")
        q0 = k0 = 0
        for lq, lk in zip(s["lq"], s["lk"]):
            for h in range(case["Hq"]):
                k, v = s["k"][k0:k0 + lk, h // G].to(f), s["v"][k0:k0 + lk, h // G].to(f)
                for r in range(0, lq, 4096):
                    n = min(4096, lq - r)
                    a = s["q"][q0 + r:q0 + r + n, h].to(f) @ k.t() / math.sqrt(D)
                    if case["causal"]:
                        a += torch.full_like(a, -math.inf).triu(lk - lq + r + 1)
                    out[q0 + r:q0 + r + n, h] = torch.softmax(a, -1) @ v
            q0, k0 = q0 + lq, k0 + lk
        return out
    c = s["cache"]
    out = torch.zeros(s["q"].shape, dtype=f, device="cuda")
    for b, n in enumerate(_lengths(case)):
        at = s["table"][b, :-(-n // case["page"])].long()
        for h in range(case["Hkv"]):
            kv = []
            for name in ("k", "v"):
                x = c[name][:, h]
                x = (x.view(torch.uint8)[at].view(x.dtype) if x.element_size() == 1 else x[at]).to(f)
                if c[name + "_scale"] is not None:
                    x = x * c[name + "_scale"][at, h].to(f)[..., None]
                kv.append(x.flatten(0, 1)[:n])
            a = torch.softmax(s["q"][b, h * G:(h + 1) * G].to(f) @ kv[0].t() / math.sqrt(D), -1)
            out[b, h * G:(h + 1) * G] = a @ kv[1]
    return out
