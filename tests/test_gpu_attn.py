"""The attention operators on the GPU against their fp64 definitions (oracle/attn.py): sizes, masks,
strides, page tables and types where they can go wrong.  Tolerances count roundings: half a step of the
io dtype (bf16 2^-8, fp32 2^-24) once at the end, and the terms that oracle.attn.attention_tolerance
derives."""
import numpy as np
import pytest
import torch

import selective_state_space_causal_amd as ssm
from oracle import attn as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def rnd(seed, *shape, io="bf16"):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[io])


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def close(got, want, tol, what):
    got = f64(got)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    bad = np.abs(got - want) - tol
    assert bad.max() <= 0, f"{what}: {np.abs(got - want).max():.3e} off, {bad.max():.3e} over the bound"


def packed(seed, T, Hq, Hkv, D, io):
    """q, k, v as the heads of a packed projection: strided views."""
    x = rnd(seed, T, Hq + 2 * Hkv, D, io=io).to(DEV)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


# ---------------------------------------------------------------- rope

ROPE = [  # T, Hq, Hkv, D, rot, interleaved, mscale, far
    (1, 1, 1, 8, 8, False, 1.0, 0), (1, 1, 1, 8, 2, True, 1.0, 5), (5, 3, 1, 64, 64, False, 1.0, 0),
    (7, 4, 2, 128, 64, True, 1.3, 0), (3, 2, 2, 72, 72, False, 1.0, 0), (3, 2, 2, 80, 40, True, 0.5, 0),
    (9, 2, 1, 40, 10, False, 1.0, 3), (9, 2, 1, 40, 10, True, 1.0, 3), (2, 1, 1, 256, 256, False, 1.0, 10 ** 6),
    (2, 1, 1, 256, 254, True, 1.0, 10 ** 6), (4, 5, 5, 24, 24, True, 1.0, 2 ** 40), (2100, 2, 1, 64, 32, False, 1.0, 0),
    (300, 40, 8, 128, 128, False, 1.0, 7),
]


def rope_tol(x, rot, interleaved, mscale, half, want):
    """Half an io step of the result, and of the pair's magnitudes: the angle in turns rounded to fp32
    (2 pi 2^-26), cos and sin (2^-22), their factor and three more fp32 operations (2^-22): below 2^-20."""
    a = np.abs(x)
    mag = a.copy()
    h = rot // 2
    ia = np.arange(h) * 2 if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    mag[..., ia] = mag[..., ib] = a[..., ia] + a[..., ib]
    return half * np.abs(want) + 2.0 ** -20 * max(mscale, 1.0) * mag


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", ROPE)
def test_rope(case, io):
    T, Hq, Hkv, D, rot, inter, ms, far = case
    q, k, _ = packed(1, T, Hq, Hkv, D, io)
    freq, _ = ssm.rope_frequencies(rot, device=DEV)
    pos = (torch.arange(T) * 3 + far).to(DEV)
    qo, ko = ssm.rope(q, k, pos, freq, interleaved=inter, mscale=ms)
    for got, x in ((qo, q), (ko, k)):
        want = O.rope(f64(x), f64(pos), f64(freq), inter, ms)
        close(got, want, rope_tol(f64(x), rot, inter, ms, HALF[io], want), "rope")
        assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_in_place_and_q_alone(io, inter):
    T, Hq, Hkv, D = 37, 6, 2, 96
    x = rnd(2, T, Hq + 2 * Hkv, D, io=io).to(DEV)
    before = x.clone()
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    freq, _ = ssm.rope_frequencies(48, device=DEV)
    pos = torch.randint(0, 4000, (T,), generator=torch.Generator().manual_seed(0)).to(DEV)
    qo, ko = ssm.rope(q, k, pos, freq, interleaved=inter)
    q1, none = ssm.rope(q, None, pos, freq, interleaved=inter)
    assert none is None and torch.equal(q1, qo)
    ssm.rope(q, k, pos, freq, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(x[:, Hq + Hkv:], before[:, Hq + Hkv:])  # v untouched
    # heads outermost: [H, T, D] storage seen as [T, H, D]
    qt = before[:, :Hq].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(ssm.rope(qt, None, pos, freq, interleaved=inter)[0], qo)


def test_rope_no_tokens():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    freq, _ = ssm.rope_frequencies(64, device=DEV)
    qo, ko = ssm.rope(q, None, torch.empty(0, dtype=torch.int64, device=DEV), freq)
    assert qo.shape == (0, 4, 64) and ko is None


# ---------------------------------------------------------------- cache

def new_cache(pages, Hkv, page, D, kind, io, fill=None):
    dtype = DT[io] if kind == "io" else {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[kind]
    c = ssm.KVCache.allocate(pages, page, Hkv, D, dtype, DEV)
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x7F if fill is None else fill)  # e4m3 and bf16: NaN; int8: 127
    for t in (c.k_scale, c.v_scale):
        if t is not None:
            t.fill_(float("nan") if fill is None else fill)
    return c


def values(c, n):
    """What the cache holds, as fp64 values [pages, H, page, D]."""
    x = f64(getattr(c, n).float())
    s = getattr(c, n + "_scale")
    return x if s is None else x * f64(s)[..., None]


WRITE = [  # T, Hkv, D, page, kind, rot (0: no rotation), Hq, interleaved
    (1, 1, 8, 16, "int8", 0, 0, False), (1, 2, 64, 16, "e4m3", 64, 4, False), (33, 3, 72, 16, "int8", 0, 0, False),
    (50, 2, 80, 32, "e4m3", 0, 0, False), (129, 8, 128, 64, "e4m3", 128, 16, False), (65, 1, 256, 64, "int8", 0, 0, False),
    (40, 2, 40, 16, "e4m3", 10, 2, True), (40, 2, 128, 1024, "io", 64, 0, True), (17, 4, 96, 16, "io", 0, 0, False),
    (3000, 2, 64, 64, "int8", 0, 0, False), (20, 2, 24, 16, "int8", 24, 6, False),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", WRITE)
def test_kv_write(case, io):
    T, Hkv, D, page, kind, rot, Hq, inter = case
    q, k, v = packed(3, T, max(Hq, 1), Hkv, D, io)
    if T > 2:
        k[1] *= 1000.0
        v[2] = 0.0
        k[0, 0] = 2.0 ** -110  # below the smallest stored magnitude
    pages = -(-T // page) + 2
    c = new_cache(pages, Hkv, page, D, kind, io)
    perm = torch.randperm(pages * page, generator=torch.Generator().manual_seed(4))[:T]
    skip = torch.arange(T) % 7 == 5
    slots = torch.where(skip, torch.where(torch.arange(T) % 2 == 0, -1, pages * page), perm).to(DEV)
    pos = torch.arange(T).to(DEV) * 5
    kw = {}
    if rot:
        freq, _ = ssm.rope_frequencies(rot, device=DEV)
        kw = dict(positions=pos, freq=freq, interleaved=inter, mscale=1.1, k_out=torch.empty(T, Hkv, D, dtype=DT[io], device=DEV))
        if Hq:
            kw["q"] = q
    before = [t.clone() for t in (c.k, c.v)]
    qo = ssm.kv_write(k, v, c, slots, **kw)
    stored_k = k
    if rot:
        rq, stored_k = ssm.rope(q, k, pos, freq, interleaved=inter, mscale=1.1)
        assert torch.equal(kw["k_out"], stored_k)
        assert (qo is None) == (Hq == 0) and (qo is None or torch.equal(qo, rq))
    written = torch.zeros(pages * page, dtype=torch.bool)
    written[perm[~skip]] = True
    written = written.view(pages, page)
    for n, x, old in (("k", stored_k, before[0]), ("v", v, before[1])):
        got = getattr(c, n).cpu()
        rows = got.permute(0, 2, 1, 3).reshape(pages * page, Hkv, D)[perm[~skip]]
        src = x.cpu()[~skip]
        if kind == "io":
            assert torch.equal(rows, src)
        else:
            want, scale = O.quantize(src.float().numpy(), kind)
            assert np.array_equal(f64(rows.float()), want)
            s = getattr(c, n + "_scale").cpu().permute(0, 2, 1).reshape(pages * page, Hkv)[perm[~skip]]
            assert np.array_equal(s.numpy(), scale)
        # nothing else was written
        keep = ~written.view(pages, 1, page, 1).expand(pages, Hkv, page, D)
        assert torch.equal(got.view(torch.uint8).reshape(pages, Hkv, page, -1)[~written.view(pages, 1, page).expand(pages, Hkv, page)],
                           old.cpu().view(torch.uint8).reshape(pages, Hkv, page, -1)[~written.view(pages, 1, page).expand(pages, Hkv, page)])
        assert keep.any()


@pytest.mark.parametrize("kind,io", [("int8", "bf16"), ("int8", "f32"), ("e4m3", "bf16"), ("e4m3", "f32"), ("io", "bf16"),
                                     ("io", "f32")])
@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 8, 16), (31, 3, 72, 16), (100, 2, 128, 64), (9, 4, 256, 32), (5000, 2, 64, 128)])
def test_kv_read(T, Hkv, D, page, kind, io):
    pages = 5 if T < 1000 else 40
    c = new_cache(pages, Hkv, page, D, kind, io, fill=0)
    n = pages * page
    x = rnd(5, n, 2 * Hkv, D, io=io).to(DEV)
    ssm.kv_write(x[:, :Hkv], x[:, Hkv:], c, torch.arange(n, device=DEV))
    slots = torch.randint(-3, n + 3, (T,), generator=torch.Generator().manual_seed(6)).to(DEV)
    k, v = ssm.kv_read(c, slots, dtype=DT[io])
    sl = slots.cpu().numpy()
    ok = (sl >= 0) & (sl < n)
    for got, name in ((k, "k"), (v, "v")):
        val = values(c, name).transpose(0, 2, 1, 3).reshape(n, Hkv, D)
        want = np.where(ok[:, None, None], val[np.clip(sl, 0, n - 1)], 0.0)
        # one fp32 product and one rounding to the io dtype
        close(got, want, (0 if kind == "io" else HALF[io] + 2.0 ** -24) * np.abs(want), "kv_read")


# ---------------------------------------------------------------- prefill

PREFILL = [  # lens q, past keys, Hq, Hkv, D, causal
    ([1], [0], 1, 1, 8, True), ([1], [0], 1, 1, 64, False), ([5], [0], 2, 1, 64, True), ([33], [0], 2, 2, 128, True),
    ([64, 1, 0, 65], [0, 0, 0, 0], 4, 2, 64, True), ([130], [70], 3, 1, 128, True), ([20, 31], [100, 1], 8, 2, 80, True),
    ([40], [-13], 4, 2, 64, True),  # fewer keys than queries: the first 13 see none
    ([7, 9], [-7, 3], 2, 2, 72, False),  # no keys at all
    ([150], [0], 2, 1, 256, True), ([90], [33], 2, 2, 192, False), ([70], [0], 4, 4, 136, True),
    ([6], [0], 17, 1, 40, True), ([3] * 70 + [200] + [2] * 60, [1] * 131, 2, 2, 64, True),
    ([300], [0], 1, 1, 128, False), ([257], [511], 2, 1, 96, True), ([20], [0], 64, 1, 112, True),
]


def prefill_case(lens, past, Hq, Hkv, D, io, seed=7):
    cu_q = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    lk = np.maximum(np.array(lens) + np.array(past), 0)
    cu_k = np.concatenate([[0], np.cumsum(lk)]).astype(np.int32)
    q = rnd(seed, max(int(cu_q[-1]), 1), Hq, D, io=io)
    k = rnd(seed + 1, int(cu_k[-1]), Hkv, D, io=io)
    v = rnd(seed + 2, int(cu_k[-1]), Hkv, D, io=io)
    return q, k, v, cu_q, cu_k


def check_attn(got, lse, ref, io, D, what, untouched=None):
    out, rlse, mag, smax, qkmax = ref
    keys = 1 << 10
    tol, ltol = O.attention_tolerance(HALF[io], HALF["bf16"] if io == "bf16" else 0.0, out, mag, smax, qkmax, D, keys)
    close(got, out, tol, what)
    if lse is not None:
        l = f64(lse)
        empty = np.isinf(rlse)
        assert np.array_equal(np.isneginf(l), empty), f"{what}: lse of empty rows"
        d = np.abs(np.where(empty, 0, l) - np.where(empty, 0, rlse))
        assert np.all(d <= ltol + 2.0 ** -22 * np.abs(np.where(empty, 0, rlse))), f"{what}: lse {d.max():.3e} off"
        assert np.all(f64(got)[empty] == 0), f"{what}: rows without keys are zero"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", PREFILL)
def test_attn_prefill(case, io):
    lens, past, Hq, Hkv, D, causal = case
    q, k, v, cu_q, cu_k = prefill_case(lens, past, Hq, Hkv, D, io)
    cq, ck = torch.from_numpy(cu_q).to(DEV), torch.from_numpy(cu_k).to(DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cq, ck, causal=causal, lse=lse)
    ref = O.prefill(f64(q), f64(k), f64(v), cu_q, cu_k, causal, D ** -0.5)
    n = int(cu_q[-1])
    check_attn(out[:n], lse[:n], [r[:n] for r in ref], io, D, f"{case}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attn_prefill_layouts_scale_and_gaps(io):
    """Packed projection views, heads-outermost storage, a strided output, another scale, and rows that
    belong to no sequence (NaN there: never read for others, and their outputs untouched)."""
    lens, Hq, Hkv, D = [40, 25], 6, 2, 64
    T = sum(lens) + 10
    x = rnd(11, T, Hq + 2 * Hkv, D, io=io)
    x[sum(lens):] = float("nan")
    xd = x.to(DEV)
    cu = torch.tensor([0, 40, 65], dtype=torch.int32, device=DEV)
    q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    big = torch.full((T, Hq + 1, D), 3.0, dtype=DT[io], device=DEV)
    out = ssm.attn_prefill(q, k, v, cu, scale=0.3, out=big[:, 1:])
    ref = O.prefill(f64(x[:, :Hq]), f64(x[:, Hq:Hq + Hkv]), f64(x[:, Hq + Hkv:]), [0, 40, 65], [0, 40, 65], True, 0.3)
    check_attn(out[:65], None, [r[:65] for r in ref], io, D, "strided")
    assert torch.all(big[65:] == 3.0) and torch.all(big[:, 0] == 3.0)
    t = lambda y: y.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    assert torch.equal(ssm.attn_prefill(t(q), t(k), t(v), cu, scale=0.3)[:65], out[:65])


def test_attn_prefill_bad_offsets_are_clamped():
    """Offsets outside the tensors are clamped, descending ones make empty sequences: no access past an end."""
    q, k, v = packed(12, 50, 2, 1, 64, "bf16")
    cu_q = torch.tensor([-5, 20, 10, 1000], dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([0, 20, 2 ** 31 - 1, 50], dtype=torch.int32, device=DEV)
    out = torch.zeros(50, 2, 64, dtype=torch.bfloat16, device=DEV)
    ssm.attn_prefill(q, k, v, cu_q, cu_k, out=out)
    ref = O.prefill(f64(q)[:20], f64(k), f64(v), [0, 20], [0, 20], True, 64 ** -0.5)
    check_attn(out[:20][:10], None, [r[:10] for r in ref], "bf16", 64, "first sequence")


def test_attn_prefill_large_scores():
    """Scores of +-10^4: the running maximum has to be subtracted before the exponential."""
    lens = [200]
    q, k, v, cu_q, cu_k = prefill_case(lens, [0], 2, 2, 64, "f32")
    q = q * 100
    k = k * 100
    cq = torch.from_numpy(cu_q).to(DEV)
    out = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cq)
    ref = O.prefill(f64(q), f64(k), f64(v), cu_q, cu_k, True, 64 ** -0.5)
    check_attn(out, None, ref, "f32", 64, "large scores")


# ---------------------------------------------------------------- decode

DECODE = [  # lens, Hq, Hkv, D, page, kind
    ([1], 1, 1, 8, 16, "int8"), ([17], 2, 1, 64, 16, "e4m3"), ([0, 5, 64, 65], 4, 2, 64, 16, "io"),
    ([300, 1], 12, 4, 72, 16, "int8"), ([129, 1000], 8, 1, 128, 64, "e4m3"), ([33], 16, 1, 80, 32, "int8"),
    ([50, 2], 17, 1, 64, 16, "e4m3"), ([70], 40, 2, 40, 1024, "int8"), ([90], 4, 4, 256, 16, "e4m3"),
    ([31, 32, 33], 6, 2, 192, 32, "int8"), ([513], 3, 1, 136, 64, "io"), ([2500], 2, 2, 128, 64, "int8"),
    ([7] * 70, 2, 1, 64, 16, "io"), ([40], 32, 1, 256, 16, "io"),
]


def decode_case(lens, Hq, Hkv, D, page, kind, io, seed=20):
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + 2
    c = new_cache(pages, Hkv, page, D, kind, io)  # everything unwritten is NaN (int8: 127 times NaN)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    W = max(max(need), 1) + 1
    table = torch.full((len(lens), W), -1, dtype=torch.int32)
    at, slots = 0, []
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        j = torch.arange(max(n, 0))
        slots.append(table[b, j // page].long() * page + j % page)
    slots = torch.cat(slots).to(DEV)
    x = rnd(seed, max(len(slots), 1), 2 * Hkv, D, io=io).to(DEV)[:len(slots)]
    if len(slots):
        ssm.kv_write(x[:, :Hkv], x[:, Hkv:], c, slots)
    return c, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), rnd(seed + 1, len(lens), Hq, D, io=io).to(DEV)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", DECODE)
def test_attn_decode(case, io):
    lens, Hq, Hkv, D, page, kind = case
    c, table, n, q = decode_case(lens, Hq, Hkv, D, page, kind, io)
    lse = torch.empty(len(lens), Hq, device=DEV)
    out = ssm.attn_decode_step(q, c, table, n, lse=lse)
    ref = O.decode(f64(q), values(c, "k"), values(c, "v"), table.cpu().numpy(), lens, D ** -0.5)
    check_attn(out, lse, ref, io, D, f"{case}")
    assert torch.equal(ssm.attn_decode_step(q, c, table, n), out)  # the same bits again


@pytest.mark.parametrize("kind", ["int8", "e4m3", "io"])
def test_attn_decode_bad_pages_and_lengths(kind):
    """Pages outside the cache are not seen, lengths are clamped to the table, NaN past a length stays out."""
    lens, page = [100, 64, 40, 33], 16
    c, table, n, q = decode_case(lens, 4, 2, 64, page, kind, "bf16")
    table[0, 2] = 10 ** 6
    table[1, 0] = -7
    table[2, :] = 2 ** 31 - 1
    n = torch.tensor([100, 64, 40, -3], dtype=torch.int32, device=DEV)
    lse = torch.empty(4, 4, device=DEV)
    out = ssm.attn_decode_step(q, c, table, n, lse=lse)
    ref = O.decode(f64(q), values(c, "k"), values(c, "v"), table.cpu().numpy(), n.cpu().numpy(), 64 ** -0.5)
    check_attn(out, lse, ref, "bf16", 64, "bad pages")
    assert torch.all(out[2:] == 0)
    # a length past the table is the table's
    full = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    full[0, 0], full[0, 1] = int(table[3, 0]), int(table[3, 1])
    a = ssm.attn_decode_step(q[3:4], c, full, torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=DEV))
    b = ssm.attn_decode_step(q[3:4], c, full, torch.tensor([32], dtype=torch.int32, device=DEV))
    assert torch.equal(a, b)


def test_attn_decode_strided_q_and_out():
    c, table, n, q = decode_case([45, 80], 4, 2, 64, 16, "e4m3", "bf16")
    want = ssm.attn_decode_step(q, c, table, n)
    wide = torch.zeros(2, 7, 64, dtype=torch.bfloat16, device=DEV)
    wide[:, 2:6] = q
    big = torch.full((2, 6, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    ssm.attn_decode_step(wide[:, 2:6], c, table, n, out=big[:, :4])
    assert torch.equal(big[:, :4], want) and torch.all(big[:, 4:] == 5.0)


def test_prefill_and_decode_agree():
    """The last token of a prompt by attn_prefill, and by attn_decode_step against the cache that the prompt
    left (unquantised): the same formula, so both are within their tolerance of it."""
    T, Hq, Hkv, D, page = 75, 8, 2, 128, 16
    q, k, v = packed(30, T, Hq, Hkv, D, "bf16")
    c = new_cache(6, Hkv, page, D, "io", "bf16")
    ssm.kv_write(k, v, c, torch.arange(T, device=DEV))
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    whole = ssm.attn_prefill(q, k, v, cu)
    one = ssm.attn_decode_step(q[-1:], c, torch.arange(6, dtype=torch.int32, device=DEV)[None],
                               torch.tensor([T], dtype=torch.int32, device=DEV))
    ref = O.prefill(f64(q), f64(k), f64(v), [0, T], [0, T], True, D ** -0.5)
    check_attn(whole, None, ref, "bf16", D, "prefill")
    check_attn(one, None, [r[-1:] for r in ref], "bf16", D, "decode")


# ---------------------------------------------------------------- streams and graphs

def test_attn_on_another_stream():
    s = torch.cuda.Stream()
    c, table, n, q = decode_case([500, 30], 8, 2, 128, 16, "int8", "bf16")
    want = ssm.attn_decode_step(q, c, table, n)
    qp, k, v = packed(31, 200, 4, 2, 64, "bf16")
    cu = torch.tensor([0, 90, 200], dtype=torch.int32, device=DEV)
    wantp = ssm.attn_prefill(qp, k, v, cu)
    s.wait_stream(torch.cuda.current_stream())
    got = [ssm.attn_decode_step(q, c, table, n, stream=s) for _ in range(3)]
    gotp = ssm.attn_prefill(qp, k, v, cu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(g, want) for g in got) and torch.equal(gotp, wantp)


def test_attn_decode_graph_replays():
    """A decode step (rotation, cache write, attention) captured once and replayed with new inputs in the
    same buffers, against the eager calls."""
    B, Hq, Hkv, D, page = 3, 8, 2, 64, 16
    lens0 = [40, 7, 100]
    c, table, n, _ = decode_case(lens0, Hq, Hkv, D, page, "e4m3", "bf16")
    c2 = ssm.KVCache(c.k.clone(), c.v.clone(), c.k_scale.clone(), c.v_scale.clone())
    freq, m = ssm.rope_frequencies(D, device=DEV)
    x = torch.empty(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    n += 1
    ws = torch.empty(max(1, ssm.attn_decode_workspace_bytes(B, Hq, c, table.shape[1])), dtype=torch.uint8, device=DEV)
    slots, pos = torch.empty(B, dtype=torch.int64, device=DEV), torch.empty(B, dtype=torch.int64, device=DEV)
    qo, out = (torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def fill(i):
        x.copy_(rnd(40 + i, B, Hq + 2 * Hkv, D).to(DEV))
        pos.copy_(n.long() - 1)
        slots.copy_(table.long().gather(1, (pos // page)[:, None])[:, 0] * page + pos % page)

    def step(cache):
        ssm.kv_write(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, slots, q=x[:, :Hq], positions=pos, freq=freq, q_out=qo)
        ssm.attn_decode_step(qo, cache, table, n, out=out, workspace=ws)

    fill(0)
    step(c2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c)
    for i in range(4):
        fill(i)
        g.replay()
        got = out.clone()
        torch.cuda.synchronize()
        step(c2)
        assert torch.equal(out, got), i
        assert torch.equal(c.k.view(torch.uint8), c2.k.view(torch.uint8))
        n += 1


# ---------------------------------------------------------------- many tiles, many chunks

def whole_sequences(q, k, v, cu_q, cu_k, causal, scale):
    """O.prefill by whole matrices of each sequence and head (the same five results)."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse, mag = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf), np.zeros((T, Hq, D))
    smax, qkmax = np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        if lq <= 0 or lk <= 0:
            continue
        seen = np.minimum(np.maximum(np.arange(lq) + 1 + lk - lq, 0), lk) if causal else np.full(lq, lk)
        mask = np.arange(lk)[None, :] < seen[:, None]
        some = seen > 0
        rows = slice(cu_q[b], cu_q[b + 1])
        for h in range(Hq):
            kk, vv, qq = k[cu_k[b]:cu_k[b + 1], h // G], v[cu_k[b]:cu_k[b + 1], h // G], q[rows, h]
            s = np.where(mask, scale * (qq @ kk.T), -np.inf)
            m = np.where(some, s.max(-1, initial=-np.inf), 0.0)
            p = np.exp(s - m[:, None])
            l = np.where(some, p.sum(-1), 1.0)
            w = p / l[:, None]
            out[rows, h], mag[rows, h] = w @ vv, w @ np.abs(vv)
            lse[rows, h] = np.where(some, m + np.log(l), -np.inf)
            smax[rows, h] = np.where(some, np.abs(np.where(mask, s, 0.0)).max(-1), 0.0)
            qkmax[rows, h] = np.where(some, np.where(mask, scale * (np.abs(qq) @ np.abs(kk).T), 0.0).max(-1), 0.0)
    return out, lse, mag, smax, qkmax


def test_whole_sequences_is_the_oracle():
    q, k, v, cu_q, cu_k = prefill_case([5, 0, 9, 4], [3, 2, -4, -9], 4, 2, 16, "f32")
    for causal in (True, False):
        for a, b in zip(whole_sequences(f64(q), f64(k), f64(v), cu_q, cu_k, causal, 0.25),
                        O.prefill(f64(q), f64(k), f64(v), cu_q, cu_k, causal, 0.25)):
            np.testing.assert_allclose(a, b, atol=1e-12)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,longest,Hq,Hkv,D,causal", [
    (61, 150, 32, 1, 64, True), (64, 120, 32, 1, 128, True), (200, 60, 32, 1, 96, True), (7, 700, 64, 2, 72, False),
    (30, 260, 32, 1, 256, True), (40, 180, 40, 2, 192, True)])
def test_attn_prefill_many_tiles(B, longest, Hq, Hkv, D, causal, io):
    """More tiles of rows than workgroups, of sequences of all lengths (none among them), some with past keys, some
    with fewer keys than queries: each workgroup goes from tile to tile."""
    g = np.random.default_rng(B)
    lens = [int(n) for n in g.integers(0, longest, B)]
    past = [int(n) for n in g.choice([0, 0, 0, 1, 50, -20], B)]
    q, k, v, cu_q, cu_k = prefill_case(lens, past, Hq, Hkv, D, io)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), torch.from_numpy(cu_q).to(DEV), torch.from_numpy(cu_k).to(DEV),
                           causal=causal, lse=lse)
    ref = whole_sequences(f64(q), f64(k), f64(v), cu_q, cu_k, causal, D ** -0.5)
    check_attn(out, lse, ref, io, D, "many tiles")


@pytest.mark.parametrize("io,kind", [("bf16", "int8"), ("bf16", "e4m3"), ("f32", "io")])
def test_attn_decode_many_chunks(io, kind):
    """A sequence in more than 64 chunks, beside short ones in the same call."""
    lens, Hq, Hkv, D, page = [20011, 5, 0, 16640], 6, 2, 72, 32
    c, table, n, q = decode_case(lens, Hq, Hkv, D, page, kind, io)
    lse = torch.empty(len(lens), Hq, device=DEV)
    out = ssm.attn_decode_step(q, c, table, n, lse=lse)
    ref = O.decode(f64(q), values(c, "k"), values(c, "v"), table.cpu().numpy(), lens, D ** -0.5)
    o, rlse, mag, smax, qkmax = ref
    tol, ltol = O.attention_tolerance(HALF[io], HALF["bf16"] if io == "bf16" else 0.0, o, mag, smax, qkmax, D, 1 << 15)
    close(out, o, tol, "many chunks")
    got, empty = f64(lse), np.isinf(rlse)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(np.where(empty, 0, got) - np.where(empty, 0, rlse)) <= ltol + 2.0 ** -22 * np.abs(np.where(empty, 0, rlse)))
    assert torch.equal(ssm.attn_decode_step(q, c, table, n), out)


@pytest.mark.parametrize("B", [64, 150])
@pytest.mark.parametrize("case", [c for c in PREFILL if sum(c[0]) <= 300])
def test_attn_prefill_edges_in_large_calls(case, B):
    """The edges of PREFILL in calls of many sequences, which run another kernel than a few rows do: the sequences
    in turn until there are B, as views of a packed projection, into a strided output."""
    lens, past, Hq, Hkv, D, causal = case
    n = len(lens)
    lq = [lens[i % n] for i in range(B)]
    lk = [max(lens[i % n] + past[i % n], 0) for i in range(B)]
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (lq, lk))
    Tq, Tk = int(cu_q[-1]), int(cu_k[-1])
    x = rnd(50, Tq + 3, Hq + 2, D)
    y = rnd(51, Tk + 3, 2 * Hkv + 1, D)
    x[Tq:], y[Tk:] = float("nan"), float("nan")
    q, k, v = x[:, 1:Hq + 1], y[:, :Hkv], y[:, Hkv + 1:]
    xd, yd = x.to(DEV), y.to(DEV)
    big = torch.full((Tq + 3, Hq + 1, D), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Tq + 3, Hq), 7.0, device=DEV)
    out = ssm.attn_prefill(xd[:, 1:Hq + 1], yd[:, :Hkv], yd[:, Hkv + 1:], torch.from_numpy(cu_q).to(DEV),
                           torch.from_numpy(cu_k).to(DEV), causal=causal, out=big[:, 1:], lse=lse)
    ref = whole_sequences(f64(q)[:Tq], f64(k)[:Tk], f64(v)[:Tk], cu_q, cu_k, causal, D ** -0.5)
    check_attn(out[:Tq], lse[:Tq], ref, "bf16", D, f"{case} x {B}")
    assert torch.all(big[Tq:] == 3.0) and torch.all(big[:, 0] == 3.0) and torch.all(lse[Tq:] == 7.0)


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([700], 8, 2, 128), ([90, 1500], 4, 4, 64), ([300] * 20, 8, 2, 128), ([7] * 90, 4, 1, 72)])
def test_attn_prefill_graph_replays(lens, Hq, Hkv, D):
    """A captured call replayed on new inputs in the same buffers against the eager call; one graph for the
    kernel of few rows and one for the other."""
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(DEV)
    x = torch.empty(sum(lens), Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    out = torch.empty(sum(lens), Hq, D, dtype=torch.bfloat16, device=DEV)
    x.copy_(rnd(60, *x.shape).to(DEV))
    ssm.attn_prefill(q, k, v, cu, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssm.attn_prefill(q, k, v, cu, out=out)
    for i in range(4):
        x.copy_(rnd(61 + i, *x.shape).to(DEV))
        out.zero_()
        g.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(ssm.attn_prefill(q, k, v, cu), got), i


@pytest.mark.parametrize("lens,past,Hq,Hkv,D", [([2200, 3000], [0, 40], 12, 1, 64), ([2500], [700], 16, 2, 96), ([2304], [0], 24, 3, 128)])
def test_attn_prefill_long_sequences(lens, past, Hq, Hkv, D):
    """Sequences of more than 2048 keys."""
    q, k, v, cu_q, cu_k = prefill_case(lens, past, Hq, Hkv, D, "bf16")
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), torch.from_numpy(cu_q).to(DEV), torch.from_numpy(cu_k).to(DEV), lse=lse)
    ref = whole_sequences(f64(q), f64(k), f64(v), cu_q, cu_k, True, D ** -0.5)
    o, rlse, mag, smax, qkmax = ref
    tol, ltol = O.attention_tolerance(HALF["bf16"], HALF["bf16"], o, mag, smax, qkmax, D, 1 << 12)
    close(out, o, tol, "long sequences")
    assert np.all(np.abs(f64(lse) - rlse) <= ltol + 2.0 ** -22 * np.abs(rlse))


@pytest.mark.parametrize("Hkv,D,causal", [  # Hkv: 66 tiles of 128 rows to a key head
    (2, 64, True), (2, 80, True), (2, 96, True), (3, 128, True), (1, 128, False), (2, 256, True), (1, 224, False),  # 64 rows
    (4, 64, True), (4, 72, True), (4, 128, True), (3, 120, False), (2, 192, True), (3, 136, False)])  # 128 rows
def test_attn_prefill_shared_keys(Hkv, D, causal):
    """Tiles of rows whose keys are shared by waves: sequences of all lengths, none and one among them, rows that see
    no key, shares that see none, as views of a packed projection into a strided output."""
    lq, past, G = [300, 1, 0, 37, 64, 65, 5], [700, 500, 300, 900, 0, 1, -3], 16
    lk = [max(a + b, 0) for a, b in zip(lq, past)]
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (lq, lk))
    Tq, Tk, Hq = int(cu_q[-1]), int(cu_k[-1]), Hkv * G
    x, y = rnd(70, Tq + 3, Hq + 2, D), rnd(71, Tk + 3, 2 * Hkv + 1, D)
    x[Tq:], y[Tk:] = float("nan"), float("nan")
    q, k, v = x[:, 1:Hq + 1], y[:, :Hkv], y[:, Hkv + 1:]
    xd, yd = x.to(DEV), y.to(DEV)
    big = torch.full((Tq + 3, Hq + 1, D), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Tq + 3, Hq), 7.0, device=DEV)
    args = (xd[:Tq, 1:Hq + 1], yd[:Tk, :Hkv], yd[:Tk, Hkv + 1:], torch.from_numpy(cu_q).to(DEV), torch.from_numpy(cu_k).to(DEV))
    out = ssm.attn_prefill(*args, causal=causal, out=big[:Tq, 1:], lse=lse[:Tq])
    ref = whole_sequences(f64(q)[:Tq], f64(k)[:Tk], f64(v)[:Tk], cu_q, cu_k, causal, D ** -0.5)
    check_attn(out, lse[:Tq], ref, "bf16", D, f"{Hkv} {D}")
    assert torch.all(big[Tq:] == 3.0) and torch.all(big[:, 0] == 3.0) and torch.all(lse[Tq:] == 7.0)
    again = ssm.attn_prefill(*args, causal=causal)
    assert torch.equal(again, out)


@pytest.mark.parametrize("Hkv,D", [(2, 128), (2, 256), (2, 192), (4, 64)])
def test_attn_prefill_shared_keys_graph_replays(Hkv, D):
    test_attn_prefill_graph_replays([700, 0, 350], Hkv * 8, Hkv, D)


@pytest.mark.parametrize("new,past,Hq,Hkv,D,causal", [(2000, 5000, 40, 1, 64, True), (1700, 4500, 48, 1, 128, False),
                                                      (6200, 0, 26, 2, 96, True)])
def test_attn_prefill_very_long_sequence(new, past, Hq, Hkv, D, causal):
    """Thousands of keys and rows: the first, some middle and the last tokens, and the last key head, against the
    same rows as sequences of their own."""
    g = torch.Generator().manual_seed(80)
    q, k, v = (torch.randn(n, h, D, generator=g).bfloat16() for n, h in ((new, Hq), (new + past, Hkv), (new + past, Hkv)))
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (new, new + past))
    out = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_q, cu_k, causal=causal)
    G = Hq // Hkv
    for first, last in ((0, 20), (new // 2, new // 2 + 20), (new - 20, new)):
        keys = past + last if causal else past + new
        kv = [f64(t)[:keys, -1:] for t in (k, v)]
        o, _, mag, smax, qkmax = whole_sequences(f64(q)[first:last, -G:], *kv, np.array([0, last - first]), np.array([0, keys]),
                                                 causal, D ** -0.5)
        tol, _ = O.attention_tolerance(HALF["bf16"], HALF["bf16"], o, mag, smax, qkmax, D, 1 << 13)
        close(out[first:last, -G:], o, tol, f"tokens from {first}")


# ---------------------------------------------------------------- the binding's two halves

def test_native_and_python_bindings_agree(monkeypatch):
    """Every call through the native half of the binding and through attn.py alone: the same bits, given outputs filled
    and returned as they are, and the same refusals."""
    from selective_state_space_causal_amd import attn as A
    assert A._bound() is not A._NoNative, "the native binding is not built"
    T, Hq, Hkv, D, page = 70, 6, 2, 64, 16
    q, k, v = packed(70, T, Hq, Hkv, D, "bf16")
    freq, m = ssm.rope_frequencies(32, scaling="yarn", factor=4.0, device=DEV)
    pos, slots = torch.arange(T, device=DEV) * 3, torch.randperm(96, generator=torch.Generator().manual_seed(1))[:T].to(DEV)
    cu = torch.tensor([0, 30, T], dtype=torch.int32, device=DEV)
    table = torch.arange(6, dtype=torch.int32, device=DEV)[None].repeat(2, 1)
    lens = torch.tensor([90, 0], dtype=torch.int32, device=DEV)
    caches = {kind: new_cache(6, Hkv, page, D, kind, "bf16", fill=0) for kind in ("int8", "e4m3", "io")}
    big = new_cache(600, Hkv, page, D, "e4m3", "bf16", fill=0)  # a table of several chunks: with a workspace
    wide = torch.arange(600, dtype=torch.int32, device=DEV)[None]

    def calls():
        res = []
        for inter in (False, True):
            res += ssm.rope(q, k, pos, freq, interleaved=inter, mscale=m)
        res.append(ssm.rope(q, None, pos, freq)[0])
        qo, ko = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
        r = ssm.rope(q, k, pos, freq, q_out=qo, k_out=ko)
        assert r[0] is qo and r[1] is ko
        res += r
        for c in caches.values():
            c.k.view(torch.uint8).zero_()
            assert ssm.kv_write(k, v, c, slots) is None
            res.append(c.k.view(torch.uint8).clone())
            res.append(ssm.kv_write(k, v, c, slots, q=q, positions=pos, freq=freq, mscale=m))
            ko = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
            assert ssm.kv_write(k, v, c, slots, q=q, positions=pos, freq=freq, mscale=m, q_out=qo, k_out=ko) is qo
            assert ssm.kv_write(k, v, c, slots, positions=pos, freq=freq, interleaved=True, k_out=ko) is None
            res += [qo.clone(), ko, c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()]
            res += ssm.kv_read(c, slots)
            if c.io_only is None:
                res += ssm.kv_read(c, slots, dtype=torch.float32)
            lse = torch.empty(2, Hq, device=DEV)
            res += [ssm.attn_decode_step(q[:2], c, table, lens, lse=lse), lse]
            out = torch.empty(2, Hq, D, dtype=torch.bfloat16, device=DEV)
            assert ssm.attn_decode_step(q[:2], c, table, lens, scale=0.3, out=out) is out
            res.append(out)
        res.append(ssm.attn_decode_step(q[:1], big, wide, torch.tensor([9000], dtype=torch.int32, device=DEV)))
        lse = torch.empty(T, Hq, device=DEV)
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        assert ssm.attn_prefill(q, k, v, cu, cu, causal=False, scale=0.2, out=out, lse=lse) is out
        return [t.clone() for t in res] + [out, lse, ssm.attn_prefill(q, k, v, cu)]

    def refusals():
        c = caches["int8"]
        bad = [lambda: ssm.rope(q, None, pos[:-1], freq), lambda: ssm.rope(q, None, pos, freq.float()), lambda: ssm.rope(q.half(), None, pos, freq),
               lambda: ssm.rope(q, None, pos, freq, k_out=k), lambda: ssm.rope(q, None, pos.cpu(), freq), lambda: ssm.rope(q, k, pos, freq, q_out=k),
               lambda: ssm.rope(q[..., ::2], None, pos, freq), lambda: ssm.rope(q, None, pos, freq, q_out=q[:, 1:]),
               lambda: ssm.rope(q[..., :12].contiguous(), None, pos, freq[:4]), lambda: ssm.kv_write(k, v[:-1], c, slots),
               lambda: ssm.kv_write(k, v, c, slots, q=q), lambda: ssm.kv_write(k, v, c, slots, positions=pos),
               lambda: ssm.kv_write(k.float(), v, c, slots), lambda: ssm.kv_write(k.float(), v.float(), caches["io"], slots),
               lambda: ssm.kv_write(k, v, c, slots.int()), lambda: ssm.kv_read(c, slots[:, None]), lambda: ssm.kv_read(c, slots, dtype=torch.float16),
               lambda: ssm.kv_read(caches["io"], slots, dtype=torch.float32), lambda: ssm.kv_read(c, slots, k_out=k, v_out=k),
               lambda: ssm.attn_prefill(q, k, v, cu.long()), lambda: ssm.attn_prefill(q, k, v[:-1], cu), lambda: ssm.attn_prefill(q, k, v, cu, scale=-1.0),
               lambda: ssm.attn_prefill(q, k, v, cu, out=q), lambda: ssm.attn_prefill(q[:, :5], k, v, cu), lambda: ssm.attn_prefill(q, k, v, cu[:1]),
               lambda: ssm.attn_decode_step(q[:2], c, table[:1], lens), lambda: ssm.attn_decode_step(q[:2], c, table, lens.long()),
               lambda: ssm.attn_decode_step(q[:2], c, table[0], lens), lambda: ssm.attn_decode_step(q[:2].float(), caches["io"], table, lens),
               lambda: ssm.attn_decode_step(q[:2, :, :32], c, table, lens), lambda: ssm.attn_decode_step(q[:2], c, table, lens, out=q[:2])]
        res = []
        for f in bad:
            with pytest.raises((ValueError, TypeError, ssm.SsmError)) as e:
                f()
            res.append((type(e.value), str(e.value)))
        return res

    def described():
        res = []
        for c in (*caches.values(), big):
            n = ssm.KVCache(c.k, c.v, c.k_scale, c.v_scale)
            res.append([bytes(n._desc[:56]), *(getattr(n, x) for x in n.__slots__ if x not in ("_desc", "address"))])
        c = caches["int8"]
        for bad in ((c.k, c.v), (c.k, c.v[:2], c.k_scale, c.v_scale), (c.k, c.v, c.k_scale[:2], c.v_scale), (c.k[:, :, ::2], c.v[:, :, ::2]),
                    (c.k, c.v, c.k_scale.double(), c.v_scale), (c.k.half(), c.v.half()), (c.k[0], c.v[0]), (c.k, c.v.cpu(), c.k_scale, c.v_scale),
                    (caches["io"].k, caches["io"].v, c.k_scale, c.v_scale), (c.k, None, c.k_scale, c.v_scale)):
            with pytest.raises((ValueError, TypeError)) as e:
                ssm.KVCache(*bad)
            res.append((type(e.value), str(e.value)))
        return res

    native, said, caches_native = calls(), refusals(), described()
    monkeypatch.setattr(A, "_native", A._NoNative)
    for a, b in zip(caches_native, described()):
        assert all(x is y if isinstance(x, torch.Tensor) else x == y for x, y in zip(a, b))
    for i, (a, b) in enumerate(zip(native, calls())):
        assert torch.equal(a, b), i
    assert refusals() == said
