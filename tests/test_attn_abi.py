"""C ABI of the attention operators (include/ssm_attn.h) without a GPU: exports and host-side
validation.  Every call below is invalid on purpose (or has no tokens) and must be answered before any
HIP call, so the fake device addresses are never dereferenced or launched on."""
import ctypes
import math
import os
import re

import pytest
import torch

from selective_state_space_causal_amd import _lib as L
from selective_state_space_causal_amd import attn as A

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake-pointer tests run only without a GPU")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssm_attn.h")
OK, NULL, SHAPE, DTYPE, ALIGN, ALIAS, WORKSPACE = range(7)
BASE, STEP = 0x7F0000000000, 1 << 36
T, HQ, HK, D, PAGE, PAGES, B, W = 10, 4, 2, 64, 16, 8, 3, 500  # 8000 tokens: several chunks, with a workspace


def at(i, off=0):
    return BASE + i * STEP + off


def view(i, heads=HQ, off=0, ts=None, hs=D):
    return A._View(at(i, off), heads * D if ts is None else ts, hs)


def cache(kind=A.KV_I8, k=None, v=None, ks=None, vs=None, pages=PAGES, page=PAGE, heads=HK, dim=D):
    return A._Cache(at(20) if k is None else k, at(21) if v is None else v, at(22) if ks is None else ks,
                    at(23) if vs is None else vs, pages, page, heads, dim, kind)


def rope_desc(pos=None, freq=None, pairs=D // 2, inter=0, ms=1.0):
    return A._Rope(at(30) if pos is None else pos, at(31) if freq is None else freq, pairs, inter, ms)


def test_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ssm_[a-z0-9_]+)\s*\(", src)))
    assert names == ["ssm_attn_decode_step", "ssm_attn_decode_workspace_bytes", "ssm_attn_prefill", "ssm_kv_read",
                     "ssm_kv_write", "ssm_rope"]
    lib = L.load()
    for n in names:
        assert hasattr(lib, n), n


def rope(tokens=T, hq=HQ, hk=HK, dim=D, io=L.SSM_BF16, r="", q="", qo="", k="", ko=""):
    pick = lambda x, d: d if x == "" else x  # noqa: E731
    return L.load().ssm_rope(tokens, hq, hk, dim, io, pick(r, rope_desc()), pick(q, view(0)), pick(qo, view(1)),
                             pick(k, view(2, HK)), pick(ko, view(3, HK)), None)


def test_rope_validation():
    assert rope(tokens=0) == OK
    assert rope(tokens=-1) == SHAPE and rope(tokens=2 ** 31) == SHAPE
    assert rope(io=2) == DTYPE
    for dim in (0, 4, 12, 264):
        assert rope(dim=dim) == SHAPE
    assert rope(hq=0) == SHAPE and rope(hk=-1) == SHAPE and rope(hq=1025) == SHAPE and rope(hk=1025) == SHAPE
    assert rope(r=None) == NULL and rope(q=None) == NULL and rope(qo=None) == NULL and rope(k=None) == NULL
    assert rope(ko=None) == NULL and rope(q=A._View(None, D, D)) == NULL
    assert rope(r=A._Rope(None, at(31), 32, 0, 1.0)) == NULL and rope(r=A._Rope(at(30), None, 32, 0, 1.0)) == NULL
    assert rope(r=rope_desc(pairs=0)) == SHAPE and rope(r=rope_desc(pairs=33)) == SHAPE
    assert rope(r=rope_desc(pairs=2 ** 31 - 1)) == SHAPE
    assert rope(r=rope_desc(inter=2)) == SHAPE and rope(r=rope_desc(ms=math.nan)) == SHAPE
    assert rope(r=rope_desc(pos=at(30, 4))) == ALIGN and rope(r=rope_desc(freq=at(31, 4))) == ALIGN
    assert rope(q=view(0, off=8)) == ALIGN and rope(q=view(0, ts=HQ * D + 4)) == ALIGN and rope(q=view(0, hs=D + 2)) == ALIGN
    assert rope(q=view(0, ts=-D)) == SHAPE and rope(q=view(0, ts=2 ** 23 + 8)) == SHAPE
    assert rope(q=view(0, hs=2 ** 48 + 8)) == SHAPE
    assert rope(qo=view(0, off=HQ * D * 2)) == ALIAS          # shifted by a token: overlaps q, not in place
    assert rope(qo=view(2, HQ)) == ALIAS                       # over k
    assert rope(ko=view(1, HK)) == ALIAS                       # over q_out
    assert rope(qo=view(1, ts=0)) == ALIAS                     # the outputs of tokens fall on each other
    assert rope(qo=view(1, hs=D - 8)) == ALIAS                 # heads fall on each other
    assert rope(qo=A._View(at(30), HQ * D, D)) == ALIAS        # over the positions
    assert rope(ko=A._View(at(31), HK * D, D)) == ALIAS        # over the frequencies


def write(tokens=T, io=L.SSM_BF16, c="", slots="", k="", v="", r=None, hq=0, q=None, qo=None, ko=None):
    pick = lambda x, d: d if x == "" else x  # noqa: E731
    return L.load().ssm_kv_write(tokens, io, pick(c, cache()), pick(slots, at(32)), pick(k, view(2, HK)),
                                 pick(v, view(3, HK)), r, hq, q, qo, ko, None)


def test_kv_write_validation():
    assert write(tokens=0) == OK
    assert write(tokens=-1) == SHAPE and write(tokens=2 ** 31) == SHAPE and write(io=5) == DTYPE
    assert write(c=None) == NULL and write(slots=None) == NULL and write(k=None) == NULL and write(v=None) == NULL
    for bad in (cache(k=0), cache(v=0), cache(ks=0), cache(vs=0)):
        assert write(c=bad) == NULL
    for bad in (cache(page=8), cache(page=48), cache(page=2048), cache(pages=0), cache(pages=2 ** 31), cache(heads=0),
                cache(dim=60), cache(dim=264)):
        assert write(c=bad) == SHAPE
    assert write(c=cache(kind=3)) == DTYPE and write(c=cache(kind=-1)) == DTYPE
    assert write(c=cache(k=at(20, 8))) == ALIGN and write(c=cache(ks=at(22, 4))) == ALIGN and write(slots=at(32, 4)) == ALIGN
    assert write(k=view(2, HK, off=2)) == ALIGN
    assert write(hq=HQ) == SHAPE and write(ko=view(4, HK)) == SHAPE and write(hq=-1) == SHAPE  # q, k_out need a rotation
    assert write(r=rope_desc(), hq=HQ) == NULL
    assert write(r=rope_desc(pairs=40)) == SHAPE
    assert write(c=cache(v=at(20, 16 * 64))) == ALIAS          # k and v pages overlap
    assert write(c=cache(ks=at(21))) == ALIAS
    assert write(slots=at(20)) == ALIAS and write(k=A._View(at(21), HK * D, D)) == ALIAS
    r = rope_desc()
    assert write(r=r, hq=HQ, q=view(0), qo=A._View(at(20), HQ * D, D)) == ALIAS
    assert write(r=r, hq=HQ, q=view(0), qo=A._View(at(3), HQ * D, D)) == ALIAS   # q_out over v
    assert write(r=r, hq=HQ, q=view(0), qo=A._View(at(2), HQ * D, D)) == ALIAS   # q_out over k
    assert write(r=r, ko=A._View(at(3), HK * D, D)) == ALIAS                     # k_out over v
    assert write(r=r, hq=HQ, q=view(0), qo=view(1), ko=A._View(at(0), HK * D, D)) == ALIAS
    assert write(r=r, hq=HQ, q=view(0), qo=view(1), ko=A._View(at(1), HK * D, D)) == ALIAS
    assert write(r=rope_desc(pos=at(20))) == ALIAS


def read(tokens=T, io=L.SSM_BF16, c="", slots="", k="", v=""):
    pick = lambda x, d: d if x == "" else x  # noqa: E731
    return L.load().ssm_kv_read(tokens, io, pick(c, cache()), pick(slots, at(32)), pick(k, view(2, HK)),
                                pick(v, view(3, HK)), None)


def test_kv_read_validation():
    assert read(tokens=0) == OK and read(tokens=-1) == SHAPE and read(io=-1) == DTYPE
    assert read(c=None) == NULL and read(slots=None) == NULL and read(k=None) == NULL and read(v=None) == NULL
    assert read(c=cache(page=100)) == SHAPE and read(slots=at(32, 1)) == ALIGN and read(v=view(3, HK, off=4)) == ALIGN
    assert read(v=view(2, HK)) == ALIAS and read(k=A._View(at(20), HK * D, D)) == ALIAS
    assert read(k=view(2, HK, ts=0)) == ALIAS and read(k=A._View(at(32), HK * D, D)) == ALIAS


def dims(b=B, tq=T, tk=T, hq=HQ, hk=HK, dim=D, io=L.SSM_BF16, causal=1, scale=0.125):
    return A._Dims(b, tq, tk, hq, hk, dim, io, causal, scale)


def prefill(d="", q="", k="", v="", cq="", ck="", out="", lse=None):
    pick = lambda x, y: y if x == "" else x  # noqa: E731
    return L.load().ssm_attn_prefill(pick(d, dims()), pick(q, view(0)), pick(k, view(2, HK)), pick(v, view(3, HK)),
                                     pick(cq, at(33)), pick(ck, at(34)), pick(out, view(1)), lse, None)


def test_attn_prefill_validation():
    assert prefill(d=dims(tq=0)) == OK
    assert prefill(d=None) == NULL and prefill(q=None) == NULL and prefill(k=None) == NULL and prefill(out=None) == NULL
    assert prefill(cq=None) == NULL and prefill(ck=None) == NULL
    for bad in (dims(b=0), dims(b=65536), dims(tq=-1), dims(tk=-1), dims(tk=2 ** 31), dims(hq=5), dims(hk=0), dims(hq=0),
                dims(dim=20), dims(dim=512), dims(causal=2), dims(scale=0.0), dims(scale=-1.0), dims(scale=math.inf),
                dims(scale=math.nan), dims(scale=3e38), dims(tq=2 ** 30 + 1)):
        assert prefill(d=bad) == SHAPE
    assert prefill(d=dims(io=3)) == DTYPE
    assert prefill(cq=at(33, 2)) == ALIGN and prefill(lse=at(35, 1)) == ALIGN and prefill(q=view(0, off=8)) == ALIGN
    assert prefill(out=view(0)) == ALIAS and prefill(out=A._View(at(3), HQ * D, D)) == ALIAS
    assert prefill(out=A._View(at(33), HQ * D, D)) == ALIAS and prefill(lse=at(1, 64)) == ALIAS
    assert prefill(lse=at(2)) == ALIAS and prefill(lse=at(34)) == ALIAS and prefill(lse=at(0)) == ALIAS
    assert prefill(out=view(1, ts=D)) == ALIAS


def decode(b=B, hq=HQ, io=L.SSM_BF16, scale=0.1, c="", q="", table="", width=W, lens="", out="", lse=None, ws="", n=1 << 30):
    pick = lambda x, y: y if x == "" else x  # noqa: E731
    return L.load().ssm_attn_decode_step(b, hq, io, scale, pick(c, cache()), pick(q, view(0)), pick(table, at(36)), width,
                                         pick(lens, at(37)), pick(out, view(1)), lse, pick(ws, at(38)), n, None)


def test_attn_decode_validation():
    lib = L.load()
    need = lib.ssm_attn_decode_workspace_bytes(B, HQ, cache(), W)
    assert need > 0 and need % 4 == 0
    for b, hq, c, w in ((0, HQ, cache(), W), (B, 5, cache(), W), (B, HQ, cache(page=12), W), (B, HQ, cache(), 0),
                        (B, HQ, cache(), 2 ** 40), (B, 0, cache(), W), (65536, HQ, cache(), W)):
        assert lib.ssm_attn_decode_workspace_bytes(b, hq, c, w) == 0
        assert decode(b=b, hq=hq, c=c, width=w) == SHAPE
    assert lib.ssm_attn_decode_workspace_bytes(B, HQ, None, W) == 0
    assert decode(c=None) == NULL and decode(q=None) == NULL and decode(table=None) == NULL and decode(lens=None) == NULL
    assert decode(out=None) == NULL and decode(io=9) == DTYPE and decode(c=cache(kind=7)) == DTYPE
    for s in (0.0, -0.5, math.nan, math.inf, 3e38):
        assert decode(scale=s) == SHAPE
    assert decode(ws=None) == WORKSPACE and decode(n=need - 1) == WORKSPACE and decode(ws=at(38, 4)) == ALIGN
    assert decode(table=at(36, 2)) == ALIGN and decode(lens=at(37, 1)) == ALIGN and decode(lse=at(39, 2)) == ALIGN
    assert decode(out=view(0)) == ALIAS and decode(out=A._View(at(20), HQ * D, D)) == ALIAS
    assert decode(out=A._View(at(36), HQ * D, D)) == ALIAS and decode(lse=at(1)) == ALIAS and decode(lse=at(37)) == ALIAS
    assert decode(ws=at(1)) == ALIAS and decode(ws=at(0)) == ALIAS and decode(ws=at(21)) == ALIAS and decode(lse=at(38)) == ALIAS


def test_binding_refuses_host_tensors():
    q = torch.zeros(4, 2, 16)
    pos, freq = torch.arange(4), A.rope_frequencies(16, device="cpu")[0]
    with pytest.raises(ValueError, match="GPU"):
        A.rope(q, None, pos, freq)
    with pytest.raises(ValueError):
        A.KVCache(torch.zeros(2, 1, 16, 8), torch.zeros(2, 1, 16, 8))
    with pytest.raises(TypeError):
        A.KVCache(torch.zeros(2, 1, 16, 8, dtype=torch.float16), torch.zeros(2, 1, 16, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        A.attn_prefill(q, q, q, torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(TypeError):
        A.attn_prefill(q.half(), q.half(), q.half(), torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError, match="tokens"):
        A.rope(q[0], None, pos, freq)


def test_rope_frequencies():
    f, m = A.rope_frequencies(8, base=100.0, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0
    assert torch.allclose(f, torch.tensor([100.0 ** (-i / 4) for i in range(4)], dtype=torch.float64))
    assert torch.allclose(A.rope_frequencies(8, base=100.0, scaling="linear", factor=4.0, device="cpu")[0], f / 4)
    n = A.rope_frequencies(8, base=100.0, scaling="ntk", factor=4.0, device="cpu")[0]
    assert n[0] == 1.0 and abs(float(n[-1]) - float(f[-1]) / 4) < 1e-12 and torch.all(n <= f)
    f, _ = A.rope_frequencies(64, device="cpu")
    y, m = A.rope_frequencies(64, scaling="yarn", factor=8.0, device="cpu")
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-12
    assert y[0] == f[0] and abs(float(y[-1] * 8 / f[-1]) - 1) < 1e-12 and torch.all(y <= f) and torch.all(y >= f / 8)
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=1.0), dict(rot_dim=8, factor=0.0),
                dict(rot_dim=8, scaling="cubic"), dict(rot_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            A.rope_frequencies(device="cpu", **bad)


def test_binding_refuses_cpu_tensors_with_an_index():
    q = torch.zeros(4, 2, 16, device="cpu:0")
    pos, freq = torch.arange(4, device="cpu:0"), A.rope_frequencies(16, device="cpu:0")[0]
    with pytest.raises(ValueError, match="GPU"):
        A.rope(q, None, pos, freq)
    k = torch.zeros(2, 1, 16, 8, device="cpu:0")
    with pytest.raises(ValueError, match="GPU"):
        A.KVCache(k, k)
    with pytest.raises(ValueError, match="required"):
        A.KVCache(k.to(torch.int8), k.to(torch.int8))


def test_packed_structures_are_the_declared_ones():
    """What the binding packs by hand has the layout of the structures."""
    buf = A._Buffer()
    A._cache_fields(buf, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9)
    c = A._Cache.from_buffer(buf)
    assert [getattr(c, n) for n, _ in A._Cache._fields_] == list(range(1, 10))
    A._views_rope(buf, 0, *range(12), 21, 22, 23, 1, 0.5)
    for i in range(4):
        v = A._View.from_buffer(buf, i * A._VIEW)
        assert (v.data or 0, v.token_stride, v.head_stride) == (3 * i, 3 * i + 1, 3 * i + 2)
    r = A._Rope.from_buffer(buf, 4 * A._VIEW)
    assert (r.positions, r.freq, r.pairs, r.interleaved, r.mscale) == (21, 22, 23, 1, 0.5)
    A._five_views_rope(buf, 0, *range(15), 21, 22, 23, 1, 0.5)
    r = A._Rope.from_buffer(buf, 5 * A._VIEW)
    assert (r.positions, r.freq, r.pairs, r.interleaved, r.mscale) == (21, 22, 23, 1, 0.5)
    A._four_views_dims(buf, 0, *range(12), 31, 32, 33, 34, 35, 36, 1, 0, 0.25)
    d = A._Dims.from_buffer(buf, 4 * A._VIEW)
    assert [getattr(d, n) for n, _ in A._Dims._fields_] == [31, 32, 33, 34, 35, 36, 1, 0, 0.25]
    A._two_views(buf, 0, *range(40, 46))
    v = A._View.from_buffer(buf, A._VIEW)
    assert (v.data, v.token_stride, v.head_stride) == (43, 44, 45)
