"""A call on a residual stream that is refused has not touched the stream: the mixer layer and the attention block look at what their
later calls would refuse before the norm adds hidden to it.  Without a GPU: host tensors that say they are on one, and the norm
replaced by a mark that it was reached.  The same calls with nothing wrong reach it."""
import pytest
import torch

from selective_state_space_causal_amd import _lib, attn, attn_layer, block, layer

B, L, DM, D, R, N = 2, 8, 32, 16, 4, 16
F32, BF16 = torch.float32, torch.bfloat16


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda:0"))

    def get_device(self):
        return 0


class OnAnother(OnGpu):
    device = property(lambda self: torch.device("cuda:1"))

    def get_device(self):
        return 1


def gpu(*shape, dtype=F32, make=torch.zeros):
    return make(*shape, dtype=dtype).as_subclass(OnGpu)


class Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def without_a_gpu(monkeypatch):
    def empty(*shape, dtype=F32, device=None):
        return make(*shape, dtype=dtype).as_subclass(OnGpu)

    def block_input(*args, **kw):
        raise Reached

    make = torch.empty
    for module in (layer, attn_layer):
        monkeypatch.setattr(module, "block_input", block_input)
    monkeypatch.setattr(layer, "q4_dequantize", lambda w, out, stream: out)
    monkeypatch.setattr(torch, "empty", empty)


class Projector:
    handle = 1

    def __call__(self, *args, **kw):
        raise AssertionError("launched")


def four_bit(M, K):
    shapes = block._q4_shapes(M, K)
    return block.Q4Weight(*(gpu(*s, dtype=torch.uint8) for s in shapes), M, K)


def mixer(rows, io, q4):
    """The arguments of a mixer layer's calls, all in order."""
    w = {k: gpu(*s, dtype=io) for k, s in dict(in_x=(D, DM), in_z=(D, DM), in_xz=(2 * D, DM), out=(DM, D), x_all=(R + 2 * N, D), x_dt=(R, D),
                                              x_B=(N, D), x_C=(N, D), dt=(D, R)).items()}
    if q4:
        for k in ("in_x", "in_z", "in_xz", "out"):
            w[k] = four_bit(*w[k].shape)
    p = {k: gpu(*s) for k, s in dict(A=(D, N), Dskip=(D,), dt_bias=(D,), conv_w=(D, 4), conv_b=(D,)).items()}
    return dict(w=w, p=p, proj=Projector(), h=gpu(rows, D, N), conv=gpu(rows, D, 3), bufs=None)


def call(a, rows, io, decode, fused=True):
    hidden = gpu(rows, *(() if decode else (L,)), DM, dtype=io)
    kw = dict(norm=gpu(DM), residual=gpu(*hidden.shape))
    if decode:
        return layer.mixer_decode_step(hidden, a["w"], a["p"], a["proj"], a["h"], a["conv"], fused=fused, bufs=a["bufs"], **kw)
    return layer.mixer_prefill(hidden, a["w"], a["p"], a["proj"], **kw)


FORMS = [(rows, io, q4, decode, fused) for rows in (1, 2) for io in (F32, BF16) for q4 in (False, True)
         for decode, fused in ((False, False), (True, False), (True, True))]


@pytest.mark.parametrize("rows,io,q4,decode,fused", FORMS)
def test_a_mixer_call_in_order_reaches_the_norm(rows, io, q4, decode, fused):
    a = mixer(rows, io, q4)
    with pytest.raises(Reached):
        call(a, rows, io, decode, fused)
    if not decode and not fused:
        del a["w"]["x_all"]  # the three parts do
        with pytest.raises(Reached):
            call(a, rows, io, decode)


def moved(t):
    """One value further on: the same tensor at an address that is not a multiple of 16 bytes."""
    return torch.zeros(t.numel() + 1, dtype=t.dtype)[1:].view(t.shape).as_subclass(OnGpu)


def strided(t):
    return torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2].as_subclass(OnGpu)


SPOILS = {
    "missing": lambda t: None,
    "wider": lambda t: gpu(*t.shape[:-1], t.shape[-1] + 16, dtype=t.dtype),
    "taller": lambda t: gpu(t.shape[0] + 1, *t.shape[1:], dtype=t.dtype),
    "type": lambda t: t.to(torch.float16).as_subclass(OnGpu),
    "device": lambda t: t.as_subclass(OnAnother),
    "host": lambda t: t.as_subclass(torch.Tensor),
    "strided": strided,
    "moved": moved,
}


def used(rows, q4, decode, fused, io):
    """Names of the weights that a call reads as tensors."""
    stacked = rows == 1
    names = [] if q4 else ["in_xz", "out"] if stacked else ["in_x", "in_z", "out"]
    if decode and fused or decode and rows == 1 or not decode and io == BF16:
        names.append("x_all")
    else:
        names += ["x_dt", "x_B", "x_C"]
    return names + ["dt"]


@pytest.mark.parametrize("how", sorted(SPOILS))
@pytest.mark.parametrize("rows,io,q4,decode,fused", FORMS)
def test_a_mixer_s_weights_are_looked_at_before_the_norm(rows, io, q4, decode, fused, how):
    for k in used(rows, q4, decode, fused, io):
        if how == "moved" and decode and fused and k in ("x_all", "dt"):
            continue  # taken at any address
        if how in ("missing", "taller") and k in ("in_x", "x_dt") or how == "host" and k == "in_x":
            continue  # decides the sizes of all
        a = mixer(rows, io, q4)
        a["w"][k] = SPOILS[how](a["w"][k])
        if a["w"][k] is None:
            del a["w"][k]
            if k == "in_xz" or k == "x_all" and not (decode and fused):
                continue  # then its parts are read
        with pytest.raises((ValueError, TypeError, KeyError)):
            call(a, rows, io, decode, fused)


@pytest.mark.parametrize("rows,io,q4,decode,fused", [f for f in FORMS if f[2]])
def test_a_mixer_s_4_bit_weights_are_looked_at_before_the_norm(rows, io, q4, decode, fused):
    for k in ["in_xz", "out"] if rows == 1 else ["in_x", "in_z", "out"]:
        M, K = mixer(rows, io, True)["w"][k].shape
        for bad in (four_bit(M, K + 16), four_bit(M + 16, K), four_bit(M, K)._replace(codes=gpu(1, 1, 64, 8, dtype=torch.uint8)),
                    four_bit(M, K)._replace(scales=gpu(1, 1, 64, 4)), gpu(M, K, dtype=torch.float16)):
            if k == "in_x" and bad.shape[0] != M:
                continue  # decides the sizes of all
            a = mixer(rows, io, True)
            a["w"][k] = bad
            if not decode and isinstance(bad, block.Q4Weight) and tuple(bad.shape) == (M, K):
                continue  # read back before the norm, by a call that looks at it
            with pytest.raises((ValueError, TypeError)):
                call(a, rows, io, decode, fused)


@pytest.mark.parametrize("how", sorted(SPOILS))
@pytest.mark.parametrize("rows,io,q4,decode,fused", FORMS)
def test_a_mixer_s_parameters_and_state_are_looked_at_before_the_norm(rows, io, q4, decode, fused, how):
    for k in ("A", "Dskip", "dt_bias", "conv_w", "conv_b"):
        if how == "moved" and k not in ("A", "conv_w") or how == "missing" and k == "conv_b":
            continue
        a = mixer(rows, io, q4)
        a["p"][k] = SPOILS[how](a["p"][k])
        if a["p"][k] is None:
            del a["p"][k]
        with pytest.raises((ValueError, TypeError, KeyError)):
            call(a, rows, io, decode, fused)
    for k in ("h", "conv") if decode else ():
        if how == "moved" and k == "conv":
            continue
        a = mixer(rows, io, q4)
        a[k] = SPOILS[how](a[k])
        with pytest.raises((ValueError, TypeError)):
            call(a, rows, io, decode, fused)


@pytest.mark.parametrize("how", ["missing", "wider", "type", "device", "strided"])
@pytest.mark.parametrize("rows,io,q4,decode,fused", [f for f in FORMS if f[3]])
def test_a_decode_step_s_buffers_are_looked_at_before_the_norm(rows, io, q4, decode, fused, how):
    a = mixer(rows, io, q4)
    hidden = gpu(rows, DM, dtype=io)
    names = set(layer.alloc_decode_buffers(hidden, a["w"], N, fused, normed=True)) - {"normed", "xo"}
    assert {"x", "z", "y", "out"} < names
    for k in names:
        a["bufs"] = layer.alloc_decode_buffers(hidden, a["w"], N, fused, normed=True)
        if k == "ws" and how in ("wider", "type"):
            a["bufs"][k] = a["bufs"][k][:-1]  # any type of enough bytes does
        elif how == "missing" and k == "xz":
            continue  # then x and z are written on their own
        else:
            a["bufs"][k] = SPOILS[how](a["bufs"][k])
        if a["bufs"][k] is None:
            del a["bufs"][k]
        with pytest.raises((ValueError, TypeError, KeyError)):
            call(a, rows, io, True, fused)


@pytest.mark.parametrize("decode,fused", [(False, False), (True, False), (True, True)])
def test_other_things_that_a_mixer_refuses(decode, fused):
    def refused(a):
        with pytest.raises((ValueError, TypeError, AttributeError)):
            call(a, 2, BF16, decode, fused)
    for proj in (None, type("Closed", (), {"handle": None})()):
        refused(dict(mixer(2, BF16, False), proj=proj))
    if decode and fused:  # d_state 16 only
        a = mixer(2, BF16, False)
        a["p"]["A"], a["h"] = gpu(D, 8), gpu(2, D, 8)
        a["w"]["x_all"] = gpu(R + 16, D, dtype=BF16)
        refused(a)
        with pytest.raises(Reached):  # and no projector where nothing is left to project
            call(dict(mixer(2, BF16, True), proj=None), 2, BF16, True, True)


# ---------------------------------------------------------------- the attention block

HQ, HKV, HD, PAGE, T = 4, 2, 16, 16, 6


class Cache:
    """What an attention block knows of a cache."""
    kv_heads, head_dim, page_size, pages, device = HKV, HD, PAGE, 8, torch.device("cuda:0")
    io_only, k = None, None
    check_io = attn.KVCache.check_io

    def _sizes(self):
        return self.pages, self.page_size, self.kv_heads, self.head_dim


def attention(decode, q4):
    w = {"qkv": gpu((HQ + 2 * HKV) * HD, DM), "out": gpu(DM, HQ * HD)}
    if q4:
        w = {k: four_bit(*v.shape) for k, v in w.items()}
    a = dict(hidden=gpu(T, DM), w=w, heads=HQ, cache=Cache(), freq=gpu(HD // 2, dtype=torch.float64), mscale=1.0)
    if decode:
        a.update(table=gpu(T, 3, dtype=torch.int32), lens=gpu(T, dtype=torch.int32), workspace=None)
    else:
        a.update(slots=gpu(T, dtype=torch.int64), positions=gpu(T, dtype=torch.int64), cu_q=gpu(3, dtype=torch.int32), context_slots=None,
                 cu_k=None)
    return a


def attend(a, decode):
    kw = dict(norm=gpu(DM), residual=gpu(T, DM), mscale=a["mscale"])
    if decode:
        return attn_layer.attn_block_decode(a["hidden"], a["w"], a["heads"], a["cache"], a["table"], a["lens"], a["freq"],
                                            workspace=a["workspace"], **kw)
    return attn_layer.attn_block_prefill(a["hidden"], a["w"], a["heads"], a["cache"], a["slots"], a["cu_q"], a["positions"], a["freq"],
                                         context_slots=a["context_slots"], cu_k=a["cu_k"], **kw)


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("q4", [False, True])
def test_an_attention_call_in_order_reaches_the_norm(decode, q4):
    a = attention(decode, q4)
    with pytest.raises(Reached):
        attend(a, decode)
    if not decode:
        a.update(context_slots=gpu(11, dtype=torch.int64), cu_k=gpu(3, dtype=torch.int32))
    else:
        a["workspace"] = torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(OnGpu)
    with pytest.raises(Reached):
        attend(a, decode)


@pytest.mark.parametrize("how", ["wider", "taller", "type", "device", "host", "strided"])
@pytest.mark.parametrize("decode", [False, True])
def test_an_attention_block_s_tensors_are_looked_at_before_the_norm(decode, how):
    names = ("table", "lens", "freq") if decode else ("slots", "positions", "cu_q", "freq", "context_slots", "cu_k")
    for k in (*names, "qkv", "out"):
        a = attention(decode, False)
        if not decode:
            a.update(context_slots=gpu(11, dtype=torch.int64), cu_k=gpu(3, dtype=torch.int32))
        at = a["w"] if k in ("qkv", "out") else a
        if how in ("wider", "taller") and k == "context_slots" or (how, k) in (("wider", "table"), ("taller", "out")):
            continue  # as many as there are
        if how == "strided" and k in ("qkv", "out"):
            continue  # a plain product takes it
        at[k] = SPOILS[how](at[k])
        if how == "wider" and k == "freq":
            assert at[k].numel() > HD // 2
        with pytest.raises((ValueError, TypeError)):
            attend(a, decode)


def changed(**kw):
    return type("Changed", (Cache,), kw)()


@pytest.mark.parametrize("decode", [False, True])
def test_other_things_that_an_attention_block_refuses(decode):
    class OfBf16(Cache):
        io_only, k = BF16, torch.zeros(1, dtype=BF16)
    bad = [dict(cache=OfBf16()), dict(cache=changed(device=torch.device("cuda:1"))), dict(cache=changed(page_size=24)),
           dict(cache=changed(pages=0)), dict(mscale=float("nan")), dict(w={"qkv": attention(decode, False)["w"]["qkv"]}),
           dict(heads=3, w={"qkv": gpu(7 * HD, DM), "out": gpu(DM, 3 * HD)}),
           dict(w=dict(attention(decode, True)["w"], out=four_bit(DM, HQ * HD + 16))),
           dict(w=dict(attention(decode, True)["w"], qkv=four_bit((HQ + 2 * HKV) * HD, DM)._replace(codes=gpu(1, 1, 64, 16, dtype=torch.uint8)))),
           dict(freq=gpu(0, dtype=torch.float64))]
    if decode:
        bad += [dict(table=gpu(T, 0, dtype=torch.int32)), dict(workspace=torch.zeros(4, dtype=torch.uint8).as_subclass(OnAnother))]
    else:
        bad += [dict(cu_q=gpu(1, dtype=torch.int32)), dict(cu_q=gpu(3, 1, dtype=torch.int32))]
    for b in bad:
        with pytest.raises((ValueError, TypeError, KeyError)):
            attend(dict(attention(decode, False), **b), decode)


def test_nothing_is_looked_at_twice_without_a_residual_stream():
    """Without a stream to keep, the calls look at their own arguments as before."""
    a = mixer(2, BF16, False)
    a["w"]["out"] = None
    with pytest.raises(Reached):
        layer.mixer_decode_step(gpu(2, DM, dtype=BF16), a["w"], a["p"], a["proj"], a["h"], a["conv"], norm=gpu(DM))
