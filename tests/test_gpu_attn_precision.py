"""The precision of prompt and decode attention as a whole (tests/attn_precision.py), in every form of the kernels: the bound
is one that a lost part of an operand, a dropped step of keys or misplaced values exceed."""
import numpy as np
import pytest
import torch

import selective_state_space_causal_amd as ssm
from tests import attn_precision as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def on_gpu(x, io):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[io]).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, io, c, lse, what):
    name, factor = P.excess(f64(got), ref, P.HALF[io], c, None if lse is None else f64(lse))
    assert factor <= 1, f"{what}: {name} {factor:.2f} times the bound"


def prompt_case(lens, past, Hq, Hkv, D, io, seed):
    rng = np.random.default_rng(seed)
    lk = [max(a + b, 0) for a, b in zip(lens, past)]
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (lens, lk))
    kv = [P.keys_values(rng, n, (Hkv, D), io) for n in lk]
    k, v = (np.concatenate([x[i] for x in kv]) for i in range(2))
    return on_gpu(rng.standard_normal((cu_q[-1], Hq, D)), io), on_gpu(k, io), on_gpu(v, io), cu_q, cu_k


def check_prompt(lens, past, Hq, Hkv, D, causal, io, tokens=None):
    q, k, v, cu_q, cu_k = prompt_case(lens, past, Hq, Hkv, D, io, D + len(lens))
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = ssm.attn_prefill(q, k, v, torch.from_numpy(cu_q).to(DEV), torch.from_numpy(cu_k).to(DEV), causal=causal, lse=lse)
    ref = P.prompt(f64(q), f64(k), f64(v), cu_q, cu_k, causal, D ** -0.5, tokens)
    if tokens is not None:
        out, lse = out[tokens], lse[tokens]
    within(out, ref, io, P.C_F32 if io == "f32" else P.C_PROMPT, lse, f"{lens[:3]} {Hq} {Hkv} {D} {causal} {io}")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,past,Hq,Hkv,D", [
    ([271], [0], 4, 1, 64), ([1100], [0], 16, 2, 64), ([1, 90], [700, 2], 6, 3, 40), ([743, 0, 300], [0, 50, 100], 6, 2, 96),
    ([500], [300], 4, 2, 128), ([260, 33], [0, 900], 4, 2, 120), ([260], [0], 4, 1, 192), ([271], [0], 3, 3, 256), ([1, 1, 1], [999, 63, 0], 8, 2, 128)])
def test_fp32_prompts(lens, past, Hq, Hkv, D, causal):
    check_prompt(lens, past, Hq, Hkv, D, causal, "f32")


@pytest.mark.parametrize("lens,past,Hq,Hkv,D,causal", [
    # few rows, keys split over waves from memory
    ([271], [0], 4, 1, 64, True), ([300, 20], [0, 700], 8, 2, 128, True), ([90], [400], 4, 2, 192, False), ([271], [0], 4, 1, 256, True),
    # tiles of 64 rows, four shares of their keys (two past 192 channels)
    ([1000], [300], 24, 1, 64, True), ([600, 450], [0, 300], 16, 1, 80, True), ([500, 37], [600, 0], 24, 1, 128, True), ([900], [100], 16, 1, 256, True),
    # of 128 rows, two shares
    ([1000], [300], 40, 1, 64, True), ([700, 300], [0, 300], 40, 1, 96, True), ([500, 470], [600, 0], 40, 1, 128, True), ([900], [200], 40, 1, 192, True),
    # of 128 rows, one
    ([150] * 6, [0, 1, 70] * 2, 48, 1, 64, True), ([700], [0], 160, 1, 96, False), ([130] * 8, [0] * 8, 64, 1, 128, True),
    ([400], [0], 160, 1, 192, False), ([200] * 5, [0] * 5, 64, 1, 256, True)])
def test_bf16_prompts(lens, past, Hq, Hkv, D, causal):
    check_prompt(lens, past, Hq, Hkv, D, causal, "bf16")


@pytest.mark.parametrize("new,past,Hq,D", [(2000, 5000, 40, 64), (1700, 4500, 48, 128)])
def test_bf16_prompts_of_256_rows_to_a_tile(new, past, Hq, D):
    """Some tokens of a long sequence."""
    tokens = np.r_[0:6, 900:906, new - 6:new]
    check_prompt([new], [past], Hq, 1, D, True, "bf16", tokens)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (4, 2, 128), (4, 2, 256), (6, 3, 64), (6, 3, 96), (6, 3, 128), (6, 3, 192)])
def test_shared_keys_in_many_sequences(Hq, Hkv, D):
    """More than 64 sequences, whose tiles are found by a scan of them all, with keys that waves share (two key heads: four
    shares of 64 rows, two past 192 channels; three: two shares of 128): of all lengths, none, and fewer keys than queries."""
    rng = np.random.default_rng(Hkv * D)
    lens = [int(x) for x in rng.integers(0, 37, 70)]
    past = [int(x) for x in rng.choice([0, 300, 500, -10], 70, p=[0.1, 0.4, 0.4, 0.1])]
    lens[3], past[3], lens[69], past[69] = 0, 200, 36, 511
    keys, tiles = sum(max(a + b, 0) for a, b in zip(lens, past)), (sum(lens) * 2 // 128 + 70) * Hkv
    assert keys >= 256 * 70 and (128 < tiles <= 260 if Hkv == 2 else 260 < tiles <= 320)
    check_prompt(lens, past, Hq, Hkv, D, True, "bf16")


KIND = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def decode_case(lens, Hq, Hkv, D, page, kind, io, seed):
    """A cache in shuffled pages, its unwritten rows NaN; keys and values as cached, per sequence."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + 1, max(need) + 1
    c = ssm.KVCache.allocate(pages, page, Hkv, D, KIND.get(kind, DT[io]), DEV)
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x7F)
    for t in (c.k_scale, c.v_scale):
        if t is not None:
            t.fill_(float("nan"))
    order, table = rng.permutation(pages), np.full((len(lens), width), -1, np.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        j = np.arange(n)
        slots.append(table[b, j // page].astype(np.int64) * page + j % page)
    held = []
    for s in slots:
        if len(s):
            s = torch.from_numpy(s).to(DEV)
            k, v = (on_gpu(x, io) for x in P.keys_values(rng, len(s), (Hkv, D), io))
            ssm.kv_write(k, v, c, s)
        else:
            s = torch.empty(0, dtype=torch.int64, device=DEV)
        rows = []
        for x, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
            x = x.permute(0, 2, 1, 3).reshape(-1, Hkv, D)[s] if x.element_size() > 1 else \
                x.view(torch.uint8).permute(0, 2, 1, 3).reshape(-1, Hkv, D)[s].view(x.dtype)
            x = f64(x)
            rows.append(x if scale is None else x * f64(scale.permute(0, 2, 1).reshape(-1, Hkv)[s])[..., None])
        held.append(rows)
    q = on_gpu(rng.standard_normal((len(lens), Hq, D)), io)
    return c, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), q, held


def check_decode(lens, Hq, Hkv, D, page, kind, io):
    c, table, n, q, held = decode_case(lens, Hq, Hkv, D, page, kind, io, D + len(lens))
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = ssm.attn_decode_step(q, c, table, n, lse=lse)
    refs = [P.prompt(f64(q[b:b + 1]), k, v, [0, 1], [0, len(k)], False, D ** -0.5) for b, (k, v) in enumerate(held)]
    ref = tuple(np.concatenate(x) for x in zip(*refs))
    within(out, ref, io, P.C_F32 if io == "f32" else P.C_DECODE, lse, f"{lens} {Hq} {Hkv} {D} {kind} {io}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["int8", "e4m3", "io"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ([700, 90, 0], 4, 2, 64, 16), ([450, 33], 12, 2, 72, 32), ([500, 480], 16, 1, 128, 64), ([300, 512], 17, 1, 136, 16), ([511], 6, 2, 192, 16),
    ([200, 400], 8, 4, 256, 64)])
def test_decode(lens, Hq, Hkv, D, page, kind, io):
    check_decode(lens, Hq, Hkv, D, page, kind, io)


@pytest.mark.parametrize("io,kind", [("f32", "int8"), ("f32", "e4m3"), ("f32", "io"), ("bf16", "int8"), ("bf16", "e4m3"), ("bf16", "io")])
@pytest.mark.parametrize("D", [72, 128, 256])
def test_decode_in_many_chunks(D, kind, io):
    """Sequences in more than 64 chunks beside short ones."""
    check_decode([20011, 5, 0, 16640], 6, 2, D, 32, kind, io)
