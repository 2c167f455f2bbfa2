"""The plain forms of the paged append, the 4-bit cache and the sampling
controls, pinned to what they must satisfy; and the refusals of the calls
(nothing here needs a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import _serving_ref as ref
from speculative_decoding_verification_sv_gb300 import binding as sv


def test_rounding_is_half_a_step():
    r = np.random.default_rng(0)
    x = r.standard_normal((50, 128)) * np.exp(3 * r.standard_normal((50, 1)))
    x = ref.bf16_round(x)
    c, s = ref.quantise(x)
    assert c.min() >= 1 and c.max() <= 15
    assert np.all(np.abs((c - 8) * s[..., None] - x.reshape(50, 4, 32)) <= s[..., None] / 2)
    assert np.all(np.abs(x.reshape(50, 4, 32)).max(-1) <= 7 * s)
    # the values and 136 s are exactly bf16
    assert np.array_equal(ref.bf16_round((c - 8) * s[..., None]), (c - 8) * s[..., None])
    assert np.array_equal(ref.bf16_round(136 * s), 136 * s)


@pytest.mark.parametrize("is_v", [False, True])
def test_block_layout_round_trip(is_v):
    r = np.random.default_rng(1)
    blk = np.zeros(ref.Q4, np.uint8)
    rows = ref.bf16_round(r.standard_normal((ref.PAGE, 128)))
    for p in range(ref.PAGE):
        ref.put_row(blk, p, rows[p], is_v)
    c, s = ref.quantise(rows)
    assert np.array_equal(ref.get_rows(blk, is_v), ((c - 8) * s[..., None]).reshape(ref.PAGE, 128))
    # one position written again leaves the others as they are
    before = ref.get_rows(blk, is_v)
    ref.put_row(blk, 13, rows[0], is_v)
    after = ref.get_rows(blk, is_v)
    assert np.array_equal(np.delete(after, 13, 0), np.delete(before, 13, 0))
    assert np.array_equal(after[13], before[0])


def test_rotation_keeps_pair_lengths_and_relative_angles():
    r = np.random.default_rng(2)
    rope = ref.rope_table(200, 128)
    x, y = ref.bf16_round(r.standard_normal((2, 1, 128)))
    for inter in (False, True):
        a = [float(ref.rotate(x, p, rope, inter)[0] @ ref.rotate(y, p + 7, rope, inter)[0]) for p in (0, 40, 180)]
        # each of the 128 products' two factors is rounded to bf16 (2^-8)
        tol = 2 * 2.0 ** -8 * 2 * float(np.abs(x[0]) @ np.abs(y[0])) + 1e-3
        assert max(a) - min(a) <= 2 * tol


def test_penalties_by_hand():
    x = np.array([[[2.0, -1.0, 0.5, 3.0], [2.0, -1.0, 0.5, 3.0]]], np.float32)
    y = ref.logits(x, tok=np.array([[1, 2]]), hist=np.array([[3, 0, 0, 9]]), hist_len=np.array([3]), prompt_len=np.array([1]),
                   repetition=[2.0], frequency=[0.25], presence=[0.5], bias=[{2: 10.0}])
    # row 0: 0 twice generated, 3 in the prompt, 1 the pending token
    assert y[0, 0].tolist() == [1.0 - 0.5 - 0.5, -2.0 - 0.25 - 0.5, 10.5, 1.5]
    # row 1: also the draft 2
    assert y[0, 1].tolist() == [0.0, -2.75, 0.25 - 0.25 - 0.5 + 10.0, 1.5]
    keys = ref.argmax_keys(y.reshape(2, 4))
    assert (~keys[:, 0] & 0xFFFFFFFF).tolist() == [2, 2]


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

F = ctypes.c_void_p(0x10000)     # never dereferenced
ODD = ctypes.c_void_p(0x10004)
ARG, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4


def _append(q4=False, **kw):
    a = dict(k=F, v=F, ks=256, vs=256, N=4, off=F, B=2, H=2, D=128, rope=F, pos=64, rot=128, kp=F, vp=F, np=8, tab=F, mp=4, ln=F,
             flags=0)
    a.update(kw)
    mid = [a["H"]] if q4 else [a["H"], a["D"]]
    f = sv.lib.sv_kv_append_q4 if q4 else sv.lib.sv_kv_append_paged
    return f(a["k"], a["v"], a["ks"], a["vs"], a["N"], a["off"], a["B"], *mid, a["rope"], a["pos"], a["rot"], a["kp"], a["vp"],
             a["np"], a["tab"], a["mp"], a["ln"], a["flags"], None)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw,want", [
    ({"N": 0, "k": None}, 0), ({"N": -1}, SHAPE), ({"k": None}, ARG), ({"v": ODD}, ARG), ({"off": None}, ARG), ({"ln": None}, ARG),
    ({"tab": None}, ARG), ({"kp": ODD}, ARG), ({"ks": 248}, SHAPE), ({"vs": 260}, SHAPE), ({"B": 0}, SHAPE), ({"H": 0}, SHAPE),
    ({"np": 0}, SHAPE), ({"mp": 0}, SHAPE), ({"mp": 2 ** 26}, SHAPE), ({"rope": ODD}, ARG), ({"rot": 24}, SHAPE), ({"rot": 144}, SHAPE),
    ({"rot": 0}, SHAPE), ({"pos": 0}, SHAPE), ({"flags": 2}, ARG)])
def test_append_refusals(q4, kw, want):
    assert _append(q4, **kw) == want


def test_append_head_dim_refusals():
    assert _append(D=12) == SHAPE and _append(D=2048, ks=4096, vs=4096) == SHAPE


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("B", [2 ** 30 + 1, 2 ** 31 - 1])
def test_append_refuses_sequences_past_its_search(q4, B):
    assert _append(q4, B=B) == SHAPE


@pytest.mark.parametrize("at,val,want", [
    (0, None, ARG), (1, ODD, ARG), (2, 0, SHAPE), (3, None, ARG), (4, 0, SHAPE), (5, ODD, ARG), (7, 0, SHAPE), (8, 0, SHAPE),
    (9, 0, SHAPE), (10, 129, SHAPE), (10, 0, SHAPE), (11, None, ARG), (13, None, ARG), (4, 2 ** 26, SHAPE)])
def test_commit_q4_refusals(at, val, want):
    a = [F, F, 8, F, 4, F, F, 2, 2, 2, 5, F, F, F, None]
    a[at] = val
    assert sv.lib.sv_kv_commit_q4(*a) == want


@pytest.mark.parametrize("at,val,want", [
    (10, 0, 0), (10, -1, SHAPE), (0, None, ARG), (1, ODD, ARG), (2, 0, SHAPE), (3, None, ARG), (4, 0, SHAPE), (5, 0, SHAPE), (6, 0, SHAPE),
    (7, 0, SHAPE), (8, None, ARG), (9, None, ARG), (11, ODD, ARG), (12, None, ARG), (10, 2 ** 30 + 1, SHAPE)])
def test_gather_q4_refusals(at, val, want):
    a = [F, F, 8, F, 4, 2, 2, 2, F, F, 16, F, F, None]
    a[at] = val
    assert sv.lib.sv_kv_gather_q4(*a) == want


@pytest.mark.parametrize("shape,kw,want", [
    ((1, 5, 12, 2, 64, 256), {}, UNSUPPORTED), ((1, 5, 12, 5, 128, 256), {}, SHAPE), ((1, 129, 12, 2, 128, 256), {}, SHAPE),
    ((1, 5, 12, 2, 128, 320), {}, SHAPE), ((1, 5, 12, 2, 128, 256), {"np": 0}, SHAPE), ((1, 5, 12, 2, 128, 256), {"q": None}, ARG),
    ((1, 5, 12, 2, 128, 256), {"kp": ODD}, ARG), ((1, 5, 12, 2, 128, 256), {"tab": None}, ARG),
    ((1, 5, 12, 2, 128, 256), {"scale": 0.0}, ARG), ((1, 5, 12, 2, 128, 256), {"scale": float("nan")}, ARG),
    ((1, 5, 12, 2, 128, 256), {"flags": 2}, ARG), ((1, 5, 12, 2, 128, 256), {"out": None}, ARG)])
def test_attn_q4_refusals(shape, kw, want):
    a = dict(q=F, kp=F, np=8, tab=F, scale=0.1, out=F, flags=0)
    a.update(kw)
    s = sv._AttnShape(*shape)
    assert sv.lib.sv_verify_attn_q4(ctypes.byref(s), a["q"], a["kp"], F, a["np"], a["tab"], 4, F, F, F, None, a["scale"], a["out"], F,
                                    1 << 30, a["flags"], None) == want


def _logits(**kw):
    a = dict(x=F, B=1, R=5, V=1000, hist=F, cap=64, hl=F, pl=F, tok=F, par=None, off=None, bt=None, bv=None, nb=0, mask=None, mv=-1e30,
             out=ctypes.c_void_p(0x1000000), key=None, kb=0)
    a.update(kw)
    return sv.lib.sv_logits_process(a["x"], a["B"], a["R"], a["V"], a["hist"], a["cap"], a["hl"], a["pl"], a["tok"], a["par"], None, None,
                                    None, a["off"], a["bt"], a["bv"], a["nb"], a["mask"], a["mv"], a["out"], a["key"], a["kb"], None)


@pytest.mark.parametrize("kw,want", [
    ({"x": None}, ARG), ({"x": ODD}, ARG), ({"out": None}, ARG), ({"B": 0}, SHAPE), ({"R": 0}, SHAPE), ({"R": 129}, SHAPE),
    ({"V": 0}, SHAPE), ({"B": 65536}, SHAPE), ({"hl": None}, ARG), ({"hist": ODD}, ARG), ({"cap": 0}, SHAPE), ({"tok": None, "par": F}, ARG),
    ({"off": F, "nb": -1}, SHAPE), ({"off": F, "nb": 3}, ARG), ({"mv": float("nan")}, ARG), ({"key": F, "kb": 5 * 8 * 8 - 1}, WORKSPACE),
    ({"out": ctypes.c_void_p(0x10010)}, ARG)])
def test_logits_refusals(kw, want):
    assert _logits(**kw) == want


@pytest.mark.parametrize("kw", [{"off": F, "bt": F, "bv": F, "nb": n} for n in (2 ** 30 + 1, 2 ** 31 - 1)] + [{"cap": 2 ** 28 + 1}])
def test_logits_refuses_more_entries_than_it_can_walk(kw):
    assert _logits(**kw) == SHAPE


def test_binding_refuses_host_tensors_and_wrong_shapes():
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, d=bf: torch.zeros(*s, dtype=d)  # noqa: E731
    with pytest.raises(ValueError):
        sv.kv_append_paged(z(4, 2, 128), z(4, 2, 128), z(3, d=i32), z(8, 2, 64, 128), z(8, 2, 64, 128), z(2, 4, d=i32), z(2, d=i32))
    with pytest.raises(ValueError):
        sv.kv_append_q4(z(4, 2, 64), z(4, 2, 64), z(3, d=i32), z(8, 2, 4608, d=torch.uint8), z(8, 2, 4608, d=torch.uint8),
                        z(2, 4, d=i32), z(2, d=i32))
    with pytest.raises(ValueError):
        sv.kv_commit_q4(z(1, 8, 2, 4608), z(1, 8, 2, 4608), z(2, 4, d=i32), z(1, 2, 2, 5, 128), z(1, 2, 2, 5, 128), z(2, 5, d=i32),
                        z(2, d=i32), z(2, d=i32))
    with pytest.raises(ValueError):
        sv.kv_gather_q4(z(8, 2, 4608), z(8, 2, 4608), z(2, 4, d=i32), z(2, d=i32), z(2, d=i32), 5)
    with pytest.raises(ValueError):
        sv.verify_attn_q4(z(2, 5, 12, 128), z(8, 2, 4608), z(8, 2, 4608), z(2, 4, d=i32), z(2, d=i32), z(2, 2, 5, 128), z(2, 2, 5, 128))
    with pytest.raises(ValueError):
        sv.logits_process(z(2, 100, d=torch.float32))
    with pytest.raises(ValueError):
        sv.logits_process(z(1, 2, 100, d=torch.float32))
