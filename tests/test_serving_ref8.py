"""The plain forms of the 8-bit cache's calls, pinned to what they must satisfy; and
the refusals of the calls (nothing here needs a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import _serving_ref as ref
import _serving_ref8 as ref8
from speculative_decoding_verification_sv_gb300 import binding as sv


def test_codes_are_torchs():
    r = np.random.default_rng(0)
    x = np.concatenate([r.standard_normal(4000) * np.exp(4 * r.standard_normal(4000)), ref8.E4M3[:127], ref8.E4M3[:126] + np.diff(ref8.E4M3[:127]) / 2,
                        [0.0, -0.0, np.nan]]).clip(-448, 448)
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = ref8.encode(x.astype(np.float32))
    assert np.array_equal(got & 127, want & 127) and np.array_equal(got[:-1], want[:-1])


@pytest.mark.parametrize("amax,e", [(0.0, -120), (448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0), (2.0 ** -133, -120), (255 * 2.0 ** 120, 119)])
def test_scale_is_the_least_that_holds(amax, e):
    assert ref8.exponent(amax) == e


def test_rounding_is_half_a_step():
    r = np.random.default_rng(1)
    blk = np.zeros(ref8.Q8, np.uint8)
    rows = ref.bf16_round(r.standard_normal((16, 128)) * np.exp(2 * r.standard_normal((16, 1))))
    ref8.put_rows(blk, 16, rows, True)
    s, got = ref8.scales(blk)[1], ref8.get_rows(blk, True)[16:32]
    assert 224 * s < np.abs(rows).max() <= 448 * s
    assert np.all(np.abs(got - rows) <= np.maximum(2.0 ** -4 * np.abs(rows), 2.0 ** -10 * s))
    assert np.array_equal(ref.bf16_round(got), got)      # exactly bf16


@pytest.mark.parametrize("is_v", [False, True])
def test_block_layout_and_growth(is_v):
    r = np.random.default_rng(2)
    blk = np.zeros(ref8.Q8, np.uint8)
    rows = ref.bf16_round(r.standard_normal((ref8.PAGE, 128)))
    for p in range(0, 64, 16):
        ref8.put_rows(blk, p, rows[p:p + 16], is_v)
    before = ref8.get_rows(blk, is_v)
    # a row of the third run 2^7 times as large: the run's earlier rows lose what its steps
    # cannot hold, the other runs nothing
    ref8.put_rows(blk, 40, 128 * rows[40:41], is_v)
    after = ref8.get_rows(blk, is_v)
    s = ref8.scales(blk)[2]
    assert np.array_equal(after[:32], before[:32]) and np.array_equal(after[48:], before[48:])
    assert np.all(np.abs(after[32:40] - before[32:40]) <= np.maximum(0, 2.0 ** -10 * s))
    assert np.all(np.abs(after[40] - 128 * rows[40]) <= np.maximum(2.0 ** -4 * np.abs(128 * rows[40]), 2.0 ** -10 * s))
    # the run's first position written again: its own scale
    ref8.put_rows(blk, 32, rows[:1] * 2.0 ** -10, is_v)
    assert ref8.scales(blk)[2] < 2.0 ** -14


def test_row_that_is_not_finite_is_nan():
    blk = np.zeros(ref8.Q8, np.uint8)
    rows = np.ones((3, 128))
    rows[1, 5] = np.inf
    ref8.put_rows(blk, 0, rows, False)
    got = ref8.get_rows(blk, False)
    assert np.isnan(got[1]).all() and np.array_equal(got[[0, 2]], np.ones((2, 128)))


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

F = ctypes.c_void_p(0x10000)     # never dereferenced
ODD = ctypes.c_void_p(0x10004)
ARG, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4


@pytest.mark.parametrize("kw,want", [
    ({"N": 0, "k": None}, 0), ({"N": -1}, SHAPE), ({"k": None}, ARG), ({"v": ODD}, ARG), ({"off": None}, ARG), ({"ln": None}, ARG),
    ({"tab": None}, ARG), ({"kp": ODD}, ARG), ({"vp": None}, ARG), ({"ks": 248}, SHAPE), ({"vs": 260}, SHAPE), ({"B": 0}, SHAPE),
    ({"H": 0}, SHAPE), ({"np": 0}, SHAPE), ({"mp": 0}, SHAPE), ({"mp": 2 ** 26}, SHAPE), ({"rope": ODD}, ARG), ({"rot": 24}, SHAPE),
    ({"rot": 144}, SHAPE), ({"rot": 0}, SHAPE), ({"pos": 0}, SHAPE), ({"flags": 2}, ARG), ({"B": 2 ** 30 + 1}, SHAPE),
    ({"B": 2 ** 29}, SHAPE)])
def test_append_refusals(kw, want):
    a = dict(k=F, v=F, ks=256, vs=256, N=4, off=F, B=2, H=2, rope=F, pos=64, rot=128, kp=F, vp=F, np=8, tab=F, mp=4, ln=F, flags=0)
    a.update(kw)
    assert sv.lib.sv_kv_append_q8(a["k"], a["v"], a["ks"], a["vs"], a["N"], a["off"], a["B"], a["H"], a["rope"], a["pos"], a["rot"],
                                  a["kp"], a["vp"], a["np"], a["tab"], a["mp"], a["ln"], a["flags"], None) == want


@pytest.mark.parametrize("at,val,want", [
    (0, None, ARG), (1, ODD, ARG), (2, 0, SHAPE), (3, None, ARG), (4, 0, SHAPE), (5, ODD, ARG), (7, 0, SHAPE), (8, 0, SHAPE),
    (9, 0, SHAPE), (10, 129, SHAPE), (10, 0, SHAPE), (11, None, ARG), (13, None, ARG), (4, 2 ** 26, SHAPE), (8, 2 ** 29, SHAPE)])
def test_commit_refusals(at, val, want):
    a = [F, F, 8, F, 4, F, F, 2, 2, 2, 5, F, F, F, None]
    a[at] = val
    assert sv.lib.sv_kv_commit_q8(*a) == want


@pytest.mark.parametrize("at,val,want", [
    (10, 0, 0), (10, -1, SHAPE), (0, None, ARG), (1, ODD, ARG), (2, 0, SHAPE), (3, None, ARG), (4, 0, SHAPE), (5, 0, SHAPE), (6, 0, SHAPE),
    (7, 0, SHAPE), (8, None, ARG), (9, None, ARG), (11, ODD, ARG), (12, None, ARG), (10, 2 ** 30 + 1, SHAPE)])
def test_gather_refusals(at, val, want):
    a = [F, F, 8, F, 4, 2, 2, 2, F, F, 16, F, F, None]
    a[at] = val
    assert sv.lib.sv_kv_gather_q8(*a) == want


@pytest.mark.parametrize("shape,kw,want", [
    ((1, 5, 12, 2, 64, 256), {}, UNSUPPORTED), ((0, 5, 12, 2, 128, 256), {}, SHAPE), ((1, 129, 12, 2, 128, 256), {}, SHAPE),
    ((1, 5, 12, 5, 128, 256), {}, SHAPE), ((1, 5, 34, 2, 128, 256), {}, None), ((1, 5, 12, 2, 128, 255), {}, SHAPE),
    ((1, 5, 12, 2, 128, 256), {"scale": 0.0}, ARG), ((1, 5, 12, 2, 128, 256), {"scale": float("nan")}, ARG),
    ((1, 5, 12, 2, 128, 256), {"flags": 2}, ARG), ((1, 5, 12, 2, 128, 256), {"q": None}, ARG),
    ((1, 5, 12, 2, 128, 256), {"k_pool": ODD}, ARG), ((1, 5, 12, 2, 128, 256), {"num_pages": 0}, SHAPE)])
def test_attn_refusals(shape, kw, want):
    s = sv._AttnShape(*shape)
    a = dict(q=F, k_pool=F, v_pool=F, num_pages=8, table=F, mp=4, ln=F, kb=F, vb=F, parent=None, scale=0.1, out=F, ws=F, bytes=0, flags=0)
    a.update(kw)
    got = sv.lib.sv_verify_attn_q8(ctypes.byref(s), a["q"], a["k_pool"], a["v_pool"], a["num_pages"], a["table"], a["mp"], a["ln"],
                                   a["kb"], a["vb"], a["parent"], a["scale"], a["out"], a["ws"], a["bytes"], a["flags"], None)
    assert got == want if want is not None else got != 0
    assert sv.verify_attn_q8_workspace(1, 5, 12, 2, 64, 256) == 0
