"""sv_logits_process: bit equality with the plain fp32 form, agreement with
float64, the argmax keys, and what it reports."""
import numpy as np
import pytest
import torch

import _serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_sv_gb300 import binding
    return binding


def dev(x, dtype=None):
    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def tree(r, B, R):
    p = np.full((B, R), -1, np.int32)
    for j in range(1, R):
        p[:, j] = r.integers(max(0, j - 5), j, B)
    return p


def make(seed, B, R, V, H, is_tree=False, nb=0, mask=False):
    r = np.random.default_rng(seed)
    c = dict(tok=r.integers(0, V, (B, R)).astype(np.int32), parent=tree(r, B, R) if is_tree else None,
             hist=np.minimum(V - 1, (V ** r.random((B, H)) - 1)).astype(np.int32) if H else None,
             hist_len=r.integers(0, H + 1, B).astype(np.int32) if H else None, prompt_len=None,
             repetition=r.uniform(0.7, 1.6, B).astype(np.float32), frequency=r.uniform(-0.5, 1, B).astype(np.float32),
             presence=r.uniform(-1, 1, B).astype(np.float32), bias=None, mask=None)
    if H:
        c["hist_len"][0] = H
        c["prompt_len"] = r.integers(0, H + 1, B).astype(np.int32)
        c["tok"][:, :] = np.where(r.random((B, R)) < 0.5, c["tok"], c["hist"][:, :1])
    if nb:
        c["bias"] = [{int(v): float(np.float32(r.uniform(-4, 4))) for v in r.integers(0, V, r.integers(0, nb + 1))} for _ in range(B)]
    if mask:
        c["mask"] = r.integers(-2 ** 31, 2 ** 31, (B, R, (V + 31) // 32)).astype(np.int32)
        c["mask"][0, 0] = 0            # a row that allows nothing
        c["mask"][-1, -1] = -1
    x = (3 * r.standard_normal((B, R, V))).astype(np.float32)
    return x, c


def args(c):
    a = {k: dev(v) for k, v in c.items() if k != "bias"}
    if c["bias"] is not None:
        off = np.concatenate([[0], np.cumsum([len(b) for b in c["bias"]])]).astype(np.int32)
        a.update(bias_off=dev(off), bias_tok=dev(np.array([v for b in c["bias"] for v in b], np.int32)),
                 bias_val=dev(np.array([w for b in c["bias"] for w in b.values()], np.float32)))
    return a


CASES = [
    # B, R, V, H, tree, biases, mask
    (1, 1, 1, 0, False, 0, False), (1, 1, 5, 3, False, 2, True), (2, 5, 127, 40, False, 10, True), (3, 4, 128, 300, True, 0, False),
    (2, 9, 1000, 1000, False, 50, True), (4, 1, 4099, 77, False, 5, True), (1, 65, 2050, 500, True, 20, True),
    (2, 128, 640, 64, True, 0, True), (1, 128, 333, 1, False, 3, False), (5, 5, 20000, 4096, False, 300, True),
    (1, 5, 151936, 8191, False, 0, False), (17, 2, 32000, 1023, True, 9, True),
]


@pytest.mark.parametrize("B,R,V,H,is_tree,nb,mask", CASES)
def test_matches_plain(sv, B, R, V, H, is_tree, nb, mask):
    x, c = make(B * 1000 + R, B, R, V, H, is_tree, nb, mask)
    want = ref.logits(x, **c, mask_value=-np.inf)
    out, keys = sv.logits_process(dev(x), **args(c), mask_value=float("-inf"), write_argmax=True)
    assert np.array_equal(out.cpu().numpy(), want)
    assert np.array_equal(keys.cpu().numpy(), ref.argmax_keys(want.reshape(B * R, V)))
    # keys alone, and in place
    none, keys2 = sv.logits_process(dev(x), **args(c), mask_value=float("-inf"), write_logits=False, write_argmax=True)
    assert none is None and torch.equal(keys, keys2)
    y = dev(x)
    got, none = sv.logits_process(y, **args(c), mask_value=float("-inf"), out=y)
    assert got is y and none is None and np.array_equal(y.cpu().numpy(), want)
    assert sv.get_device_error() == 0
    # float64: every step is rounded by at most 2^-24 of what it gives; none of
    # the steps gives more than the sum of all magnitudes
    w64 = ref.logits(x, **c, mask_value=-np.inf, dtype=np.float64)
    n = H + R
    size = np.abs(x) * 1.6 + n * 1.0 + 1 + 4
    fin = np.isfinite(w64)
    assert np.array_equal(fin, np.isfinite(want))
    assert np.all(np.abs(want[fin] - w64[fin]) <= 6 * 2.0 ** -24 * size[fin])


@pytest.mark.parametrize("only", ["repetition", "frequency", "presence", "bias", "mask", "nothing"])
def test_one_control_alone(sv, only):
    x, c = make(11, 2, 3, 515, 90, False, 8, True)
    for k in ("repetition", "frequency", "presence", "bias", "mask"):
        if k != only:
            c[k] = None
    if only in ("bias", "mask", "nothing"):
        for k in ("tok", "hist", "hist_len", "prompt_len"):
            c[k] = None
    want = ref.logits(x, **c)
    out, _ = sv.logits_process(dev(x), **args(c))
    assert np.array_equal(out.cpu().numpy(), want)
    assert sv.get_device_error() == 0


def test_masked_places_hold_anything(sv):
    """NaN and infinities behind the mask do not show; where it allows them they
    stay, and NaN under keys is reported."""
    r = np.random.default_rng(0)
    x = r.standard_normal((1, 2, 300)).astype(np.float32)
    x[0, :, 7], x[0, :, 8], x[0, :, 9], x[0, :, 10] = np.nan, np.inf, -np.inf, np.finfo(np.float32).min
    m = np.full((1, 2, 10), -1, np.int32)
    m[0, 0, 0] = ~(0b1111 << 7)
    out, keys = sv.logits_process(dev(x), mask=dev(m), write_argmax=True)
    want = x.copy()
    want[0, 0, 7:11] = np.float32(-1e30)
    assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)
    assert np.array_equal(keys.cpu().numpy(), ref.argmax_keys(want[0]))
    assert sv.get_device_error() == 1
    sv.logits_process(dev(x[:, :1]), mask=dev(m[:, :1]), write_argmax=True)
    assert sv.get_device_error() == 0


def test_duplicate_biases_keep_the_last(sv):
    x = np.zeros((2, 1, 200), np.float32)
    out, _ = sv.logits_process(dev(x), bias_off=dev(np.array([0, 3, 5], np.int32)), bias_tok=dev(np.array([4, 9, 4, 4, 4], np.int32)),
                               bias_val=dev(np.array([1, 2, 3, 5, 7], np.float32)))
    assert out[0, 0, [4, 9]].tolist() == [3, 2] and out[1, 0, [4, 9]].tolist() == [7, 0]
    assert int((out != 0).sum()) == 3


def test_bad_inputs_are_reported(sv):
    x, c = make(3, 3, 4, 700, 60, True, 0, False)
    base = ref.logits(x, **c)

    def call(flag, want, **kw):
        a = args(c)
        a.update({k: dev(v) for k, v in kw.items()})
        out, _ = sv.logits_process(dev(x), **a)
        assert sv.get_device_error() == flag
        assert np.array_equal(out.cpu().numpy(), want)
    call(0, base)
    h = c["hist"].copy()
    h[0, 0], h[2, 0] = -1, 700
    call(2, ref.logits(x, **{**c, "hist": h}), hist=h)
    t = c["tok"].copy()
    t[1, 2] = 5000
    call(2, ref.logits(x, **{**c, "tok": t}), tok=t)
    hl = c["hist_len"].copy()
    hl[0], hl[1] = 100, -2
    call(4, ref.logits(x, **{**c, "hist_len": np.clip(hl, 0, 60)}), hist_len=hl)
    rep, fr = c["repetition"].copy(), c["frequency"].copy()
    rep[0], rep[1], fr[2] = 0.0, np.nan, np.inf
    call(0x02000000, ref.logits(x, **{**c, "repetition": [1, 1, rep[2]], "frequency": [fr[0], fr[1], 0]}), repetition=rep, frequency=fr)
    call(0x01000000, base, bias_off=np.array([0, 3, 2, 9], np.int32), bias_tok=np.zeros(0, np.int32), bias_val=np.zeros(0, np.float32))
    p = c["parent"].copy()
    p[0] = [-1, 0, 3, 0]      # row 2's path is malformed: it is its own token alone
    a = args(c)
    a["parent"] = dev(p)
    out, _ = sv.logits_process(dev(x), **a)
    assert sv.get_device_error() == 0x10
    q = p.copy()
    q[0, 2] = -1
    want = ref.logits(x, **{**c, "parent": q})
    assert np.array_equal(out.cpu().numpy(), want)


@pytest.mark.parametrize("bad", [dict(repetition=[1.0, 0.0]), dict(repetition=[-1.0, 1.0]), dict(frequency=[0.0, np.nan]),
                                 dict(presence=[np.inf, 0.0])])
@pytest.mark.parametrize("masked", [False, True])
def test_bad_parameters_are_reported_without_tokens(sv, bad, masked):
    """Also where there are no tokens that they would apply to."""
    x = np.random.default_rng(0).standard_normal((2, 3, 1000)).astype(np.float32)
    mask = dev(np.full((2, 3, 32), -1, np.int32)) if masked else None
    out, _ = sv.logits_process(dev(x), mask=mask, **{k: dev(np.array(v, np.float32)) for k, v in bad.items()})
    assert sv.get_device_error() == 0x02000000
    assert np.array_equal(out.cpu().numpy(), x)
