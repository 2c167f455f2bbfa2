"""The attention over the 8-bit cache at the ends of what its numbers hold: values and
scores far apart, runs that are done again, and what memory order such runs rely on."""
import numpy as np
import pytest
import torch

import _serving_ref8 as ref8
from test_gpu_q8 import _device_inputs, dev, i32, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def pools_of(k, v, P, table, lens):
    """8-bit pools that hold rows k, v [B][H, len, 128] (float64), NaN behind them."""
    H = k[0].shape[0]
    out = []
    for rows, is_v in ((k, False), (v, True)):
        pool = np.full((P, H, ref8.Q8), 0x7F, np.uint8)
        for b in range(len(lens)):
            for p in range(0, lens[b], 16):
                for h in range(H):
                    ref8.put_rows(pool[table[b, p // 64], h], p % 64, rows[b][h, p:min(p + 16, lens[b])], is_v)
        out.append(pool)
    return out


def test_attn_units_that_end_inside_a_step_repeat(sv):  # noqa: F811
    """A CTA goes on from unit to unit, each of which ends inside a step whose other codes are
    NaN: the stage that it cleared is copied into again.  The same bits each time."""
    r = np.random.default_rng(1)
    B, R, Hq, H, mp = 48, 1, 28, 4, 64
    lens = r.integers(1, 1100, B)
    used = (lens + 63) // 64
    P = 64
    table = np.full((B, mp), -1, np.int32)
    for b in range(B):
        table[b, :used[b]] = r.permutation(P)[:used[b]]
    g = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    # (sequences share pages: the last page of each is its own, NaN from its end on)
    k, v = (r.integers(0, 127, (P + B, H, ref8.Q8)).astype(np.uint8) for _ in range(2))
    for pool, is_v in ((k, False), (v, True)):
        pool[..., 8192:8208] = np.full(4, 2.0 ** -8, "<f4").view(np.uint8)
        for b in range(B):
            table[b, used[b] - 1] = P + b
            at = ref8._code_bytes(is_v)[np.arange(64) >= (lens[b] - 1) % 64 + 1]
            pool[P + b][:, at.reshape(-1)] = 0x7F
    assert sv.verify_attn_q8_workspace(B, R, Hq, H, 128, mp * 64) > 0   # the pages are split over the SMs
    a = [mk(B, R, Hq, 128), dev(k), dev(v), i32(table), i32(lens), mk(B, H, R, 128), mk(B, H, R, 128)]
    want = sv.verify_attn_q8(*a)
    assert not bool(want.isnan().any())
    flush = torch.empty(2 ** 28, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(100):
        if i % 2:
            flush.fill_(i)
        differ += (sv.verify_attn_q8(*a) != want).any()
    assert int(differ) == 0
    assert sv.get_device_error() == 0


def test_attn_runs_done_again_repeat(sv):  # noqa: F811
    """Units that lie in several CTAs' runs, one key of which outweighs its reference by 60
    powers of two: what the run left in the workspace first is written again.  The
    same bits each time, and the heavy key's V."""
    r = np.random.default_rng(2)
    B, R, H, mp, t = 1, 1, 2, 250, 4000
    P = 70
    table = np.full((1, mp), -1, np.int32)
    table[0, :63] = r.permutation(P)[:63]
    k = r.standard_normal((H, t, 128)) * 0.01
    v = r.standard_normal((H, t, 128))
    q = np.zeros((B, R, H, 128))
    q[..., 0] = 1.0
    heavy = [700, 3100]
    for h in range(H):
        k[h, :, 0] = 0.0
        k[h, heavy[h], 0] = 60.0
    kp, vp = pools_of([k], [v], P, table, [t])
    assert sv.verify_attn_q8_workspace(B, R, H, H, 128, mp * 64) > 0
    z = torch.zeros(B, H, R, 128, dtype=torch.bfloat16, device="cuda")
    a = [torch.from_numpy(q).to(torch.bfloat16).cuda(), dev(kp), dev(vp), i32(table), i32([t]), z, z]
    want = sv.verify_attn_q8(*a, scale=0.6931471805599453)
    for h in range(H):
        x = ref8.get_rows(vp[table[0, heavy[h] // 64], h], True)[heavy[h] % 64]
        # (the others' weights are 2^-60 each; roundings of the output, 2^-8, and of P to f16, 2^-11)
        assert np.all(np.abs(want[0, 0, h].double().cpu().numpy() - x) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(x) + 1e-12)
    flush = torch.empty(2 ** 28, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(100):
        if i % 2:
            flush.fill_(i)
        differ += (sv.verify_attn_q8(*a, scale=0.6931471805599453) != want).any()
    assert int(differ) == 0
    assert sv.get_device_error() == 0


# Lets its dependents start at once, takes `ms`, and only then writes its output.
SLOW = r"""
extern "C" __global__ void slow_fill(unsigned short* out, const unsigned short* in, int n, int ms) {
    asm volatile("griddepcontrol.launch_dependents;");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (int i = 0; i < (1 << 24); ++i) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 > 1000000ull * ms) break;
        __nanosleep(1000);
    }
    for (int i = threadIdx.x; i < n; i += blockDim.x) out[i] = in[i];
}
"""


@pytest.mark.parametrize("B,mp", [(64, 33), (2, 250)])
def test_attn_cache_ready_under_a_long_kernel(sv, B, mp):  # noqa: F811
    """With cache_ready the copies start under the preceding kernel; one that takes longer than
    the limit of a wait is waited for all the same, and what it writes last is read."""
    if not hasattr(torch.cuda, "_compile_kernel"):
        pytest.skip("no way to compile a kernel here")
    slow = torch.cuda._compile_kernel(SLOW, "slow_fill")
    r = np.random.default_rng(3)
    R, Hq, H, t = 2, 12, 4, mp * 64 - 5
    P = 300
    pools = []
    for _ in range(2):
        pool = r.integers(0, 127, (P, H, ref8.Q8)).astype(np.uint8)
        pool[..., 8192:8208] = np.full(4, 2.0 ** -8, "<f4").view(np.uint8)
        pools.append(dev(pool))
    table = i32(np.stack([r.permutation(P)[:mp] for _ in range(B)]))
    g = torch.Generator(device="cuda").manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    src, kb, vb = mk(B, R, Hq, 128), mk(B, H, R, 128), mk(B, H, R, 128)
    lens = i32([t] * B)
    want = sv.verify_attn_q8(src, *pools, table, lens, kb, vb)
    q = torch.zeros_like(src)
    torch.cuda.synchronize()
    slow(grid=(1, 1, 1), block=(256, 1, 1), args=(q, src, q.numel(), 2500))
    got = sv.verify_attn_q8(q, *pools, table, lens, kb, vb, cache_ready=True)
    torch.cuda.synchronize()
    assert sv.get_device_error() == 0
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------
# scores and values far apart
# ---------------------------------------------------------------------------

LN2 = 0.6931471805599453   # the scale that makes scores powers of two


def softmax64(q, k, v, see):
    """q [R, Hq, 128], k, v [H, n, 128], see [R, n]: float64, by powers of two of q . k."""
    R, Hq, H = q.shape[0], q.shape[1], k.shape[0]
    z = torch.einsum("rhgd,hkd->rhgk", q.double().view(R, H, Hq // H, 128), k.double())
    z = z.masked_fill(~see[:, None, None, :], float("-inf"))
    p = torch.exp2(z - z.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    return (torch.einsum("rhgk,hkd->rhgd", p, v.double()).reshape(R, Hq, 128),
            torch.einsum("rhgk,hkd->rhgd", p, v.double().abs()).reshape(R, Hq, 128))


def close(got, want, wgt):
    """Where scores are one exact product each: the output's rounding (2^-8), P's to f16 (2^-11),
    and as much again for the exponentials and the scale's own rounding (2^-23 of scores up to
    2^8, in numerator and denominator), and sums in fp32."""
    return bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * wgt + 2.0 ** -126).all())


def held(pool, table, t, is_v):
    """[H, t, 128] on the GPU: what an 8-bit pool holds for a sequence."""
    n = (t + 63) // 64
    x = ref8.get_rows(pool[np.asarray(table)[:n]], is_v).transpose(1, 0, 2, 3)
    return torch.from_numpy(np.ascontiguousarray(x.reshape(pool.shape[1], n * 64, 128)[:, :t])).cuda()


def causal(R, t):
    return torch.cat([torch.ones(R, t, dtype=torch.bool), torch.ones(R, R).tril() > 0], 1).cuda()


def bf16(x):
    return torch.as_tensor(x).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("R", [40, 65])
@pytest.mark.parametrize("t,mp", [(0, 1), (100, 2), (520, 9), (520, 250)])
def test_attn_sums_near_the_end_of_their_range(sv, R, t, mp):  # noqa: F811
    """The last row's own key, which is not among the 32 that give references, lies 100 to 140
    powers of two above the others: its sum ends short of infinity, or past it."""
    r = np.random.default_rng(R + mp)
    P = mp + 1
    table = r.permutation(P)[:mp].reshape(1, mp)
    for size in (0.5, 500.0):
        v = size * r.choice([1.0, 0.75, -0.5], (1, t, 128))
        kp, vp = pools_of([np.zeros((1, t, 128))], [v], P, table, [t])
        q = torch.zeros(1, R, 1, 128)
        q[..., 0] = 1.0
        vb = bf16(size * r.choice([1.0, 0.75, -0.5], (1, 1, R, 128)))
        a = (dev(kp), dev(vp), i32(table), i32([t]))
        kc, vc = held(kp, table[0], t, False), held(vp, table[0], t, True)
        for gap in range(100, 141):
            kb = torch.zeros(1, 1, R, 128)
            kb[0, 0, R - 1, 0] = gap
            got = sv.verify_attn_q8(bf16(q), *a, bf16(kb), vb, scale=LN2)[0]
            want, wgt = softmax64(q[0].cuda(), torch.cat([kc, kb[0].cuda()], 1), torch.cat([vc, vb[0]], 1), causal(R, t))
            assert close(got, want, wgt), (size, gap, float((got.double() - want).abs().max()))
    assert sv.get_device_error() == 0


# ---------------------------------------------------------------------------
# runs that are done again
# ---------------------------------------------------------------------------

def _one_heavy_key(t, at, low, P=128):
    """A sequence of t positions (64 P at most) in pages 0 .. of one head: position `at` scores 30 and
    has V 0, the others score 30 - low and have V 1."""
    k, v = np.zeros((1, t, 128)), np.ones((1, t, 128))
    k[0, :, 0], k[0, :, 1] = 30.0, -low      # (two dims: each is held exactly)
    k[0, at, 1], v[0, at] = 0.0, 0.0
    table = np.arange(P).reshape(1, P)
    return pools_of([k], [v], P, table, [t])


@pytest.mark.parametrize("B,mp", [(160, 128), (1000, 128), (1000, 400)])
@pytest.mark.parametrize("nan_row", [False, True])
def test_attn_weights_far_below_the_largest(sv, B, mp, nan_row):  # noqa: F811
    """One key has all but a hundredth of the weight, which thousands of others share: also where a
    CTA's run is its fifth or later, or a row beside it is not finite, and is done again."""
    t, R = 8100, 2
    kp, vp = _one_heavy_key(t, 5000, 20.0)
    table = np.full((B, mp), -1, np.int32)
    table[:, :128] = np.arange(128)
    q = torch.zeros(B, R, 1, 128)
    q[..., :2] = 1.0
    if nan_row:
        q[:, 0] = float("nan")
    kb, vb = torch.zeros(B, 1, R, 128), torch.zeros(B, 1, R, 128)
    kb[..., 1] = -81.0       # the block itself has no weight
    got = sv.verify_attn_q8(bf16(q), dev(kp), dev(vp), i32(table), i32([t] * B), bf16(kb), bf16(vb), scale=LN2).double()
    w = (t - 1) * 2.0 ** -20
    want = w / (1 + w)
    # the output's rounding and P's, as much again as P's for the rest
    assert bool(((got[:, 1] - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want).all()), (want, float(got[:, 1].min()), float(got[:, 1].max()))
    assert bool(got[:, 0].isnan().all()) if nan_row else bool(((got[:, 0] - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want).all())
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("mp", [40, 400])
def test_attn_some_of_many_runs_fail(sv, mp):  # noqa: F811
    """Ragged sequences, several to a CTA, some of which hold a key far above their references: all
    give their rows."""
    r = np.random.default_rng(mp)
    B, R, Hq, H = 300, 2, 6, 2
    lens = r.integers(0, 700, B)
    P = 64
    k, v = r.standard_normal((2, H, P * 64, 128))
    k[..., 0] = 0.0
    heavy = r.integers(0, 64, P)
    for p in range(P):
        k[:, 64 * p + heavy[p], 0] = (p % 4 == 0) * r.integers(0, 90)
    kp, vp = pools_of([k], [v], P, np.arange(P).reshape(1, P), [P * 64])
    table = np.full((B, mp), -1, np.int32)
    for b in range(B):
        n = (lens[b] + 63) // 64
        table[b, :n] = r.permutation(P)[:n]
    q = r.standard_normal((B, R, Hq, 128)) * 0.05
    q[..., 0] = 1.0
    q, kb, vb = bf16(q), bf16(r.standard_normal((B, H, R, 128)) * 0.1), bf16(r.standard_normal((B, H, R, 128)))
    got = sv.verify_attn_q8(q, dev(kp), dev(vp), i32(table), i32(lens), kb, vb, scale=LN2)
    for b in range(B):
        t = int(lens[b])
        kc, vc = held(kp, table[b], t, False), held(vp, table[b], t, True)
        want, wgt = softmax64(q[b], torch.cat([kc, kb[b].double()], 1), torch.cat([vc, vb[b].double()], 1), causal(R, t))
        # scores of sums: 260 * 2^-22 of their magnitudes (below 2^8) and 2^-17 of |q|'s largest, 1, by the
        # largest sum of a row's |k| (below 2^8), each moving p twice
        s = 2 * (260 * 2.0 ** -22 * 2.0 ** 7 + 2.0 ** -17 * 2.0 ** 8)
        assert bool(((got[b].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -10 + s) * wgt).all()), b
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("B,R,Hq,H,t", [(1, 1, 28, 4, 7744), (9, 1, 8, 8, 2160), (6, 23, 12, 2, 4000), (16, 3, 28, 4, 2286), (2, 1, 28, 4, 9927)])
def test_attn_long_runs_round_p_to_f16(sv, B, R, Hq, H, t):  # noqa: F811
    """How often the output is not the bf16 next to the exact result: as often as P's rounding to 11
    bits takes it across a border (an error of deviation e crosses one of the borders between
    steps of u in 0.8 e / u of cases), not as often as 8 bits would, eight times that."""
    q, (kp, vp), table, kb, vb = _device_inputs(B, R, Hq, H, t, seed=t + 1)
    lens = i32([t - 29 * b for b in range(B)])
    k, v = sv.kv_gather_q8(kp[None], vp[None], table, i32([0] * B), lens, t)
    out = sv.verify_attn_q8(q, kp, vp, table, lens, kb, vb)
    see = torch.cat([torch.arange(t, device="cuda")[None, :] < lens[:, None],
                     torch.ones(B, R, dtype=torch.bool, device="cuda")], 1)[:, None, :].repeat(1, R, 1)
    see[:, :, t:] = torch.tril(torch.ones(R, R, dtype=torch.bool, device="cuda"))
    differ = expect = 0.0
    for h in range(H):
        kk, vv = (torch.cat([c[0, :, h].double(), n[:, h].double()], 1) for c, n in ((k, kb), (v, vb)))
        z = torch.einsum("brgd,bkd->brgk", q.view(B, R, H, Hq // H, 128)[:, :, h].double(), kk) * 128 ** -0.5
        p = torch.softmax(z.masked_fill(~see[:, :, None, :], float("-inf")), -1)
        want = torch.einsum("brgk,bkd->brgd", p, vv)
        # half a step of 11 bits, 2^-11 of a value at most, uniform; 2^-21 for what sums in fp32 add
        e = (2.0 ** -11 / 3 ** 0.5) * torch.einsum("brgk,bkd->brgd", p ** 2, vv ** 2).sqrt() + 2.0 ** -21 * torch.einsum(
            "brgk,bkd->brgd", p, vv.abs())
        u = torch.exp2(torch.floor(torch.log2(want.abs().clamp_min(1e-30))) - 7)
        expect += float((0.8 * e / u).clamp_max(1.0).sum())
        differ += float((out.view(B, R, H, Hq // H, 128)[:, :, h] != want.to(torch.bfloat16)).sum())
    n = out.numel()
    # (three deviations of a count)
    assert differ <= 2 * expect + 3 * expect ** 0.5, (differ / n, expect / n)
    assert sv.get_device_error() == 0


# ---------------------------------------------------------------------------
# values far apart
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("t,mp", [(520, 9), (520, 250), (200, 4)])
@pytest.mark.parametrize("big_at", [3, 70, 190])
def test_attn_one_large_value_of_no_weight(sv, big_at, t, mp):  # noqa: F811
    """One position's V is 2^8 to 2^60 times the others' and has no weight: it sets the unit of the
    others, or passes it, and they count as ever."""
    r = np.random.default_rng(big_at + mp)
    P = mp + 1
    table = r.permutation(P)[:mp].reshape(1, mp)
    k = np.zeros((1, t, 128))
    k[0, big_at, :2] = -200.0
    k[0, 150, 1] = 30.0
    q = torch.zeros(1, 2, 1, 128)     # row 0 sees the others alike, row 1 one of them
    q[0, 0, 0, 0] = q[0, 1, 0, 1] = 1.0
    kb = torch.zeros(1, 1, 2, 128)
    vb = bf16(r.standard_normal((1, 1, 2, 128)))
    v0 = r.standard_normal((1, t, 128)) + 0.5
    for power in (8, 11, 12, 14, 17, 20, 21, 22, 24, 27, 31, 40, 60, 100):
        v = v0.copy()
        v[0, big_at] = 2.0 ** power * np.sign(v[0, big_at])
        kp, vp = pools_of([k], [v], P, table, [t])
        got = sv.verify_attn_q8(bf16(q), dev(kp), dev(vp), i32(table), i32([t]), bf16(kb), vb, scale=LN2)[0]
        kc, vc = held(kp, table[0], t, False), held(vp, table[0], t, True)
        want, wgt = softmax64(q[0].cuda(), torch.cat([kc, kb[0].cuda()], 1), torch.cat([vc, vb[0]], 1), causal(2, t))
        assert close(got, want, wgt), (power, float((got.double() - want).abs().max()))
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("t,mp", [(130, 3), (520, 250), (1, 1)])
@pytest.mark.parametrize("least", [2.0 ** -115, 2.0 ** -100, 2.0 ** -40, 2.0 ** 60, 2.0 ** 118])
def test_attn_values_of_any_size_alone(sv, least, t, mp):  # noqa: F811
    """All of V next to nothing, or next to the largest that the cache holds."""
    r = np.random.default_rng(mp)
    P, R = mp + 1, 3
    table = r.permutation(P)[:mp].reshape(1, mp)
    v = least * r.integers(1, 9, (1, t, 128)) * r.choice([1.0, -1.0], (1, t, 128))
    kp, vp = pools_of([r.integers(-3, 4, (1, t, 128)) * 1.0], [v], P, table, [t])
    q = torch.zeros(1, R, 1, 128)
    q[0, :, 0, 5] = 1.0
    kb = torch.zeros(1, 1, R, 128)
    vb = bf16(least * r.integers(1, 9, (1, 1, R, 128)))
    got = sv.verify_attn_q8(bf16(q), dev(kp), dev(vp), i32(table), i32([t]), bf16(kb), vb, scale=LN2)[0]
    kc, vc = held(kp, table[0], t, False), held(vp, table[0], t, True)
    want, wgt = softmax64(q[0].cuda(), torch.cat([kc, kb[0].cuda()], 1), torch.cat([vc, vb[0]], 1), causal(R, t))
    assert close(got, want, wgt), float(((got.double() - want).abs() / wgt).max())
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("t,mp", [(0, 1), (100, 2), (520, 9), (520, 250)])
def test_attn_block_values_of_any_size(sv, t, mp):  # noqa: F811
    """A draft's V of 3e38, seen by the later rows alone and with or without weight there, beside an
    ordinary cache, and beside one whose values are next to nothing."""
    r = np.random.default_rng(mp + 7)
    P, R = mp + 1, 3
    table = r.permutation(P)[:mp].reshape(1, mp)
    q = torch.zeros(1, R, 1, 128)
    q[..., 0] = 1.0
    for size in (1.0, 2.0 ** -30, 2.0 ** -100):
        kp, vp = pools_of([r.integers(-2, 3, (1, t, 128)) * 1.0], [size * r.standard_normal((1, t, 128))], P, table, [t])
        kc, vc = held(kp, table[0], t, False), held(vp, table[0], t, True)
        for at in (1, 2):
            for score in (-300.0, -3.0, 0.0, 4.0):
                kb, vb = torch.zeros(1, 1, R, 128), torch.from_numpy(size * r.standard_normal((1, 1, R, 128)))
                kb[0, 0, at, 0] = score
                vb[0, 0, at] = 3e38 * torch.where(vb[0, 0, at] > 0, 1.0, -1.0)
                vb = bf16(vb)
                got = sv.verify_attn_q8(bf16(q), dev(kp), dev(vp), i32(table), i32([t]), bf16(kb), vb, scale=LN2)[0]
                want, wgt = softmax64(q[0].cuda(), torch.cat([kc, kb[0].cuda()], 1), torch.cat([vc, vb[0]], 1), causal(R, t))
                assert close(got, want, wgt), (size, at, score, got[:, 0, :3], want[:, 0, :3])
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("R,t,mp", [(3, 100, 2), (40, 520, 9), (40, 520, 250), (65, 100, 250)])
def test_attn_zeros_in_the_cache(sv, R, t, mp):  # noqa: F811
    """A pool of zeros (as a server's warm-up has it) beside a block of any values, also where the
    run is done again as the last row's own key outweighs what gives references."""
    r = np.random.default_rng(R)
    P = mp + 1
    table = r.permutation(P)[:mp].reshape(1, mp)
    kp, vp = pools_of([np.zeros((1, t, 128))], [np.zeros((1, t, 128))], P, table, [t])
    kc, vc = held(kp, table[0], t, False), held(vp, table[0], t, True)
    q = torch.zeros(1, R, 1, 128)
    q[..., 0] = 1.0
    for size in (1e-30, 1.0, 5000.0, 1e30):
        for gap in (0.0, 60.0, 131.0, 200.0):
            kb, vb = torch.zeros(1, 1, R, 128), bf16(size * r.standard_normal((1, 1, R, 128)))
            kb[0, 0, R - 1, 0] = gap
            got = sv.verify_attn_q8(bf16(q), dev(kp), dev(vp), i32(table), i32([t]), bf16(kb), vb, scale=LN2)[0]
            want, wgt = softmax64(q[0].cuda(), torch.cat([kc, kb[0].cuda()], 1), torch.cat([vc, vb[0]], 1), causal(R, t))
            assert close(got, want, wgt), (size, gap, got[R - 1, 0, :3], want[R - 1, 0, :3])
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("t,mp", [(100, 2), (520, 9), (520, 250)])
@pytest.mark.parametrize("top", [2.0 ** 7, 2.0 ** 60, 2.0 ** 110])
def test_attn_block_values_far_below_the_caches(sv, top, t, mp):  # noqa: F811
    """The cache's values have no weight and are up to 2^200 times the block's, which are all that
    the rows see."""
    r = np.random.default_rng(mp + 3)
    P, R = mp + 1, 3
    table = r.permutation(P)[:mp].reshape(1, mp)
    k = np.zeros((1, t, 128))
    k[0, :, 0] = -320.0
    kp, vp = pools_of([k], [top * r.standard_normal((1, t, 128))], P, table, [t])
    kc, vc = held(kp, table[0], t, False), held(vp, table[0], t, True)
    q = torch.zeros(1, R, 1, 128)
    q[..., 0] = 1.0
    for size in (1.0, 2.0 ** -40, 2.0 ** -90):
        kb, vb = torch.zeros(1, 1, R, 128), bf16(size * r.standard_normal((1, 1, R, 128)))
        got = sv.verify_attn_q8(bf16(q), dev(kp), dev(vp), i32(table), i32([t]), bf16(kb), vb, scale=LN2)[0]
        want, wgt = softmax64(q[0].cuda(), torch.cat([kc, kb[0].cuda()], 1), torch.cat([vc, vb[0]], 1), causal(R, t))
        assert close(got, want, wgt), (size, float((got.double() - want).abs().max()))
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("t,mp", [(520, 9), (520, 250), (200, 4)])
@pytest.mark.parametrize("which", ["first", "later", "every second", "all but one"])
def test_attn_runs_of_zeros_in_v(sv, which, t, mp):  # noqa: F811
    """Sixteen and more positions whose V is 0, before, behind and between others."""
    r = np.random.default_rng(mp + 5)
    P, R = mp + 1, 2
    table = r.permutation(P)[:mp].reshape(1, mp)
    v = r.standard_normal((1, t, 128))
    run = np.arange(t) // 16
    v[:, {"first": run < 9, "later": run > 5, "every second": run % 2 == 0, "all but one": run != 10}[which]] = 0.0
    kp, vp = pools_of([r.integers(-2, 3, (1, t, 128)) * 1.0], [v], P, table, [t])
    kc, vc = held(kp, table[0], t, False), held(vp, table[0], t, True)
    q = torch.zeros(1, R, 1, 128)
    q[..., 0] = 1.0
    kb, vb = torch.zeros(1, 1, R, 128), bf16(r.standard_normal((1, 1, R, 128)))
    got = sv.verify_attn_q8(bf16(q), dev(kp), dev(vp), i32(table), i32([t]), bf16(kb), vb, scale=LN2)[0]
    want, wgt = softmax64(q[0].cuda(), torch.cat([kc, kb[0].cuda()], 1), torch.cat([vc, vb[0]], 1), causal(R, t))
    assert close(got, want, wgt), float(((got.double() - want).abs() / wgt).max())
    assert sv.get_device_error() == 0
