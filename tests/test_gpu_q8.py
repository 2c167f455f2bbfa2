"""The 8-bit cache on the GPU: append, commit and gather bit for bit against the plain
forms, attention within the roundings it makes."""
import numpy as np
import pytest
import torch

import _serving_ref as ref
import _serving_ref8 as ref8
from speculative_decoding_verification_sv_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_sv_gb300 import binding
    return binding


def bf(x):
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def dev(x):
    return torch.from_numpy(x).cuda()


def random_pool(r, *lead, lo=-8, hi=-4):
    """Blocks of random finite codes whose scales are 2^lo .. 2^(hi - 1)."""
    pool = r.integers(0, 256, (*lead, ref8.Q8)).astype(np.uint8)
    pool[pool & 127 == 127] = 0
    s = np.ldexp(1.0, r.integers(lo, hi, (*lead, 4))).astype("<f4")
    pool[..., 8192:8208] = np.ascontiguousarray(s).view(np.uint8).reshape(*lead, 16)
    return pool


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def run_append(sv, r, B, H, counts, lens, rot, inter, mp=5, grow=1.0, kp=None, vp=None, k=None, v=None, rope_pos=None):
    P = B * mp + 2
    table = r.permutation(P)[: B * mp].reshape(B, mp).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    N = int(off[-1])
    k = ref.bf16_round(r.standard_normal((N, H, 128)) * grow) if k is None else k
    v = ref.bf16_round(r.standard_normal((N, H, 128)) * grow) if v is None else v
    k, v = bf(k).double().numpy(), bf(v).double().numpy()     # (bf16_round knows the normal range alone)
    kp = random_pool(r, P, H) if kp is None else kp
    vp = random_pool(r, P, H) if vp is None else vp
    rope = None if rot == 0 else ref.rope_table(rope_pos or mp * 64, rot)
    gk, gv = dev(kp), dev(vp)
    sv.kv_append_q8(bf(k).cuda(), bf(v).cuda(), i32(off), gk, gv, i32(table), i32(lens), None if rope is None else dev(rope),
                    interleaved=inter)
    cap = min(mp * 64, rope_pos or mp * 64)
    wk, wv = ref8.append(k, v, off, kp, vp, table, lens, rope, inter, cap)
    end = np.minimum(np.array(lens) + counts, cap)
    und = ref8.undefined((P, H, 64), table, lens, end, P)
    assert ref8.same_pool(gk.cpu().numpy(), wk, und, False)
    assert ref8.same_pool(gv.cpu().numpy(), wv, und, True)
    return gk, gv


@pytest.mark.parametrize("rot,inter", [(0, False), (128, False), (64, True), (16, False), (32, True)])
@pytest.mark.parametrize("B,H,counts,lens", [
    (1, 1, [1], [0]), (1, 2, [1], [15]), (1, 1, [16], [16]), (2, 2, [17, 3], [63, 0]), (4, 1, [100, 0, 33, 7], [9, 64, 31, 250]),
    (3, 4, [1, 1, 1], [7, 16, 130])])
def test_append_matches_plain(sv, B, H, counts, lens, rot, inter):
    run_append(sv, np.random.default_rng(B + rot), B, H, counts, lens, rot, inter)
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("grow", [2.0 ** -9, 1.0, 30.0, 1e5, 1e30, 2.0 ** -125])
def test_append_scales_grow(sv, grow):
    """New rows far above and far below what their run holds: its earlier rows keep their
    values or are held in the larger scale, down to nothing."""
    run_append(sv, np.random.default_rng(3), 3, 2, [3, 20, 1], [5, 30, 47], 0, False, grow=grow)
    assert sv.get_device_error() == 0


def test_append_token_by_token(sv):
    """Forty single tokens of growing size, each against the plain form on what was there."""
    r = np.random.default_rng(5)
    H, mp = 2, 1
    kp, vp = random_pool(r, 3, H), random_pool(r, 3, H)
    for t in range(40):
        gk, gv = run_append(sv, np.random.default_rng(9), 1, H, [1], [t], 128, False, mp=mp, kp=kp, vp=vp,
                            k=ref.bf16_round(r.standard_normal((1, H, 128)) * 1.5 ** t), v=ref.bf16_round(r.standard_normal((1, H, 128))))
        kp, vp = gk.cpu().numpy(), gv.cpu().numpy()
    assert sv.get_device_error() == 0


def test_append_extremes(sv):
    """The largest bf16, its smallest, zeros, and what lies past the largest scale."""
    r = np.random.default_rng(6)
    big = 255.0 * 2.0 ** 120
    for a in (0.0, 2.0 ** -133, big, 448 * 2.0 ** 119):
        rows = ref.bf16_round(np.where(r.standard_normal((20, 1, 128)) > 0, a, -a)) if a != 2.0 ** -133 else np.full((20, 1, 128), a)
        run_append(sv, r, 1, 1, [20], [3], 0, False, k=rows, v=rows)
    assert sv.get_device_error() == 0


def test_append_rows_that_are_not_finite(sv):
    r = np.random.default_rng(7)
    k, v = ref.bf16_round(r.standard_normal((2, 40, 2, 128)))
    k[3, 0, 17], k[20, 1, 0], v[4, 1, 127], v[39, 0, 64] = np.nan, np.inf, -np.inf, np.nan
    gk, gv = run_append(sv, r, 2, 2, [25, 15], [10, 64], 0, False, k=k, v=v)
    assert sv.get_device_error() == 1
    assert bool((gv.cpu().numpy()[..., :8192] & 127 == 127).any())


def test_append_places_that_do_not_exist(sv):
    r = np.random.default_rng(8)
    run_append(sv, r, 2, 1, [30, 9], [300, 0], 0, False)          # past the table's 320 positions
    assert sv.get_device_error() == 4
    run_append(sv, r, 2, 1, [30, 9], [80, 0], 32, False, rope_pos=100)
    assert sv.get_device_error() == 4
    run_append(sv, r, 2, 1, [30, 9], [-3, 0], 0, False)           # a negative length: nothing of the sequence
    assert sv.get_device_error() == 4


def test_append_bad_pages_and_offsets(sv):
    r = np.random.default_rng(9)
    H, mp, P = 2, 3, 8
    k, v = ref.bf16_round(r.standard_normal((2, 60, H, 128)))
    kp, vp = random_pool(r, P, H), random_pool(r, P, H)
    table = np.array([[0, -1, 2], [3, 4, 8]], np.int32)
    off = np.array([0, 50, 60], np.int32)
    gk, gv = dev(kp), dev(vp)
    sv.kv_append_q8(bf(k).cuda(), bf(v).cuda(), i32(off), gk, gv, i32(table), i32([50, 120]))
    assert sv.get_device_error() == 0x80
    wk, wv = ref8.append(k, v, off, kp, vp, table, [50, 120], None, False, mp * 64)
    und = ref8.undefined((P, H, 64), table, [50, 120], [100, 130], P)
    assert ref8.same_pool(gk.cpu().numpy(), wk, und, False) and ref8.same_pool(gv.cpu().numpy(), wv, und, True)
    # offsets that fall: that sequence's rows stay out
    gk, gv = dev(kp), dev(vp)
    sv.kv_append_q8(bf(k).cuda(), bf(v).cuda(), i32([40, 30, 60]), gk, gv, i32([[0, 1, 2], [3, 4, 5]]), i32([0, 0]))
    assert sv.get_device_error() == 0x01000000
    assert np.array_equal(gk.cpu().numpy()[:3], kp[:3])


# ---------------------------------------------------------------------------
# commit, gather
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("L,B,H,R,lens,tree,grow", [
    (1, 1, 1, 1, [0], False, 1.0), (3, 3, 2, 5, [59, 64, 7], False, 1.0), (2, 4, 1, 20, [44, 0, 63, 101], True, 20.0),
    (5, 1, 4, 9, [120], False, 1e6), (1, 2, 1, 128, [1, 62], False, 1.0), (28, 2, 4, 9, [70, 15], True, 0.01)])
def test_commit_matches_plain(sv, L, B, H, R, lens, tree, grow):
    r = np.random.default_rng(R * 10 + L)
    mp, P = 4, B * 4 + 2
    table = r.permutation(P)[: B * mp].reshape(B, mp).astype(np.int32)
    kp, vp = random_pool(r, L, P, H), random_pool(r, L, P, H)
    kb, vb = ref.bf16_round(grow * r.standard_normal((2, L, B, H, R, 128)))
    n_acc = r.integers(0, R, B).astype(np.int32)
    n_acc[0] = R - 1
    path = np.full((B, R), -1, np.int32)
    for b in range(B):
        path[b, :n_acc[b] + 1] = np.sort(r.permutation(R)[:n_acc[b] + 1]) if tree else np.arange(n_acc[b] + 1)
    ln = np.array(lens, np.int32)
    gk, gv, gl = dev(kp), dev(vp), i32(ln)
    sv.kv_commit_q8(gk, gv, i32(table), bf(kb).cuda(), bf(vb).cuda(), i32(path), i32(n_acc), gl)
    wk, wv, wl = ref8.commit(kp, vp, table, kb, vb, path, n_acc, ln)
    und = ref8.undefined((P, H, 64), table, ln, wl, P)
    assert np.array_equal(gl.cpu().numpy(), wl)
    assert ref8.same_pool(gk.cpu().numpy(), wk, und, False)
    assert ref8.same_pool(gv.cpu().numpy(), wv, und, True)
    assert sv.get_device_error() == 0


def test_commit_leaves_bad_sequences_untouched(sv):
    r = np.random.default_rng(4)
    L, B, H, R, mp = 2, 5, 1, 6, 2
    P = B * mp
    table = np.arange(P, dtype=np.int32).reshape(B, mp)
    kp, vp = random_pool(r, L, P, H), random_pool(r, L, P, H)
    kb, vb = ref.bf16_round(r.standard_normal((2, L, B, H, R, 128)))
    path = np.tile(np.arange(R, dtype=np.int32), (B, 1))
    for lens, nacc, bad, flag in (([10, 124, 3, 60, 0], [5, 5, 5, 5, 0], [1], 4), ([10, -1, 3, 60, 0], [5, 5, 5, 5, 0], [1], 4),
                                  ([10, 12, 3, 60, 0], [5, 6, -1, 5, 0], [1, 2], 0x20), ([10, 12, 3, 60, 0], [5, 5, 5, 5, 0], [2], 0x20),
                                  ([10, 12, 3, 60, 0], [5, 5, 5, 5, 0], [3], 0x80)):
        tb, pa = table.copy(), path.copy()
        if flag == 0x20 and bad == [2]:
            pa[2, 3] = R
        if flag == 0x80:
            tb[3, 1] = -1
        ln, na = np.array(lens, np.int32), np.array(nacc, np.int32)
        gk, gv, gl = dev(kp), dev(vp), i32(ln)
        sv.kv_commit_q8(gk, gv, i32(tb), bf(kb).cuda(), bf(vb).cuda(), i32(pa), i32(na), gl)
        assert sv.get_device_error() == flag
        ok = [b for b in range(B) if b not in bad]
        wk, wv, wl = ref8.commit(kp, vp, tb[ok], kb[:, ok], vb[:, ok], pa[ok], na[ok], ln[ok])
        und = ref8.undefined((P, H, 64), tb[ok], ln[ok], wl, P)
        assert ref8.same_pool(gk.cpu().numpy(), wk, und, False) and ref8.same_pool(gv.cpu().numpy(), wv, und, True)
        assert gl.cpu().numpy()[ok].tolist() == wl.tolist() and gl.cpu().numpy()[bad].tolist() == ln[bad].tolist()


@pytest.mark.parametrize("lo,hi", [(-8, -4), (-120, -100), (100, 120), (0, 9)])
@pytest.mark.parametrize("L,B,H,n,start,lens", [
    (1, 1, 1, 1, [0], [1]), (2, 3, 2, 130, [0, 61, 7], [256, 100, 0]), (1, 4, 1, 9, [5, 250, 255, 64], [256, 256, 256, 66]),
    (3, 1, 1, 256, [0], [200]), (1, 1, 2, 40, [300], [256]), (1, 2, 1, 17, [15, 16], [32, 33])])
def test_gather_matches_plain(sv, L, B, H, n, start, lens, lo, hi):
    r = np.random.default_rng(n)
    mp, P = 4, B * 4 + 1
    table = r.permutation(P)[: B * mp].reshape(B, mp).astype(np.int32)
    kp, vp = random_pool(r, L, P, H, lo=lo, hi=hi), random_pool(r, L, P, H, lo=lo, hi=hi)
    k, v = sv.kv_gather_q8(dev(kp), dev(vp), i32(table), i32(start), i32(lens), n)
    assert np.array_equal(k.double().cpu().numpy(), ref8.gather(kp, table, start, lens, n, False))
    assert np.array_equal(v.double().cpu().numpy(), ref8.gather(vp, table, start, lens, n, True))
    assert sv.get_device_error() == 0


def test_gather_bad_inputs_and_nan(sv):
    r = np.random.default_rng(0)
    kp = random_pool(r, 1, 4, 1)
    for is_v in (False, True):
        ref8.put_rows(kp[0, 1, 0], 5, np.full((1, 128), np.nan), is_v)
        g = dev(kp)
        got = sv.kv_gather_q8(g, g, i32([[1, 2]]), i32([0]), i32([100]), 100)[is_v].double().cpu().numpy()
        want = ref8.gather(kp, np.array([[1, 2]]), [0], [100], 100, is_v)
        assert np.isnan(want).any() and np.array_equal(got, want, equal_nan=True)
    kp = random_pool(r, 1, 4, 1)
    g = dev(kp)
    table = np.array([[0, 9], [1, 2]], np.int32)
    k, _ = sv.kv_gather_q8(g, g, i32(table), i32([60, 60]), i32([128, 128]), 8)
    assert sv.get_device_error() == 0x80
    assert np.array_equal(k.double().cpu().numpy(), ref8.gather(kp, table, [60, 60], [128, 128], 8, False))
    k, _ = sv.kv_gather_q8(g, g, i32([[0, 1], [1, 2]]), i32([-1, 120]), i32([128, 200]), 16)
    assert sv.get_device_error() == 4
    want = ref8.gather(kp, np.array([[0, 1], [1, 2]]), [-1, 120], [128, 128], 16, False)
    assert np.array_equal(k.double().cpu().numpy(), want)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def tol(want, wgt, big, units, keys, lost):
    """The output is rounded to bf16, a half step of 2^-8 of what it is, and P to f16, 2^-11;
    sums of 128 products (in two or four parts) move a score by at most 260 * 2^-22 of
    their magnitudes (p by that factor, twice: numerator and denominator), the
    exponentials by 2^-20; sums over the keys and their rescalings by 2^-22 a term; the
    elements of Q and of the block's K are off by 2^-17 of their row's largest (2^-10 of
    units of which the largest is at least 224), which moves a score by 2^-17 `units`.
    `lost` (below): what f16 holds of the smallest P and V."""
    p = 2.0 ** -11 + 2 * (260 * 2.0 ** -22 * big + 2.0 ** -17 * units + 2.0 ** -20) + 2 * keys * 2.0 ** -22
    return 2.0 ** -8 * np.abs(want) + 1.01 * (p * wgt + lost) + 1e-30


def lost_of(scale, v_ctx, vb, G):
    """[Hq, 128]: f16's steps end at 2^-24.  A P is 2^-5 at a key that the row sees, so that the
    sum of P is 2^-5 or more: rounding it there moves a weight by at most 2^-25 / 2^-5, and
    the result by the sum of those and |v|.  V there is in units of 2^4 times the largest scale
    of the first pages: a value moves by at most 2^-25 of that, 2^-21 of the largest scale."""
    h = []
    for k in range(vb.shape[0]):
        v = np.concatenate([v_ctx[k], np.where(np.isfinite(vb[k]), vb[k], 0.0)])
        unit = max(scale, 2.0 ** ref8.exponent(np.abs(v).max()))
        h += [2.0 ** -20 * np.abs(v).sum(0) + 2.0 ** -21 * unit] * G
    return np.stack(h)


def units_of(q, k_ctx, kb, scale):
    """The largest scale * (max |q| sum |k| + max |k| sum |q|) over the pairs."""
    a = np.abs(np.concatenate([k_ctx, kb], 1))
    qa = np.abs(q).reshape(-1, 128)
    return scale * float(qa.max() * a.sum(-1).max() + (a.max() if kb.shape[1] else 0.0) * qa.sum(-1).max())


def poison(pool, table, lens, mp, is_v):
    """Positions at and past the length hold NaN codes, and the scales of runs that hold no
    other are NaN or infinity."""
    for b in range(len(lens)):
        for p in range(lens[b], mp * 64):
            blk = pool[table[b, p // 64]]
            blk[:, ref8._code_bytes(is_v)[p % 64]] = 0x7F
            if p % 16 == 0:
                at = 8192 + p % 64 // 16 * 4
                blk[:, at:at + 4] = np.frombuffer(np.float32(np.nan if p % 32 else np.inf).tobytes(), np.uint8)


def run(sv, B, R, Hq, H, lens, parent=None, scale=None, seed=0, mp=None, lo=-8, hi=-4, **kw):
    r = np.random.default_rng(seed)
    mp = mp or max(1, (max(lens) + 63) // 64)
    P = B * mp + 1
    table = r.permutation(P)[: B * mp].reshape(B, mp).astype(np.int32)
    kp, vp = random_pool(r, P, H, lo=lo, hi=hi), random_pool(r, P, H, lo=lo, hi=hi)
    poison(kp, table, lens, mp, False)
    poison(vp, table, lens, mp, True)
    q = ref.bf16_round(r.standard_normal((B, R, Hq, 128)))
    kb, vb = ref.bf16_round(r.standard_normal((2, B, H, R, 128)))
    out = sv.verify_attn_q8(bf(q).cuda(), dev(kp), dev(vp), i32(table), i32(lens), bf(kb).cuda(), bf(vb).cuda(),
                            None if parent is None else i32(parent), scale=scale, **kw)
    got = out.double().cpu().numpy()
    s = scale or 128 ** -0.5
    for b in range(B):
        n = (lens[b] + 63) // 64
        rows = lambda pool, is_v: ref8.get_rows(pool[table[b, :n]], is_v).transpose(1, 0, 2, 3).reshape(H, n * 64, 128)[:, :lens[b]]  # noqa: E731
        k, v = rows(kp, False), rows(vp, True)
        want, wgt, big = ref.attention(q[b], k, v, kb[b], vb[b], None if parent is None else parent[b:b + 1], s)
        err = np.abs(got[b] - want)
        bound = tol(want, wgt, big, units_of(q[b], k, kb[b], s), lens[b] + R, lost_of(2.0 ** (hi - 1), v, vb[b], Hq // H))
        assert np.all(err <= bound), (b, float((err / bound).max()), np.argwhere(~(err <= bound))[:4].tolist())
    assert sv.get_device_error() == 0
    return out


@pytest.mark.parametrize("B,R,Hq,H,lens", [
    (1, 1, 1, 1, [0]), (1, 1, 1, 1, [1]), (2, 1, 8, 8, [150, 7]), (2, 5, 12, 2, [0, 1]), (3, 9, 28, 4, [63, 64, 65]),
    (4, 2, 4, 1, [127, 128, 129, 191]), (1, 5, 12, 2, [1000]), (4, 9, 28, 4, [700, 513, 640, 77]), (1, 17, 16, 2, [600]),
    (1, 128, 2, 1, [260]), (1, 8, 16, 1, [333]), (1, 3, 32, 2, [129]), (2, 65, 28, 4, [130, 5]), (8, 3, 8, 2, [9, 80, 0, 200, 64, 128, 31, 256]),
    (1, 5, 12, 2, [2500])])
def test_attn_chain(sv, B, R, Hq, H, lens):
    run(sv, B, R, Hq, H, lens, seed=R + B)


@pytest.mark.parametrize("B,R,Hq,H,lens", [(1, 2, 4, 2, [10]), (2, 9, 12, 2, [130, 64]), (1, 65, 28, 4, [513]), (2, 128, 4, 2, [0, 70]),
                                           (3, 33, 16, 2, [63, 1, 200])])
def test_attn_tree(sv, B, R, Hq, H, lens):
    r = np.random.default_rng(R)
    par = np.full((B, R), -1, np.int32)
    for b in range(B):
        for j in range(1, R):
            par[b, j] = r.integers(max(0, j - 6), j)
    run(sv, B, R, Hq, H, lens, parent=par, seed=R)


@pytest.mark.parametrize("B,R,Hq,H,mp", [(33, 1, 4, 2, 4), (70, 3, 4, 1, 6), (200, 1, 2, 2, 5)])
def test_attn_many_sequences(sv, B, R, Hq, H, mp):
    """More sequences than a warp has lanes, some of them empty."""
    lens = np.random.default_rng(B).integers(0, mp * 64 + 1, B)
    lens[[0, 31, 32, B - 1]] = [mp * 64, 0, 1, 0]
    run(sv, B, R, Hq, H, lens.tolist(), seed=B, mp=mp)


def test_attn_scale_and_capacity(sv):
    run(sv, 1, 4, 8, 2, [192], scale=0.7, seed=3)                 # a full table
    run(sv, 2, 4, 8, 2, [100, 3], scale=0.01, seed=4, mp=40)       # a table much longer than the contexts
    run(sv, 1, 5, 12, 2, [90], seed=5, cache_ready=True)


@pytest.mark.parametrize("lo,hi", [(-30, 0), (-120, -110), (5, 12)])
def test_attn_scales_far_apart(sv, lo, hi):
    """Runs whose scales differ widely, are next to nothing, or pass 2^7 (where V takes a
    product more)."""
    run(sv, 2, 5, 12, 2, [300, 77], seed=hi + 200, lo=lo, hi=hi, scale=2.0 ** -12 if hi > 1 else None)


@pytest.mark.parametrize("B,R,Hq,H,lens,is_tree,mp", [
    (1, 5, 12, 2, [1000], False, 250), (3, 5, 12, 2, [63, 0, 700], False, 500), (2, 9, 28, 4, [700, 0], False, 800),
    (3, 65, 28, 4, [130, 5, 0], True, 250), (1, 1, 1, 1, [1], False, 250), (2, 20, 16, 2, [640, 129], True, 2000)])
def test_attn_split_over_all_sms(sv, B, R, Hq, H, lens, is_tree, mp):
    """A long table (its capacity sets how the work is split): the pages are laid
    end to end over the SMs, and units in several of them joined by the second
    kernel.  Shorter tables give each unit a cluster of CTAs."""
    assert sv.verify_attn_q8_workspace(B, R, Hq, H, 128, mp * 64) > 0
    assert sv.verify_attn_q8_workspace(1, 5, 12, 2, 128, 2048) == 0
    r = np.random.default_rng(R)
    par = np.full((B, R), -1, np.int32)
    for j in range(1, R):
        par[:, j] = r.integers(max(0, j - 6), j, B)
    run(sv, B, R, Hq, H, lens, parent=par if is_tree else None, seed=R, mp=mp)
    run(sv, B, R, Hq, H, lens, parent=par if is_tree else None, seed=R, mp=mp, scale=9.0)


@pytest.mark.parametrize("t", [4096, 40, 0])
def test_attn_every_cluster_size(sv, t):
    """Page tables whose capacity gives units clusters of 1 to 8 CTAs (and none), which
    the lengths fill, hardly reach or leave empty."""
    for B, R, Hq, H in ((1, 5, 12, 2), (4, 2, 28, 4), (3, 9, 28, 4), (6, 9, 28, 4), (9, 9, 28, 4), (14, 9, 28, 4), (20, 3, 12, 4), (40, 1, 28, 4),
                        (40, 9, 28, 4), (90, 2, 12, 4)):
        q, (kp, vp), table, kb, vb = _device_inputs(B, R, Hq, H, 4096, seed=B)
        lens = i32([max(0, t - 17 * b) for b in range(B)])
        out = sv.verify_attn_q8(q, kp, vp, table, lens, kb, vb)
        k, v = sv.kv_gather_q8(kp[None], vp[None], table, i32([0] * B), lens, max(t, 1))
        k, v = torch.cat([k[0].float(), kb.float()], 2), torch.cat([v[0].float(), vb.float()], 2)
        n = max(t, 1)
        see = torch.zeros(B, R, n + R, dtype=torch.bool, device="cuda")
        see[:, :, :n] = (torch.arange(n, device="cuda")[None, :] < lens[:, None])[:, None]
        see[:, :, n:] = torch.ones(R, R, device="cuda").tril() > 0
        G = Hq // H
        z = torch.einsum("brhgd,bhkd->bhrgk", q.float().view(B, R, H, G, 128), k) * 128 ** -0.5
        p = torch.softmax(z.masked_fill(~see[:, None, :, None], float("-inf")), -1)
        want = torch.einsum("bhrgk,bhkd->brhgd", p, v).reshape(B, R, Hq, 128)
        wgt = torch.einsum("bhrgk,bhkd->brhgd", p, v.abs()).reshape(B, R, Hq, 128)
        # the output's rounding (2^-8) and P's (2^-11), and as much again as P's for both sides' sums and scores in fp32
        assert bool(((out.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * wgt + 1e-6).all()), (B, R)
    assert sv.get_device_error() == 0


def one_sequence(sv, q, kp, vp, table, t, kb, vb, scale, parent=None, lost=0):
    """One sequence's attention against the plain form (whose first `lost` positions do not count)."""
    H, R = kb.shape[1], kb.shape[2]
    out = sv.verify_attn_q8(bf(q).cuda(), dev(kp), dev(vp), i32(table), i32([t]), bf(kb).cuda(), bf(vb).cuda(),
                            None if parent is None else i32(parent), scale=scale)
    n = (t + 63) // 64
    rows = lambda pool, is_v: ref8.get_rows(pool[table[0, :n]], is_v).transpose(1, 0, 2, 3).reshape(H, n * 64, 128)[:, lost:t]  # noqa: E731
    k, v = rows(kp, False), rows(vp, True)
    seen = parent if parent is None else np.where(np.asarray(parent) >= R, -1, parent)
    want, wgt, big = ref.attention(q[0], k, v, kb[0], vb[0], seen, scale)
    bound = tol(want, wgt, big, units_of(q[0], k, kb[0], scale), t + R, lost_of(2.0 ** -5, v, vb[0], q.shape[2] // H))
    err = np.abs(out[0].double().cpu().numpy() - want)
    assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(~(err <= bound))[:4].tolist())


def filled(r, P, H, value):
    """K whose every position holds value(page's position) in every dim."""
    blk = np.zeros(ref8.Q8, np.uint8)
    for p in range(0, 64, 16):
        ref8.put_rows(blk, p, np.stack([np.full(128, value(p + i)) for i in range(16)]), False)
    return np.broadcast_to(blk, (P, H, ref8.Q8)).copy()


def test_attn_references_far_below(sv):
    """The first key's score far below the others': the sums leave their range
    and the run is done again with the running maxima, in a cluster and over all
    SMs."""
    r = np.random.default_rng(8)
    for mp in (9, 250):
        P, t, R, Hq = mp + 1, 520, 3, 4
        table = r.permutation(P)[:mp].reshape(1, mp).astype(np.int32)
        kp, vp = random_pool(r, P, 1), random_pool(r, P, 1)
        q = ref.bf16_round(np.abs(ref.bf16_round(r.standard_normal((1, R, Hq, 128)))) + 0.5)
        kb, vb = ref.bf16_round(r.standard_normal((2, 1, 1, R, 128)))
        ref8.put_rows(kp[table[0, 0], 0], 0, np.full((1, 128), -6.0), False)
        for p in (70, 300, 519):
            ref8.put_rows(kp[table[0, p // 64], 0], p % 64, np.full((1, 128), 1.0 + p / 200), False)
        one_sequence(sv, q, kp, vp, table, t, kb, vb, 0.5)
        assert sv.get_device_error() == 0


@pytest.mark.parametrize("t,H,mp", [(0, 1, 1), (0, 2, 9), (0, 2, 250), (448, 1, 7), (512, 4, 250), (70, 2, 40)])
def test_attn_malformed_row_sees_the_cache_and_itself(sv, t, H, mp):
    """Block row 0, which a malformed row does not see, has a score 739 powers of two
    above that row's own, and that one 739 above the cache's; also where a CTA's run
    holds the block alone."""
    r = np.random.default_rng(t)
    P, R = mp + 1, 2
    table = r.permutation(P)[:mp].reshape(1, mp).astype(np.int32)
    vp = random_pool(r, P, H)
    kp = filled(r, P, H, lambda p: -6.0)
    q = np.full((1, R, H, 128), 2.0)
    kb, vb = ref.bf16_round(r.standard_normal((2, 1, H, R, 128)))
    kb[0, :, 0], kb[0, :, 1] = 2.0, -2.0
    one_sequence(sv, q, kp, vp, table, t, kb, vb, 0.5, parent=np.array([[-1, 7]]))
    assert sv.get_device_error() == 0x10


def _far_below(sv, t, mp, lost):
    """The scores of the first `lost` positions are -infinity (products past fp32),
    all others hundreds of powers of two below 0."""
    r = np.random.default_rng(t + mp)
    P, R, Hq = mp + 1, 3, 4
    table = r.permutation(P)[:mp].reshape(1, mp).astype(np.int32)
    kp, vp = random_pool(r, P, 1), random_pool(r, P, 1)
    for p0 in range(0, t, 16):
        n = min(16, t - p0)
        rows = np.stack([np.full(128, -(2.0 ** 118)) if p < lost else ref.bf16_round(-(2.0 ** -10) * r.uniform(1, 1.01, 128))
                         for p in range(p0, p0 + n)])
        ref8.put_rows(kp[table[0, p0 // 64], 0], p0 % 64, rows, False)
    q = np.full((1, R, Hq, 128), 2.0 ** 15)
    vb = ref.bf16_round(r.standard_normal((1, 1, R, 128)))
    kb = ref.bf16_round(-(2.0 ** -10) * r.uniform(1, 1.01, vb.shape))
    one_sequence(sv, q, kp, vp, table, t, kb, vb, 128 ** -0.5, lost=lost)
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("mp", [6, 250])
@pytest.mark.parametrize("t,lost", [(64, 1), (130, 16), (200, 1), (1, 1), (128, 128), (200, 128), (304, 256), (300, 300), (384, 0)])
def test_attn_first_scores_not_finite(sv, t, lost, mp):
    """Up to whole steps of 128 keys whose scores are all -infinity come before the others (whose
    run they share in part: what it holds beside them is nothing, a score of 0)."""
    _far_below(sv, t, mp, lost)


def test_attn_sharp_softmax(sv):
    """Scores far apart (scale 20): the running maximum is rescaled again and
    again, and a single key takes the row."""
    run(sv, 1, 3, 4, 2, [700], scale=20.0, seed=6)


@pytest.mark.parametrize("mp", [4, 250])
def test_attn_rows_that_are_not_finite(sv, mp):
    """A NaN row of the cache that a sequence sees makes its rows NaN; beside it, and in
    block rows that another row does not see, it does nothing."""
    r = np.random.default_rng(11)
    B, R, Hq, H, P = 3, 3, 4, 2, 3 * mp + 1
    table = r.permutation(P)[: B * mp].reshape(B, mp).astype(np.int32)
    q = ref.bf16_round(r.standard_normal((B, R, Hq, 128)))
    kb, vb = ref.bf16_round(r.standard_normal((2, B, H, R, 128)))
    lens = [100, 130, 40]
    for which in ("k", "v", "kb", "vb", "q"):
        pools = {"k": random_pool(r, P, H), "v": random_pool(r, P, H)}
        a = {"q": q.copy(), "kb": kb.copy(), "vb": vb.copy()}
        if which in pools:
            ref8.put_rows(pools[which][table[1, 1], 1], 37, np.full((1, 128), np.nan), which == "v")
        elif which == "q":
            a["q"][1, 2, 3, 7] = np.inf
        else:
            a[which][1, 1, 2, 5] = np.nan
        clean = sv.verify_attn_q8(bf(q).cuda(), dev(pools["k"]), dev(pools["v"]), i32(table), i32([100, 101, 40]), bf(kb).cuda(),
                                  bf(vb).cuda())
        out = sv.verify_attn_q8(bf(a["q"]).cuda(), dev(pools["k"]), dev(pools["v"]), i32(table), i32(lens), bf(a["kb"]).cuda(),
                                bf(a["vb"]).cuda()).isnan()
        assert not bool(clean.isnan().any())
        want = np.zeros((B, R, Hq, 128), bool)
        if which in ("k", "v"):
            want[1, :, 2:] = True
        elif which == "kb":
            want[1, 2, 2:] = True
        elif which == "vb":
            want[1, 2, 2:, 5] = True
        else:
            want[1, 2, 3] = True
        assert np.array_equal(out.cpu().numpy(), want), which
    assert sv.get_device_error() == 0


def test_attn_query_rows_of_all_sizes(sv):
    """Query rows and block rows of K many powers of two apart keep their own precision, and
    V of the block its range."""
    r = np.random.default_rng(12)
    for mp in (3, 250):
        P, t, R, Hq = mp + 1, 150, 6, 8
        table = r.permutation(P)[:mp].reshape(1, mp).astype(np.int32)
        kp, vp = random_pool(r, P, 1), random_pool(r, P, 1)
        q = ref.bf16_round(r.standard_normal((1, R, Hq, 128)) * 10.0 ** np.arange(-24, 24).reshape(1, R, Hq, 1))
        kb, vb = ref.bf16_round(r.standard_normal((2, 1, 1, R, 128)))
        kb = ref.bf16_round(kb * 10.0 ** np.arange(-3, 3).reshape(1, 1, R, 1))
        out = sv.verify_attn_q8(bf(q).cuda(), dev(kp), dev(vp), i32(table), i32([t]), bf(kb).cuda(), bf(vb).cuda())[0].double().cpu().numpy()
        rows = lambda pool, is_v: ref8.get_rows(pool[table[0, :3]], is_v).transpose(1, 0, 2, 3).reshape(1, 192, 128)[:, :t]  # noqa: E731
        k, v = rows(kp, False), rows(vp, True)
        for j in range(R):
            for h in range(Hq):   # each row by itself
                one = q[0].copy()
                one[:] = one[j, h]
                want, wgt, big = ref.attention(one, k, v, kb[0], vb[0], None, 128 ** -0.5)
                bound = tol(want, wgt, big, units_of(one, k, kb[0], 128 ** -0.5), t + R,
                            lost_of(2.0 ** -5, v, vb[0], Hq))[j, h]
                assert np.all(np.abs(out[j, h] - want[j, h]) <= bound), (j, h)
    assert sv.get_device_error() == 0


def test_attn_bad_inputs_are_reported(sv):
    r = np.random.default_rng(0)
    kp, vp = random_pool(r, 3, 1), random_pool(r, 3, 1)
    q = ref.bf16_round(r.standard_normal((1, 2, 2, 128)))
    kb, vb = ref.bf16_round(r.standard_normal((2, 1, 1, 2, 128)))
    g = [dev(kp), dev(vp)]

    def call(table, ln, parent=None):
        return sv.verify_attn_q8(bf(q).cuda(), *g, i32(table), i32(ln), bf(kb).cuda(), bf(vb).cuda(),
                                 None if parent is None else i32(parent)).double().cpu().numpy()

    def check(got, k, v):
        want, wgt, big = ref.attention(q[0], k, v, kb[0], vb[0], None, 128 ** -0.5)
        lost = lost_of(2.0 ** -5, v, vb[0], 2)
        assert np.all(np.abs(got[0] - want) <= tol(want, wgt, big, units_of(q[0], k, kb[0], 128 ** -0.5), k.shape[1] + 2, lost))
    rows = lambda pool, pg, is_v: ref8.get_rows(pool[pg, 0], is_v).reshape(1, -1, 128)  # noqa: E731
    # a page outside the pool reads as zeros, on either side of a step
    for table, n, cut in (([[0, 7]], 100, None), ([[-1, 2]], 128, None)):
        got = call(table, [n])
        assert sv.get_device_error() == 0x80
        part = lambda p, is_v: np.concatenate([rows(p, [x], is_v) if 0 <= x < 3 else np.zeros((1, 64, 128)) for x in table[0]], 1)[:, :n]  # noqa: E731
        check(got, part(kp, False), part(vp, True))
    # a length past the table is clamped
    got = call([[0, 1]], [500])
    assert sv.get_device_error() == 4
    check(got, rows(kp, [0, 1], False), rows(vp, [0, 1], True))
    got = call([[0, 1]], [-5])
    assert sv.get_device_error() == 4
    check(got, np.zeros((1, 0, 128)), np.zeros((1, 0, 128)))
    # a malformed tree: the row sees itself and the cache
    call([[0, 1]], [64], parent=[[-1, 5]])
    assert sv.get_device_error() == 0x10


def _device_inputs(B, R, Hq, H, t, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mp = (t + 63) // 64
    P = B * mp
    pools = []
    for _ in range(2):
        p = torch.randint(0, 256, (P, H, ref8.Q8), generator=g, device="cuda", dtype=torch.uint8)
        p[(p & 127) == 127] = 0
        s = torch.exp2(torch.randint(-8, -5, (P, H, 4), generator=g, device="cuda").float())
        p[..., 8192:8208] = s.view(torch.uint8).view(P, H, 16)
        pools.append(p)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    table = torch.randperm(P, generator=g, device="cuda").to(torch.int32).view(B, mp)
    return mk(B, R, Hq, 128), pools, table, mk(B, H, R, 128), mk(B, H, R, 128)


@pytest.mark.parametrize("B,R,Hq,H,t", [
    (1, 1, 28, 4, 7744), (1, 1, 28, 4, 8192), (9, 1, 8, 8, 2160), (6, 23, 12, 2, 4000), (4, 1, 4, 1, 9400), (1, 38, 32, 8, 4111),
    (16, 3, 28, 4, 2286), (2, 1, 28, 4, 9927)])
def test_attn_many_steps(sv, B, R, Hq, H, t):
    """Runs long enough that every ring stage is used again: each group of 32 dims
    within twice what rounding P to bf16 and the output would leave at random (halves of
    2^-8 of their magnitudes, uniform: / sqrt(3)), its root mean square over the rows."""
    q, (kp, vp), table, kb, vb = _device_inputs(B, R, Hq, H, t, seed=t)
    lens = i32([t - 29 * b for b in range(B)])
    k, v = sv.kv_gather_q8(kp[None], vp[None], table, i32([0] * B), lens, t)
    out = sv.verify_attn_q8(q, kp, vp, table, lens, kb, vb)
    see = torch.cat([torch.arange(t, device="cuda")[None, :] < lens[:, None],
                     torch.ones(B, R, dtype=torch.bool, device="cuda")], 1)[:, None, :].repeat(1, R, 1)
    see[:, :, t:] = torch.tril(torch.ones(R, R, dtype=torch.bool, device="cuda"))
    for h in range(H):
        kk, vv = (torch.cat([c[0, :, h].double(), n[:, h].double()], 1) for c, n in ((k, kb), (v, vb)))
        z = torch.einsum("brgd,bkd->brgk", q.view(B, R, H, Hq // H, 128)[:, :, h].double(), kk) * 128 ** -0.5
        p = torch.softmax(z.masked_fill(~see[:, :, None, :], float("-inf")), -1)
        want = torch.einsum("brgk,bkd->brgd", p, vv)
        err = out.view(B, R, H, Hq // H, 128)[:, :, h].double() - want
        rms = lambda x: x.pow(2).reshape(B, R, Hq // H, 4, 32).mean((1, 2, 4)).sqrt()  # noqa: E731
        rounded = 2.0 ** -8 / 3 ** 0.5 * torch.sqrt(rms(want) ** 2 + torch.einsum("brgk,bkd->brgd", p ** 2, vv ** 2).reshape(
            B, R, Hq // H, 4, 32).mean((1, 2, 4)))
        assert bool((rms(err) <= 2 * rounded + 1e-6).all()), float((rms(err) / rounded).max())
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("B,R,Hq,H,t", [(9, 1, 8, 8, 2160), (6, 23, 12, 2, 16353), (1, 1, 28, 4, 7840), (14, 3, 12, 2, 4617)])
def test_attn_repeats_itself(sv, B, R, Hq, H, t):
    """The same call gives the same bits, with its inputs in L2 or not."""
    q, (kp, vp), table, kb, vb = _device_inputs(B, R, Hq, H, t, seed=t)
    lens = i32([t - 31 * b for b in range(B)])
    flush = torch.empty(2 ** 28, dtype=torch.uint8, device="cuda")
    want = sv.verify_attn_q8(q, kp, vp, table, lens, kb, vb)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        if i % 2:
            flush.fill_(i % 251)
        differ += (sv.verify_attn_q8(q, kp, vp, table, lens, kb, vb) != want).any()
    assert int(differ) == 0
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("B,R,Hq,H,t,tree", [(1, 5, 12, 2, 4096, False), (16, 9, 28, 4, 8192, False), (1, 65, 28, 4, 8192, True),
                                             (1, 1, 12, 2, 70000, False), (1, 20, 16, 2, 33000, False), (3, 100, 8, 1, 5000, True)])
def test_attn_full_size_against_torch64(sv, B, R, Hq, H, t, tree):
    q, (kp, vp), table, kb, vb = _device_inputs(B, R, Hq, H, t, seed=t + R)
    lens = [t - 37 * b for b in range(B)]
    par = None
    if tree:
        par = np.stack([synth.random_tree(R - 1, 8 if R < 70 else 20, 3, 5)] * B).astype(np.int32)
    out = sv.verify_attn_q8(q, kp, vp, table, i32(lens), kb, vb, None if par is None else i32(par))
    k, v = sv.kv_gather_q8(kp[None], vp[None], table, i32([0] * B), i32(lens), t)
    G = Hq // H
    for b in range(B):
        see = torch.zeros(R, R, dtype=torch.bool, device="cuda")
        for j in range(R):
            see[j, ref.row_path(par, b, j)] = True
        see = torch.cat([torch.ones(R, lens[b], dtype=torch.bool, device="cuda"), see], 1)
        for h in range(H):
            kk = torch.cat([k[0, b, h, :lens[b]], kb[b, h]]).double()
            vv = torch.cat([v[0, b, h, :lens[b]], vb[b, h]]).double()
            qq = q[b, :, h * G:(h + 1) * G].double()
            z = (qq @ kk.T) * 128 ** -0.5
            z = z.masked_fill(~see[:, None], float("-inf"))
            p = torch.softmax(z, -1)
            want, wgt = (p @ vv).cpu().numpy(), (p @ vv.abs()).cpu().numpy()
            big = float((qq.abs() @ kk.abs().T).max()) * 128 ** -0.5
            units = float(qq.abs().max() * kk.abs().sum(-1).max() + kb[b, h].double().abs().max() * qq.abs().sum(-1).max()) * 128 ** -0.5
            err = np.abs(out[b, :, h * G:(h + 1) * G].double().cpu().numpy() - want)
            # sums over a long context go through many partial sums: their error
            # grows with the square root of the terms, not with their number
            # (as does that of P's last steps)
            lost = 2.0 ** -21 * 16 * vv.pow(2).sum(0).sqrt().cpu().numpy() + 2.0 ** -25 * 2.0 ** -5
            bound = tol(want, wgt, big, units, int(16 * (lens[b] + R) ** 0.5), lost)
            assert np.all(err <= bound), (b, h, float((err / bound).max()))
    assert sv.get_device_error() == 0
