"""The 4-bit cache on the GPU: commit and gather bit for bit against the plain
forms, attention within the roundings it makes."""
import numpy as np
import pytest
import torch

import _serving_ref as ref
from speculative_decoding_verification_sv_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_sv_gb300 import binding
    return binding


def bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def random_pool(r, *lead, is_v):
    """Blocks of random codes (1..15) whose scales are what the library writes."""
    pool = r.integers(0, 256, (*lead, ref.Q4)).astype(np.uint8)
    lo, hi = pool[..., :4096] & 15, pool[..., :4096] >> 4
    pool[..., :4096] = np.maximum(lo, 1) | (np.maximum(hi, 1) << 4)
    s = np.ldexp(r.integers(8, 16, (*lead, 256)) / 8.0, r.integers(-4, -1, (*lead, 256)))
    pool[..., 4096:] = ref.f64_to_bits(s).astype("<u2").view(np.uint8).reshape(*lead, 512)
    return pool


# ---------------------------------------------------------------------------
# commit, gather
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("L,B,H,R,lens,tree", [
    (1, 1, 1, 1, [0], False), (3, 3, 2, 5, [59, 64, 7], False), (2, 4, 1, 20, [44, 0, 63, 101], True), (5, 1, 4, 9, [120], False),
    (1, 2, 1, 128, [1, 62], False)])
def test_commit_matches_plain(sv, L, B, H, R, lens, tree):
    r = np.random.default_rng(R * 10 + L)
    mp, P = 4, B * 4 + 2
    table = r.permutation(P)[: B * mp].reshape(B, mp).astype(np.int32)
    kp, vp = random_pool(r, L, P, H, is_v=False), random_pool(r, L, P, H, is_v=True)
    kb, vb = ref.bf16_round(r.standard_normal((2, L, B, H, R, 128)))
    n_acc = r.integers(0, R, B).astype(np.int32)
    n_acc[0] = R - 1
    path = np.full((B, R), -1, np.int32)
    for b in range(B):
        path[b, :n_acc[b] + 1] = np.sort(r.permutation(R)[:n_acc[b] + 1]) if tree else np.arange(n_acc[b] + 1)
    ln = np.array(lens, np.int32)
    gk, gv, gl = torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), i32(ln)
    sv.kv_commit_q4(gk, gv, i32(table), bf(kb).cuda(), bf(vb).cuda(), i32(path), i32(n_acc), gl)
    wk, wv, wl = ref.commit_q4(kp, vp, table, kb, vb, path, n_acc, ln)
    assert np.array_equal(gl.cpu().numpy(), wl)
    assert np.array_equal(gk.cpu().numpy(), wk)
    assert np.array_equal(gv.cpu().numpy(), wv)
    assert sv.get_device_error() == 0


def test_commit_leaves_bad_sequences_untouched(sv):
    r = np.random.default_rng(4)
    L, B, H, R, mp = 2, 5, 1, 6, 2
    P = B * mp
    table = np.arange(P, dtype=np.int32).reshape(B, mp)
    kp, vp = random_pool(r, L, P, H, is_v=False), random_pool(r, L, P, H, is_v=True)
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
        gk, gv, gl = torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), i32(ln)
        sv.kv_commit_q4(gk, gv, i32(tb), bf(kb).cuda(), bf(vb).cuda(), i32(pa), i32(na), gl)
        assert sv.get_device_error() == flag
        ok = [b for b in range(B) if b not in bad]
        wk, wv, wl = ref.commit_q4(kp, vp, tb[ok], kb[:, ok], vb[:, ok], pa[ok], na[ok], ln[ok])
        assert np.array_equal(gk.cpu().numpy(), wk) and np.array_equal(gv.cpu().numpy(), wv)
        assert gl.cpu().numpy()[ok].tolist() == wl.tolist() and gl.cpu().numpy()[bad].tolist() == ln[bad].tolist()


@pytest.mark.parametrize("L,B,H,n,start,lens", [
    (1, 1, 1, 1, [0], [1]), (2, 3, 2, 130, [0, 61, 7], [256, 100, 0]), (1, 4, 1, 9, [5, 250, 255, 64], [256, 256, 256, 66]),
    (3, 1, 1, 256, [0], [200]), (1, 1, 2, 40, [300], [256])])
def test_gather_matches_plain(sv, L, B, H, n, start, lens):
    r = np.random.default_rng(n)
    mp, P = 4, B * 4 + 1
    table = r.permutation(P)[: B * mp].reshape(B, mp).astype(np.int32)
    kp, vp = random_pool(r, L, P, H, is_v=False), random_pool(r, L, P, H, is_v=True)
    k, v = sv.kv_gather_q4(torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), i32(table), i32(start), i32(lens), n)
    assert np.array_equal(k.double().cpu().numpy(), ref.gather_q4(kp, table, start, lens, n, False))
    assert np.array_equal(v.double().cpu().numpy(), ref.gather_q4(vp, table, start, lens, n, True))
    assert sv.get_device_error() == 0


def test_gather_bad_inputs(sv):
    r = np.random.default_rng(0)
    kp = random_pool(r, 1, 4, 1, is_v=False)
    g = torch.from_numpy(kp).cuda()
    table = np.array([[0, 9], [1, 2]], np.int32)
    k, _ = sv.kv_gather_q4(g, g, i32(table), i32([60, 60]), i32([128, 128]), 8)
    assert sv.get_device_error() == 0x80
    assert np.array_equal(k.double().cpu().numpy(), ref.gather_q4(kp, table, [60, 60], [128, 128], 8, False))
    k, _ = sv.kv_gather_q4(g, g, i32([[0, 1], [1, 2]]), i32([-1, 120]), i32([128, 200]), 16)
    assert sv.get_device_error() == 4
    want = ref.gather_q4(kp, np.array([[0, 1], [1, 2]]), [-1, 120], [128, 128], 16, False)
    assert np.array_equal(k.double().cpu().numpy(), want)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def tol(want, wgt, big, keys):
    """P and the output are each rounded to bf16, a half step of 2^-8 of what
    they are; sums of 128 products move a score by at most 130 * 2^-22 of their
    magnitudes (p by that factor, twice: numerator and denominator), the
    exponentials by 2^-20; sums over the keys and their rescalings by 2^-22 a
    term."""
    p = 2.0 ** -8 + 2 * (130 * 2.0 ** -22 * big + 2.0 ** -20) + 2 * keys * 2.0 ** -22
    return 2.0 ** -8 * np.abs(want) + 1.01 * p * wgt + 1e-30


def run(sv, B, R, Hq, H, lens, parent=None, scale=None, seed=0, mp=None, **kw):
    r = np.random.default_rng(seed)
    mp = mp or max(1, (max(lens) + 63) // 64)
    P = B * mp + 1
    table = r.permutation(P)[: B * mp].reshape(B, mp).astype(np.int32)
    kp, vp = random_pool(r, P, H, is_v=False), random_pool(r, P, H, is_v=True)
    # positions at and past the length hold scales that are NaN or infinite
    for b in range(B):
        for p in range(lens[b], mp * 64):
            for h in range(H):
                for pool, is_v, bits in ((kp, False, 0x7FC0), (vp, True, 0x7F80)):
                    for g in range(4):
                        at = ref._scale_byte(is_v, p % 64, g)
                        pool[table[b, p // 64], h, at:at + 2] = [bits & 255, bits >> 8]
    q = ref.bf16_round(r.standard_normal((B, R, Hq, 128)))
    kb, vb = ref.bf16_round(r.standard_normal((2, B, H, R, 128)))
    out = sv.verify_attn_q4(bf(q).cuda(), torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), i32(table), i32(lens), bf(kb).cuda(),
                            bf(vb).cuda(), None if parent is None else i32(parent), scale=scale, **kw)
    got = out.double().cpu().numpy()
    for b in range(B):
        n = (lens[b] + 63) // 64
        rows = lambda pool, is_v: ref.get_rows(pool[table[b, :n]], is_v).transpose(1, 0, 2, 3).reshape(H, n * 64, 128)[:, :lens[b]]  # noqa: E731
        want, wgt, big = ref.attention(q[b], rows(kp, False), rows(vp, True), kb[b], vb[b], None if parent is None else parent[b:b + 1],
                                       scale or 128 ** -0.5)
        err = np.abs(got[b] - want)
        bound = tol(want, wgt, big, lens[b] + R)
        assert np.all(err <= bound), (b, float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())
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


@pytest.mark.parametrize("B,R,Hq,H,lens,is_tree", [
    (1, 5, 12, 2, [1000], False), (3, 9, 28, 4, [63, 0, 700], False), (2, 65, 28, 4, [130, 5], True), (1, 1, 1, 1, [1], False),
    (2, 20, 16, 2, [640, 129], True)])
def test_attn_split_over_all_sms(sv, B, R, Hq, H, lens, is_tree):
    """A long table (its capacity sets how the work is split): the pages are laid
    end to end over the SMs, and units in several of them joined by the second
    kernel.  Shorter tables give each unit a cluster of CTAs."""
    mp = 250
    assert sv.verify_attn_q4_workspace(B, R, Hq, H, 128, mp * 64) > 0
    assert sv.verify_attn_q4_workspace(1, 5, 12, 2, 128, 4096) == 0
    r = np.random.default_rng(R)
    par = np.full((B, R), -1, np.int32)
    for j in range(1, R):
        par[:, j] = r.integers(max(0, j - 6), j, B)
    run(sv, B, R, Hq, H, lens, parent=par if is_tree else None, seed=R, mp=mp)
    run(sv, B, R, Hq, H, lens, parent=par if is_tree else None, seed=R, mp=mp, scale=9.0)


def test_attn_references_far_below(sv):
    """The first key's score far below the others': the sums leave their range
    and the run is done again with the running maxima, in a cluster and over all
    SMs."""
    r = np.random.default_rng(8)
    for mp in (9, 250):
        P, t, R, Hq = mp + 1, 520, 3, 4
        table = r.permutation(P)[:mp].reshape(1, mp).astype(np.int32)
        kp, vp = random_pool(r, P, 1, is_v=False), random_pool(r, P, 1, is_v=True)
        q = np.abs(ref.bf16_round(r.standard_normal((1, R, Hq, 128)))) + 0.5
        kb, vb = ref.bf16_round(r.standard_normal((2, 1, 1, R, 128)))
        ref.put_row(kp[table[0, 0], 0], 0, np.full(128, -6.0), False)
        for p in (70, 300, 519):
            ref.put_row(kp[table[0, p // 64], 0], p % 64, np.full(128, 1.0 + p / 200), False)
        q = ref.bf16_round(q)
        out = sv.verify_attn_q4(bf(q).cuda(), torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), i32(table), i32([t]),
                                bf(kb).cuda(), bf(vb).cuda(), scale=0.5)
        rows = lambda pool, is_v: ref.get_rows(pool[table[0, :9]], is_v).transpose(1, 0, 2, 3).reshape(1, 576, 128)[:, :t]  # noqa: E731
        want, wgt, big = ref.attention(q[0], rows(kp, False), rows(vp, True), kb[0], vb[0], None, 0.5)
        assert np.all(np.abs(out[0].double().cpu().numpy() - want) <= tol(want, wgt, big, t + R))
        assert sv.get_device_error() == 0


@pytest.mark.parametrize("t,H,mp", [(0, 1, 1), (0, 2, 9), (0, 2, 250), (448, 1, 7), (512, 4, 250), (70, 2, 40)])
def test_attn_malformed_row_sees_the_cache_and_itself(sv, t, H, mp):
    """Block row 0, which a malformed row does not see, has a score 739 powers of two
    above that row's own, and that one 739 above the cache's; also where a CTA's run
    holds the block alone (7 pages in a cluster of 8; 8 pages and the block laid end to
    end in fours)."""
    r = np.random.default_rng(t)
    P, R = mp + 1, 2
    table = r.permutation(P)[:mp].reshape(1, mp).astype(np.int32)
    kp, vp = random_pool(r, P, H, is_v=False), random_pool(r, P, H, is_v=True)
    row = np.zeros(ref.Q4, np.uint8)
    for p in range(64):
        ref.put_row(row, p, np.full(128, -6.0), False)
    kp[:] = row
    q = np.full((1, R, H, 128), 2.0)
    kb, vb = ref.bf16_round(r.standard_normal((2, 1, H, R, 128)))
    kb[0, :, 0], kb[0, :, 1] = 2.0, -2.0
    out = sv.verify_attn_q4(bf(q).cuda(), torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), i32(table), i32([t]), bf(kb).cuda(),
                            bf(vb).cuda(), i32([[-1, 7]]), scale=0.5)
    assert sv.get_device_error() == 0x10
    n = (t + 63) // 64
    rows = lambda pool, is_v: ref.get_rows(pool[table[0, :n]], is_v).transpose(1, 0, 2, 3).reshape(H, n * 64, 128)[:, :t]  # noqa: E731
    want, wgt, big = ref.attention(q[0], rows(kp, False), rows(vp, True), kb[0], vb[0], np.array([[-1, -1]]), 0.5)
    assert np.all(np.abs(out[0].double().cpu().numpy() - want) <= tol(want, wgt, big, t + R))


def _far_below(sv, t, mp, lost):
    """The scores of the first `lost` positions are -infinity (products past fp32),
    all others hundreds of powers of two below 0."""
    r = np.random.default_rng(t + mp)
    P, R, Hq = mp + 1, 3, 4
    table = r.permutation(P)[:mp].reshape(1, mp).astype(np.int32)
    kp, vp = random_pool(r, P, 1, is_v=False), random_pool(r, P, 1, is_v=True)
    for p in range(t):
        row = np.full(128, -(2.0 ** 118)) if p < lost else ref.bf16_round(-(2.0 ** -10) * r.uniform(1, 1.01, 128))
        ref.put_row(kp[table[0, p // 64], 0], p % 64, row, False)
    q = np.full((1, R, Hq, 128), 2.0 ** 15)
    kb, vb = ref.bf16_round(r.standard_normal((2, 1, 1, R, 128)))
    kb = ref.bf16_round(-(2.0 ** -10) * r.uniform(1, 1.01, kb.shape))
    out = sv.verify_attn_q4(bf(q).cuda(), torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), i32(table), i32([t]), bf(kb).cuda(),
                            bf(vb).cuda())
    n = (t + 63) // 64
    rows = lambda pool, is_v: ref.get_rows(pool[table[0, :n]], is_v).transpose(1, 0, 2, 3).reshape(1, n * 64, 128)[:, lost:t]  # noqa: E731
    want, wgt, big = ref.attention(q[0], rows(kp, False), rows(vp, True), kb[0], vb[0], None, 128 ** -0.5)
    assert np.all(np.abs(out[0].double().cpu().numpy() - want) <= tol(want, wgt, big, t + R))
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("mp", [4, 250])
@pytest.mark.parametrize("t", [64, 130, 200])
def test_attn_first_score_not_finite(sv, t, mp):
    _far_below(sv, t, mp, 1)


@pytest.mark.parametrize("mp", [6, 250])
@pytest.mark.parametrize("t,lost", [(1, 1), (128, 128), (200, 128), (300, 256), (300, 300), (384, 0)])
def test_attn_first_steps_not_finite(sv, t, lost, mp):
    """Whole steps of 128 keys whose scores are all -infinity come before the others."""
    _far_below(sv, t, mp, lost)


def test_attn_sharp_softmax(sv):
    """Scores far apart (scale 20): the running maximum is rescaled again and
    again, and a single key takes the row."""
    run(sv, 1, 3, 4, 2, [700], scale=20.0, seed=6)


def test_attn_bad_inputs_are_reported(sv):
    r = np.random.default_rng(0)
    kp, vp = random_pool(r, 3, 1, is_v=False), random_pool(r, 3, 1, is_v=True)
    q = ref.bf16_round(r.standard_normal((1, 2, 2, 128)))
    kb, vb = ref.bf16_round(r.standard_normal((2, 1, 1, 2, 128)))
    g = [torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda()]

    def call(table, ln, parent=None):
        return sv.verify_attn_q4(bf(q).cuda(), *g, i32(table), i32(ln), bf(kb).cuda(), bf(vb).cuda(),
                                 None if parent is None else i32(parent)).double().cpu().numpy()

    def plain(k, v, parent=None):
        return ref.attention(q[0], k, v, kb[0], vb[0], parent, 128 ** -0.5)
    rows = lambda pool, pg, is_v: ref.get_rows(pool[pg, 0], is_v).reshape(1, -1, 128)  # noqa: E731
    # a page outside the pool reads as zeros
    got = call([[0, 7]], [100])
    assert sv.get_device_error() == 0x80
    k, v = (np.concatenate([rows(p, [0], is_v), np.zeros((1, 36, 128))], 1) for p, is_v in ((kp, False), (vp, True)))
    want, wgt, big = plain(k, v)
    assert np.all(np.abs(got[0] - want) <= tol(want, wgt, big, 102))
    # a length past the table is clamped
    got = call([[0, 1]], [500])
    assert sv.get_device_error() == 4
    want, wgt, big = plain(rows(kp, [0, 1], False), rows(vp, [0, 1], True))
    assert np.all(np.abs(got[0] - want) <= tol(want, wgt, big, 130))
    got = call([[0, 1]], [-5])
    assert sv.get_device_error() == 4
    want, wgt, big = plain(np.zeros((1, 0, 128)), np.zeros((1, 0, 128)))
    assert np.all(np.abs(got[0] - want) <= tol(want, wgt, big, 2))
    # a malformed tree: the row sees itself and the cache
    call([[0, 1]], [64], parent=[[-1, 5]])
    assert sv.get_device_error() == 0x10


@pytest.mark.parametrize("B,R,Hq,H,t", [
    (1, 1, 28, 4, 7744), (1, 1, 28, 4, 8192), (9, 1, 8, 8, 2160), (6, 23, 12, 2, 4000), (4, 1, 4, 1, 9400), (1, 38, 32, 8, 4111),
    (16, 3, 28, 4, 2286), (2, 1, 28, 4, 9927)])
def test_attn_many_steps(sv, B, R, Hq, H, t):
    """Runs long enough that every ring stage is used again: each group of 32 dims
    within twice what rounding P and the output leave at random (halves of 2^-8 of
    their magnitudes, uniform: / sqrt(3)), its root mean square over the rows."""
    q, (kp, vp), table, kb, vb = _device_inputs(B, R, Hq, H, t, seed=t)
    lens = i32([t - 29 * b for b in range(B)])
    k, v = sv.kv_gather_q4(kp[None], vp[None], table, i32([0] * B), lens, t)
    out = sv.verify_attn_q4(q, kp, vp, table, lens, kb, vb)
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
    """The same call gives the same bits, with its inputs in L2 or not (the last
    product's end has to be waited for however late it is)."""
    q, (kp, vp), table, kb, vb = _device_inputs(B, R, Hq, H, t, seed=t)
    lens = i32([t - 31 * b for b in range(B)])
    flush = torch.empty(2 ** 28, dtype=torch.uint8, device="cuda")
    want = sv.verify_attn_q4(q, kp, vp, table, lens, kb, vb)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        if i % 2:
            flush.fill_(i % 251)
        differ += (sv.verify_attn_q4(q, kp, vp, table, lens, kb, vb) != want).any()
    assert int(differ) == 0
    assert sv.get_device_error() == 0


def _device_inputs(B, R, Hq, H, t, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mp = (t + 63) // 64
    P = B * mp
    codes = lambda: torch.randint(0, 256, (P, H, ref.Q4), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    pools = []
    for _ in range(2):
        p = codes()
        s = (torch.randint(8, 16, (P, H, 256), generator=g, device="cuda") / 64.0).to(torch.bfloat16)
        p[..., 4096:] = s.view(torch.uint8).view(P, H, 512)
        pools.append(p)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    table = torch.randperm(P, generator=g, device="cuda").to(torch.int32).view(B, mp)
    return mk(B, R, Hq, 128), pools, table, mk(B, H, R, 128), mk(B, H, R, 128)


@pytest.mark.parametrize("B,R,Hq,H,t,tree", [(1, 5, 12, 2, 4096, False), (16, 9, 28, 4, 8192, False), (1, 65, 28, 4, 8192, True),
                                             (1, 1, 12, 2, 70000, False), (1, 20, 16, 2, 33000, False), (3, 100, 8, 1, 5000, True)])
def test_attn_full_size_against_torch64(sv, B, R, Hq, H, t, tree):
    q, (kp, vp), table, kb, vb = _device_inputs(B, R, Hq, H, t, seed=t + R)
    lens = [t - 37 * b for b in range(B)]
    par = None
    if tree:
        par = np.stack([synth.random_tree(R - 1, 8 if R < 70 else 20, 3, 5)] * B).astype(np.int32)
    out = sv.verify_attn_q4(q, kp, vp, table, i32(lens), kb, vb, None if par is None else i32(par))
    k, v = sv.kv_gather_q4(kp[None], vp[None], table, i32([0] * B), i32(lens), t)
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
            err = np.abs(out[b, :, h * G:(h + 1) * G].double().cpu().numpy() - want)
            # sums over a long context go through many partial sums: their error
            # grows with the square root of the terms, not with their number
            bound = tol(want, wgt, big, int(16 * (lens[b] + R) ** 0.5))
            assert np.all(err <= bound), (b, h, float((err / bound).max()))
    assert sv.get_device_error() == 0
