"""sv_kv_append_paged and sv_kv_append_q4: bit equality of the whole pools with
the plain form (so everything beside the new rows is also compared), and of the
rotation with float64 within its roundings."""
import numpy as np
import pytest
import torch

import _serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_sv_gb300 import binding
    return binding


def bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def make(seed, counts, length, H, D, max_pages, extra_rows=0, first=0, P=None):
    r = np.random.default_rng(seed)
    off = first + np.concatenate([[0], np.cumsum(counts)])
    N = int(off[-1]) + extra_rows
    B = len(counts)
    P = P or B * max_pages + 2
    table = r.permutation(P)[: B * max_pages].reshape(B, max_pages).astype(np.int32)
    k, v = ref.bf16_round(r.standard_normal((2, N, H, D)))
    return r, off.astype(np.int32), N, table, k, v, P


CASES = [
    # counts, lengths, H, rot, interleaved
    ([5], [0], 1, 128, False),
    ([1, 1, 1], [0, 63, 64], 2, 128, True),
    ([70, 0, 3, 130], [0, 5, 61, 100], 2, 64, False),
    ([9, 8, 7, 1, 0, 2], [7, 8, 1, 250, 9, 6], 1, 32, True),
    ([17, 33], [3, 120], 4, 16, False),
    ([40], [11], 2, 0, False),
    ([1] * 70, list(range(70)), 1, 128, False),
    ([0, 0, 0], [4, 5, 6], 1, 128, False),
]


@pytest.mark.parametrize("counts,length,H,rot,inter", CASES)
@pytest.mark.parametrize("q4", [False, True])
def test_append_matches_plain(sv, counts, length, H, rot, inter, q4):
    D, mp = 128, 5
    r, off, N, table, k, v, P = make(len(counts) * 7 + rot, counts, length, H, D, mp, extra_rows=3, first=2)
    rope = ref.rope_table(mp * 64, rot) if rot else None
    shape = (P, H, ref.Q4) if q4 else (P, H, 64, D)
    kp, vp = (r.integers(0, 256, shape).astype(np.uint8) for _ in range(2)) if q4 else \
        (r.integers(0, 65536, shape).astype(np.uint16) for _ in range(2))
    up = lambda a: torch.from_numpy(a).cuda() if q4 else torch.from_numpy(a.view(np.int16).copy()).cuda().view(torch.bfloat16)  # noqa: E731
    gk, gv = up(kp), up(vp)
    # K and V as slices of a fused projection's rows
    fused = torch.full((N, 3, H, D), 9.0, dtype=torch.bfloat16)
    fused[:, 1], fused[:, 2] = bf(k), bf(v)
    fused = fused.cuda().view(N, 3 * H, D)
    fn, plain = (sv.kv_append_q4, ref.append_q4) if q4 else (sv.kv_append_paged, ref.append_bf16)
    fn(fused[:, H:2 * H], fused[:, 2 * H:], i32(off), gk, gv, i32(table), i32(length),
       rope=None if rope is None else torch.from_numpy(rope).cuda(), interleaved=inter)
    wk, wv = plain(k, v, off, kp, vp, table, length, rope, inter, mp * 64)
    down = (lambda t: t.cpu().numpy()) if q4 else (lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16))
    assert np.array_equal(down(gk), wk)
    assert np.array_equal(down(gv), wv)
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_append_many_sequences(sv, q4):
    """Thousands of sequences, most of them without new rows: the search over the
    offsets takes three rounds."""
    B, H, D = 3000, 1, 128
    r = np.random.default_rng(1)
    counts = np.where(r.random(B) < 0.1, r.integers(1, 4, B), 0)
    counts[[0, -1]] = 2
    length = r.integers(0, 60, B).astype(np.int32)
    _, off, N, table, k, v, P = make(2, counts, length, H, D, 1, extra_rows=2, first=1)
    pools = [torch.zeros(*((P, H, ref.Q4) if q4 else (P, H, 64, D)), dtype=torch.uint8 if q4 else torch.bfloat16, device="cuda")
             for _ in range(2)]
    (sv.kv_append_q4 if q4 else sv.kv_append_paged)(bf(k).cuda(), bf(v).cuda(), i32(off), *pools, i32(table), i32(length))
    zero = np.zeros((P, H, ref.Q4) if q4 else (P, H, 64, D), np.uint8 if q4 else np.uint16)
    want = (ref.append_q4 if q4 else ref.append_bf16)(k, v, off, zero, zero, table, length, None, False, 64)
    down = (lambda t: t.cpu().numpy()) if q4 else (lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16))
    assert all(np.array_equal(down(g), w) for g, w in zip(pools, want))
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("D,H,rot,inter", [(8, 3, 0, False), (16, 1, 16, True), (64, 2, 48, False), (256, 1, 256, False), (40, 2, 32, True)])
def test_append_head_dims(sv, D, H, rot, inter):
    r, off, N, table, k, v, P = make(D, [37, 1], [60, 0], H, D, 2)
    rope = ref.rope_table(128, rot) if rot else None
    kp = r.integers(0, 65536, (P, H, 64, D)).astype(np.uint16)
    gk = torch.from_numpy(kp.view(np.int16).copy()).cuda().view(torch.bfloat16)
    gv = gk.clone()
    sv.kv_append_paged(bf(k).cuda(), bf(v).cuda(), i32(off), gk, gv, i32(table), i32([60, 0]),
                       rope=None if rope is None else torch.from_numpy(rope).cuda(), interleaved=inter)
    wk, wv = ref.append_bf16(k, v, off, kp, kp, table, [60, 0], rope, inter, 128)
    assert np.array_equal(gk.view(torch.int16).cpu().numpy().view(np.uint16), wk)
    assert np.array_equal(gv.view(torch.int16).cpu().numpy().view(np.uint16), wv)
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_at_far_positions(sv, inter):
    """Positions past 100000: the result is the formula's on the table's values,
    within a bf16 half step (2^-8) and three fp32 ones (2^-24) of the products."""
    t, n, rot = 100_003, 50, 128
    mp = (t + n + 63) // 64
    rope = ref.rope_table(mp * 64, rot)
    r = np.random.default_rng(5)
    k, v = ref.bf16_round(r.standard_normal((2, n, 1, 128)))
    table = np.arange(mp, dtype=np.int32)[None]
    gk = torch.zeros(mp, 1, 64, 128, dtype=torch.bfloat16, device="cuda")
    gv = gk.clone()
    sv.kv_append_paged(bf(k).cuda(), bf(v).cuda(), i32([0, n]), gk, gv, i32(table), i32([t]), rope=torch.from_numpy(rope).cuda(),
                       interleaved=inter)
    got = gk.view(-1, 128)[t:t + n].double().cpu().numpy()
    i, j = ref._pairs(rot, inter)
    c, s = rope[t:t + n, :64].astype(np.float64), rope[t:t + n, 64:].astype(np.float64)
    x = k[:, 0]
    want, size = np.zeros_like(x), np.zeros_like(x)
    want[:, i], want[:, j] = x[:, i] * c - x[:, j] * s, x[:, j] * c + x[:, i] * s
    size[:, i] = size[:, j] = np.abs(x[:, i]) + np.abs(x[:, j])
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -24 * 2 * size)
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_append_drops_what_has_no_place(sv, q4):
    """Rows past the capacity, past the rope table, on bad pages, of a negative
    length and of bad offsets are dropped and reported; the others land."""
    H, D, mp = 1, 128, 2
    counts = [10, 10, 10, 10]
    r, off, N, table, k, v, P = make(3, counts, None, H, D, mp)
    length = np.array([120, -3, 60, 90], np.int32)     # 0: past 128 after 8 rows; 1: negative; 3: past the rope table at 96
    table[2, 1] = P                                     # 2: its second page is outside the pool
    rope = ref.rope_table(96, 64)
    shape = (P, H, ref.Q4) if q4 else (P, H, 64, D)
    kp = r.integers(0, 256, shape).astype(np.uint8) if q4 else r.integers(0, 65536, shape).astype(np.uint16)
    up = lambda a: torch.from_numpy(a.copy()).cuda() if q4 else torch.from_numpy(a.view(np.int16).copy()).cuda().view(torch.bfloat16)  # noqa: E731
    down = (lambda t: t.cpu().numpy()) if q4 else (lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16))
    fn, plain = (sv.kv_append_q4, ref.append_q4) if q4 else (sv.kv_append_paged, ref.append_bf16)

    def check(off, length, rp, cap, flag):
        gk, gv = up(kp), up(kp)
        fn(bf(k).cuda(), bf(v).cuda(), i32(off), gk, gv, i32(table), i32(length), rope=None if rp is None else torch.from_numpy(rp).cuda())
        ok = [b for b in range(4) if length[b] >= 0 and 0 <= off[b] <= off[b + 1] <= N]
        o = np.array([off[b] for b in range(5)])
        wk, wv = kp, kp
        for b in ok:
            wk, wv = plain(k, v, o[b:b + 2], wk, wv, table[b:b + 1], length[b:b + 1], rp, False, cap)
        assert np.array_equal(down(gk), wk) and np.array_equal(down(gv), wv)
        assert sv.get_device_error() == flag

    check(off, length, rope, 96, 0x84)
    check(off, length, None, 128, 0x84)
    check(off, np.array([120, 3, 0, 90], np.int32), None, 128, 0x4)
    check(off, np.array([0, 3, 60, 90], np.int32), None, 128, 0x80)
    check(np.array([0, 10, 20, 30, N + 1], np.int32), np.array([0, 3, 0, 90], np.int32), None, 128, 0x01000000)


def test_append_q4_non_finite_group(sv):
    """A group with NaN or infinity reads back as NaN; its neighbours keep their
    values."""
    x = np.zeros((3, 1, 128))
    x[:] = np.linspace(-2, 2, 128)
    x = ref.bf16_round(x)
    k, v = bf(x), bf(x)
    k[1, 0, 40], v[2, 0, 100] = float("nan"), float("inf")
    kp = torch.zeros(1, 1, ref.Q4, dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    sv.kv_append_q4(k.cuda(), v.cuda(), i32([0, 3]), kp, vp, i32([[0]]), i32([6]))
    assert sv.get_device_error() == 1
    c, s = ref.quantise(x)
    want = ((c - 8) * s[..., None]).reshape(3, 128)
    wk, wv = want.copy(), want.copy()
    wk[1, 32:64], wv[2, 96:] = np.nan, np.nan
    assert np.array_equal(ref.get_rows(kp.cpu().numpy()[0, 0], False)[6:9], wk, equal_nan=True)
    assert np.array_equal(ref.get_rows(vp.cpu().numpy()[0, 0], True)[6:9], wv, equal_nan=True)
    g = sv.kv_gather_q4(kp[None], vp[None], i32([[0]]), i32([6]), i32([9]), 3)
    assert np.array_equal(g[0].double().cpu().numpy().reshape(3, 128), wk, equal_nan=True)
    assert np.array_equal(g[1].double().cpu().numpy().reshape(3, 128), wv, equal_nan=True)


def test_append_q4_extreme_magnitudes(sv):
    """Groups near the ends of bf16's range: the scale stays within its limits."""
    mags = [0.0, 2.0 ** -130, 2.0 ** -110, 2.0 ** -98, 1.0, 448.0, 2.0 ** 118, 2.0 ** 121, 3e38]
    r = np.random.default_rng(0)
    x = np.stack([ref.bf16_round(r.uniform(-1, 1, 128)) * m for m in mags])[:, None]
    x = bf(x).double().numpy()     # subnormals as bf16 holds them
    kp = torch.zeros(1, 1, ref.Q4, dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    sv.kv_append_q4(bf(x).cuda(), bf(x).cuda(), i32([0, len(mags)]), kp, vp, i32([[0]]), i32([0]))
    c, s = ref.quantise(x)
    want = ((c - 8) * s[..., None]).reshape(-1, 128)
    assert np.array_equal(ref.get_rows(kp.cpu().numpy()[0, 0], False)[:len(mags)], want)
    assert np.array_equal(ref.get_rows(vp.cpu().numpy()[0, 0], True)[:len(mags)], want)
    assert sv.get_device_error() == 0


def test_empty_append_does_nothing(sv):
    e = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    pool = torch.ones(3, 2, 64, 128, dtype=torch.bfloat16, device="cuda")
    sv.kv_append_paged(e, e, i32([0, 0]), pool, pool.clone(), i32([[0, 1]]), i32([3]))
    assert bool((pool == 1).all())


def test_padding_rows_are_not_read(sv):
    """Rows before the first sequence and behind the last are left alone.  The rows
    lie in host memory here, which takes many times a launch's time to read."""
    N, D = 1 << 17, 1024
    rows = torch.zeros(N, 1, D, dtype=torch.bfloat16).pin_memory()
    pages = N // 64
    kp, vp = (torch.zeros(pages, 1, 64, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, length = i32(np.arange(pages)[None]), i32([0])

    def us(off):
        off, best = i32(off), float("inf")
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            assert sv.lib.sv_kv_append_paged(rows.data_ptr(), rows.data_ptr(), D, D, N, off.data_ptr(), 1, 1, D, None, 0, 0, kp.data_ptr(),
                                             vp.data_ptr(), pages, table.data_ptr(), pages, length.data_ptr(), 0,
                                             torch.cuda.current_stream().cuda_stream) == 0
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 1e3)
        return best
    real, before, behind = us([0, N]), us([N - 3, N]), us([0, 3])
    assert max(before, behind) < real / 4, (real, before, behind)
    assert sv.get_device_error() == 0


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("off,N", [
    ([0, 20, 10, 30], 30), ([0, 4, 2], 4), ([5, 0, 0], 5), ([0, 100, 3, 130], 130), ([0, 3, 3, 1, 3], 9), ([0, 40, 40, 90, 20], 90),
    (list(range(70)) + [68], 69), ([0] * 150 + [9, 2] + [9] * 150, 9), ([0, 5, -7, 5], 5), ([0, 2, 1000, 9], 9)])
def test_offsets_that_fall_are_reported(sv, q4, off, N):
    """Wherever they fall.  Rows of the sequences whose offsets name rows land at
    their places or, where the offsets fall, nowhere."""
    H, D, B, mp = 1, 128, len(off) - 1, 3
    r = np.random.default_rng(N)
    k, v = ref.bf16_round(r.standard_normal((2, N, H, D)))
    P = B * mp
    table, length = r.permutation(P).reshape(B, mp).astype(np.int32), r.integers(0, 50, B).astype(np.int32)
    pools = [torch.zeros(*((P, H, ref.Q4) if q4 else (P, H, 64, D)), dtype=torch.uint8 if q4 else torch.bfloat16, device="cuda")
             for _ in range(2)]
    (sv.kv_append_q4 if q4 else sv.kv_append_paged)(bf(k).cuda(), bf(v).cuda(), i32(off), *pools, i32(table), i32(length))
    assert sv.get_device_error() == 0x01000000
    good = [b for b in range(B) if 0 <= off[b] <= off[b + 1] <= N]
    for pool, x, is_v in ((pools[0], k, False), (pools[1], v, True)):
        rows = ref.get_rows(pool.cpu().numpy(), is_v)[:, 0] if q4 else pool[:, 0].double().cpu().numpy()
        free = np.ones((P, 64), bool)
        if q4:
            c, s = ref.quantise(x[:, 0])
            x = ((c - 8) * s[..., None]).reshape(N, 1, D)
        for b in good:
            for i in range(off[b], off[b + 1]):
                p = int(length[b]) + i - off[b]
                got = rows[table[b, p // 64], p % 64]
                free[table[b, p // 64], p % 64] = False
                assert np.array_equal(got, x[i, 0]) or not got.any(), (b, i)
        assert not rows[free].any()
