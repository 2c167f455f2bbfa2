"""Plain numpy forms of the 8-bit cache's calls: what their documentation says,
written out run by run in float64."""
import numpy as np

import _serving_ref as ref

D, PAGE, RUN, Q8 = 128, 64, 16, 8320
E4M3 = np.array([(-1.0) ** (c >> 7) * (np.ldexp(c & 7, -9) if (c >> 3) & 15 == 0 else np.ldexp(8 + (c & 7), ((c >> 3) & 15) - 10))
                 for c in range(256)])
E4M3[[127, 255]] = np.nan


def _code_bytes(is_v):
    """[64, 128]: the byte of a (position, dim) in a block."""
    p, d = np.arange(PAGE)[:, None], np.arange(D)[None, :]
    return p // 8 * 1024 + d * 8 + p % 8 if is_v else p * 128 + (d // 16 ^ p % 8) * 16 + d % 16


def encode(x):
    """float64 -> e4m3 codes, to nearest, ties to even; +-448 past that, NaN 0x7f."""
    x = np.asarray(x, np.float64)
    y = np.clip(np.where(np.isnan(x), 0.0, x), -448, 448)
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    mag = np.abs(np.rint(y / step) * step)
    code = np.searchsorted(E4M3[:127], mag).astype(np.uint8)
    assert np.array_equal(E4M3[code], mag)
    return np.where(np.isnan(x), 0x7F, code | (np.signbit(x).astype(np.uint8) << 7)).astype(np.uint8)


def exponent(amax):
    """The least e in [-120, 119] with amax <= 448 * 2^e."""
    e = -120
    while e < 119 and amax > 448 * 2.0 ** e:
        e += 1
    return e


def scales(block):
    return np.ascontiguousarray(block[..., 8192:8208]).view("<f4").astype(np.float64)


def get_rows(block, is_v):
    """uint8 [..., 8320] -> float64 values [..., 64, 128]."""
    return E4M3[block[..., _code_bytes(is_v)]] * scales(block).repeat(RUN, -1)[..., None]


def put_rows(block, pos, rows, is_v):
    """Writes float64 rows [n, 128] to positions pos .. of a (page, head) block (uint8
    [8320], in place; they must lie in one run)."""
    at = _code_bytes(is_v)
    n, r = len(rows), pos // RUN
    assert (pos + n - 1) // RUN == r
    bad = ~np.isfinite(rows).all(-1)
    e = exponent(np.abs(rows[~bad]).max() if not bad.all() else 0.0)
    if pos % RUN:
        old = int(np.log2(scales(block)[r]))
        e = max(e, old)
        if e != old:
            k = at[r * RUN:pos]
            block[k] = encode(np.where(np.signbit(E4M3[block[k]]), -1.0, 1.0) * np.ldexp(np.abs(E4M3[block[k]]), old - e))
    with np.errstate(invalid="ignore"):
        block[at[pos:pos + n]] = encode(np.where(bad[:, None], np.nan, np.ldexp(np.where(bad[:, None], 0.0, rows), -e)))
    block[8192 + 4 * r:8196 + 4 * r] = np.frombuffer(np.float32(2.0 ** e).tobytes(), np.uint8)


def _write(pool, pages, length, rows, is_v):
    """rows [n, H, 128] to positions length .. of one sequence; pool [P, H, 8320] in place."""
    i = 0
    while i < len(rows):
        p = length + i
        n = min(len(rows) - i, RUN - p % RUN)
        pg = pages[p // PAGE]
        if 0 <= pg < pool.shape[0]:
            for h in range(rows.shape[1]):
                put_rows(pool[pg, h], p % PAGE, rows[i:i + n, h], is_v)
        i += n


def append(k, v, row_off, k_pool, v_pool, table, length, rope, interleaved, cap):
    kp, vp = k_pool.copy(), v_pool.copy()
    for b in range(len(length)):
        n = max(0, min(int(row_off[b + 1]), int(row_off[b]) + cap - int(length[b])) - int(row_off[b]))
        if length[b] < 0 or n == 0:
            continue
        at = np.arange(n) + int(row_off[b])
        kr = np.stack([ref.rotate(k[i], int(length[b]) + j, rope, interleaved) for j, i in enumerate(at)])
        _write(kp, table[b], int(length[b]), kr, False)
        _write(vp, table[b], int(length[b]), v[at], True)
    return kp, vp


def commit(k_pool, v_pool, table, k_blk, v_blk, path, n_acc, length):
    """pools uint8 [L, P, H, 8320], blocks float64 [L, B, H, R, D]."""
    kp, vp, ln = k_pool.copy(), v_pool.copy(), length.copy()
    for b in range(len(length)):
        rows = path[b, :n_acc[b] + 1]
        for a in range(k_blk.shape[0]):
            _write(kp[a], table[b], int(length[b]), k_blk[a, b][:, rows].transpose(1, 0, 2), False)
            _write(vp[a], table[b], int(length[b]), v_blk[a, b][:, rows].transpose(1, 0, 2), True)
        ln[b] += n_acc[b] + 1
    return kp, vp, ln


def undefined(shape, table, length, end, pages):
    """True at the codes [P, H, 64] (positions) that hold nothing defined after rows
    were written up to each end: those behind it in its run."""
    u = np.zeros(shape, bool)
    for b in range(len(length)):
        if end[b] > length[b] and end[b] % RUN:
            pg = table[b, end[b] // PAGE]
            if 0 <= pg < pages:
                u[pg, :, end[b] % PAGE:(end[b] // RUN * RUN + RUN - 1) % PAGE + 1] = True
    return u


def same_pool(got, want, undef, is_v):
    """Pools [..., P, H, 8320] equal but for the positions where undef [P, H, 64]."""
    at = _code_bytes(is_v)
    g, w = got[..., at], want[..., at]
    keep = np.broadcast_to(~undef[..., None], g.shape)
    return np.array_equal(g[keep], w[keep]) and np.array_equal(got[..., 8192:], want[..., 8192:])


def gather(pool, table, start, length, n, is_v):
    """uint8 [L, P, H, 8320] -> float64 [L, B, H, n, D]."""
    L, P, H = pool.shape[:3]
    out = np.zeros((L, len(start), H, n, D))
    for b in range(len(start)):
        for i in range(n):
            p = int(start[b]) + i
            if 0 <= start[b] and p < length[b] and 0 <= table[b, p // PAGE] < P:
                out[:, b, :, i] = get_rows(pool[:, table[b, p // PAGE]], is_v)[:, :, p % PAGE]
    return out
