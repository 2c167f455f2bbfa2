"""Plain numpy forms of the paged append, the 4-bit cache and the sampling
controls: what each call's documentation says, written out element by element
or in float64.  bf16 is held as float64 values or as raw uint16 bits."""
import numpy as np

D, PAGE, Q4 = 128, 64, 4608
SHIFT = np.array([4 * (e // 2) + 16 * (e % 2) for e in range(8)])


def bf16_round(x):
    """float -> nearest bf16 (ties to even), as float64 (normal range)."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256) / 256, e)


def bits_to_f64(b):
    return (np.asarray(b, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bits(x):
    """Values that are bf16 exactly -> their bits."""
    return (np.asarray(x, np.float64).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def rope_table(positions, rot, base=10000.0):
    f = base ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(positions)[:, None] * f[None, :]
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(rows, pos, rope, interleaved):
    """float64 bf16-valued rows [..., D] at positions pos (broadcast over the
    leading axes) -> rotated, each product and sum rounded to fp32, then bf16."""
    if rope is None:
        return rows
    rot = rope.shape[1]
    i, j = _pairs(rot, interleaved)
    x = rows.astype(np.float32)
    c, s = rope[pos][..., :rot // 2], rope[pos][..., rot // 2:]
    y = x.copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return bf16_round(y)


def quantise(rows):
    """float64 [..., 128] -> (codes [..., 4, 32] int, scales [..., 4] float64)."""
    g = rows.reshape(*rows.shape[:-1], 4, 32)
    with np.errstate(invalid="ignore"):
        a = np.abs(g).max(-1)
        bad = ~np.isfinite(g).all(-1)
        a = np.where(bad, 1.0, a)
        m, e = np.frexp(a / 7)
        s = np.where(a > 0, np.clip(np.ldexp(np.ceil(m * 16) / 16, e), 2.0 ** -100, 2.0 ** 118), 0.0)
        gg = np.where(bad[..., None], 0.0, g)
        q = np.clip(np.rint(gg / np.where(s > 0, s, 1.0)[..., None]), -7, 7).astype(int)
    return q + 8, np.where(bad, np.nan, s)


def _word_slot(is_v, pos, d):
    """(byte offset of the word, bit) of one element of a block."""
    if is_v:
        return (pos // 8) * 512 + d * 4, int(SHIFT[pos % 8])
    return (d // 32) * 1024 + pos * 16 + (d % 32) // 8 * 4, int(SHIFT[d % 8])


def _scale_byte(is_v, pos, g):
    return 4096 + (g * 128 + pos * 2 if is_v else pos * 8 + g * 2)


def put_row(block, pos, row, is_v):
    """Quantises a float64 row [128] into position pos of a (page, head) block
    (uint8 [4608], in place)."""
    c, s = quantise(row)
    for g in range(4):
        b = np.uint16(0x7FC0) if np.isnan(s[g]) else f64_to_bits(s[g])
        block[_scale_byte(is_v, pos, g):][:2] = np.frombuffer(np.uint16(b).tobytes(), np.uint8)
    for d in range(D):
        at, bit = _word_slot(is_v, pos, d)
        k = at + bit // 8
        block[k] = (block[k] & (0xFF ^ (15 << bit % 8))) | (int(c[d // 32, d % 32]) << bit % 8)


def get_rows(block, is_v):
    """uint8 [..., 4608] -> float64 values [..., 64, 128]."""
    p, d = np.arange(PAGE)[:, None], np.arange(D)[None, :]
    e = (p if is_v else d) % 8 + 0 * (p + d)
    bit = SHIFT[e]
    byte = (p // 8 * 512 + d * 4 if is_v else d // 32 * 1024 + p * 16 + d % 32 // 8 * 4) + bit // 8
    c = (block[..., byte].astype(int) >> (bit % 8)) & 15
    sb = 4096 + (d // 32 * 128 + p * 2 if is_v else p * 8 + d // 32 * 2)
    s = bits_to_f64(block[..., sb].astype(np.uint16) | (block[..., sb + 1].astype(np.uint16) << 8))
    return (c - 8) * s


def places(row_off, length, table, cap):
    """(row, sequence, position, page) of each appended row that has a place."""
    got = []
    for b in range(len(length)):
        for i in range(row_off[b], row_off[b + 1]):
            p = int(length[b]) + i - int(row_off[b])
            if 0 <= p < cap:
                got.append((i, b, p, int(table[b, p // PAGE])))
    return got


def append_bf16(k, v, row_off, k_pool, v_pool, table, length, rope, interleaved, cap):
    """k, v float64 [N, H, D]; pools uint16 bits [P, H, 64, D]; returns new pools."""
    kp, vp = k_pool.copy(), v_pool.copy()
    for i, b, p, pg in places(row_off, length, table, cap):
        if 0 <= pg < kp.shape[0]:
            kp[pg, :, p % PAGE] = f64_to_bits(rotate(k[i], p, rope, interleaved))
            vp[pg, :, p % PAGE] = f64_to_bits(v[i])
    return kp, vp


def append_q4(k, v, row_off, k_pool, v_pool, table, length, rope, interleaved, cap):
    kp, vp = k_pool.copy(), v_pool.copy()
    for i, b, p, pg in places(row_off, length, table, cap):
        if 0 <= pg < kp.shape[0]:
            kr = rotate(k[i], p, rope, interleaved)
            for h in range(k.shape[1]):
                put_row(kp[pg, h], p % PAGE, kr[h], False)
                put_row(vp[pg, h], p % PAGE, v[i, h], True)
    return kp, vp


def commit_q4(k_pool, v_pool, table, k_blk, v_blk, path, n_acc, length):
    """pools uint8 [L, P, H, 4608], blocks float64 [L, B, H, R, D]."""
    kp, vp, ln = k_pool.copy(), v_pool.copy(), length.copy()
    L, B, H = k_blk.shape[:3]
    for b in range(B):
        for i in range(n_acc[b] + 1):
            p = int(length[b]) + i
            pg = table[b, p // PAGE]
            for l in range(L):
                for h in range(H):
                    put_row(kp[l, pg, h], p % PAGE, k_blk[l, b, h, path[b, i]], False)
                    put_row(vp[l, pg, h], p % PAGE, v_blk[l, b, h, path[b, i]], True)
        ln[b] += n_acc[b] + 1
    return kp, vp, ln


def gather_q4(pool, table, start, length, n, is_v):
    """uint8 [L, P, H, 4608] -> float64 [L, B, H, n, D]."""
    L, P, H = pool.shape[:3]
    out = np.zeros((L, len(start), H, n, D))
    for b in range(len(start)):
        for i in range(n):
            p = int(start[b]) + i
            if 0 <= start[b] and p < length[b] and 0 <= table[b, p // PAGE] < P:
                out[:, b, :, i] = get_rows(pool[:, table[b, p // PAGE]], is_v)[:, :, p % PAGE]
    return out


def row_path(parent, b, j):
    """Block rows that row j sees: itself and its ancestors (or 0..j)."""
    if parent is None:
        return list(range(j + 1))
    got = []
    while j >= 0:
        got.append(j)
        j = int(parent[b, j])
    return got


def attention(q, k_ctx, v_ctx, k_blk, v_blk, parent, scale):
    """One sequence in float64: q [R, Hq, D], contexts [H, t, D], blocks [H, R, D].
    Returns (out, weight), weight = sum p |v| / sum p, what the rounding of P
    is relative to, and the largest score bound scale * sum |q||k|."""
    R, Hq, _ = q.shape
    H = k_blk.shape[0]
    G, t = Hq // H, k_ctx.shape[1]
    out, wgt, big = np.zeros_like(q), np.zeros_like(q), 0.0
    for j in range(R):
        see = row_path(parent, 0, j)
        for h in range(Hq):
            k = np.concatenate([k_ctx[h // G], k_blk[h // G][see]])
            v = np.concatenate([v_ctx[h // G], v_blk[h // G][see]])
            z = scale * (k @ q[j, h])
            p = np.exp(z - z.max())
            out[j, h], wgt[j, h] = p @ v / p.sum(), p @ np.abs(v) / p.sum()
            big = max(big, scale * float((np.abs(k) @ np.abs(q[j, h])).max()))
    return out, wgt, big


def logits(x, tok=None, parent=None, hist=None, hist_len=None, prompt_len=None, repetition=None, frequency=None, presence=None,
           bias=None, mask=None, mask_value=-1e30, dtype=np.float32):
    """The controls in `dtype` (float32: each step rounded by itself).  bias: a
    list of {token: value} per sequence."""
    B, R, V = x.shape
    y = x.astype(dtype)
    inside = lambda a: a[(a >= 0) & (a < V)]  # noqa: E731
    for b in range(B):
        n0, prompt = np.zeros(V, np.int64), np.zeros(V, bool)
        if hist is not None:
            hl, pl = int(hist_len[b]), 0 if prompt_len is None else int(prompt_len[b])
            np.add.at(n0, inside(hist[b, pl:hl]), 1) if hl > pl else None
            prompt[inside(hist[b, :min(pl, hl)])] = True
        for j in range(R):
            n = n0.copy()
            if tok is not None:
                np.add.at(n, inside(tok[b, row_path(parent, b, j)]), 1)
            seen = prompt | (n > 0)
            if repetition is not None:
                r = dtype(repetition[b])
                y[b, j] = np.where(seen, np.where(y[b, j] > 0, y[b, j] / r, y[b, j] * r), y[b, j])
            f = dtype(0 if frequency is None else frequency[b])
            p = dtype(0 if presence is None else presence[b])
            y[b, j] = np.where(n > 0, (y[b, j] - f * n.astype(dtype)) - p, y[b, j])
            if bias is not None:
                for v, a in bias[b].items():
                    if 0 <= v < V:
                        y[b, j, v] += dtype(a)
            if mask is not None:
                m = np.asarray(mask[b, j]).astype(np.int64) & 0xFFFFFFFF
                ok = (m[np.arange(V) // 32] >> (np.arange(V) % 32)) & 1
                y[b, j] = np.where(ok != 0, y[b, j], dtype(mask_value))
    return y


def argmax_keys(x):
    """fp32 [N, V] -> int64 bit patterns [N, ceil(V / 128)]."""
    N, V = x.shape
    u = (x + np.float32(0)).view(np.uint32).astype(np.uint64)
    o = np.where(u >> np.uint64(31) != 0, np.uint64(0xFFFFFFFF) - u, u + np.uint64(2 ** 31))
    o = np.where(np.isnan(x), np.uint64(0), o)
    key = (o << np.uint64(32)) | (np.uint64(0xFFFFFFFF) - np.arange(V, dtype=np.uint64))
    S = (V + 127) // 128
    pad = np.zeros((N, S * 128), np.uint64)
    pad[:, :V] = key
    return pad.reshape(N, S, 128).max(-1).view(np.int64)
