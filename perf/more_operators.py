"""The 8-bit paged KV cache: what is measured, and its operators' plain forms.

Four groups of cases, by `kind`:
  append8   rows of K and V into a cache held in 8 bits, K rotated by its position on the way, then a window read back
  commit8   the accepted rows of a verify block of every layer into the 8-bit cache, and those rows read back
  gather8   a window of the 8-bit cache read back as bf16 rows
  attn8     attention of a verify block's rows over the 8-bit cache

The 8-bit cache: 16 positions of one head share a scale, a power of two; a value is an e4m3 code times its block's scale.
A (page, head) block is 8320 bytes: 8192 codes, then four fp32 scales (16 positions each), then 112 bytes of nothing.  K's
codes are [64 positions][8 places][16 dims], dims 16 c .. of position p at place c ^ (p % 8); V's are [8 octets of
positions][128 dims][8 positions].  The scale is the smallest 2^e, -120 <= e <= 119, with |x| <= 448 * 2^e for all that was
written to the 16 positions since the first of them was: where later rows need a larger one, the earlier are held anew.  A
row with NaN or infinity in it is held as NaN throughout and has no part in the scale.
"""
import random

import numpy as np
import torch

own = False

D = 128        # head dim
PAGE = 64      # positions a page
RUN = 16       # positions a scale
BLOCK8 = 8320  # bytes of one (page, head) of the 8-bit cache
NEG = float("-inf")


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # eight prompts of about 2048 tokens prefilled together, one layer of the 7B head layout, all read back
        {"name": "append8 prompts 8x2048", "kind": "append8", "B": 8, "n": 2048, "t": 0, "ragged": 300, "Hkv": 4, "rot": 128,
         "pairs": False, "back": 2048},
        # a prefill chunk of 1000 tokens behind about 7100 cached ones, the whole context read back for the chunk's attention
        {"name": "append8 chunk 4x1000", "kind": "append8", "B": 4, "n": 1000, "t": 7100, "ragged": 77, "Hkv": 4, "rot": 128,
         "pairs": False, "back": 8100},
        # one token for each of 64 sequences in mid-generation, 1.5B layout, and the last 32 positions of each read back
        {"name": "append8 one token x64", "kind": "append8", "B": 64, "n": 1, "t": 4096, "ragged": 2000, "Hkv": 2, "rot": 64,
         "pairs": True, "back": 32},
        # the end of the headline round (28 layers, k = 4, batch 1) on an 8-bit cache
        {"name": "commit8 1.5B b1", "kind": "commit8", "L": 28, "B": 1, "R": 5, "t": 4096, "ragged": 0, "Hkv": 2},
        # the same for the 7B layout at batch 16, k = 8
        {"name": "commit8 7B b16", "kind": "commit8", "L": 28, "B": 16, "R": 9, "t": 8192, "ragged": 500, "Hkv": 4},
        # a whole batch's cache turned to bf16: one layer of 8 contexts of 8192
        {"name": "gather8 8x8192", "kind": "gather8", "L": 1, "B": 8, "n": 8192, "t": 8192, "ragged": 1000, "Hkv": 4},
        # a short odd window of one sequence, from its middle
        {"name": "gather8 window 77", "kind": "gather8", "L": 1, "B": 1, "n": 77, "t": 1001, "ragged": 0, "Hkv": 2},
        # the headline round's attention
        {"name": "attn8 1.5B b1 t4096", "kind": "attn8", "B": 1, "R": 5, "Hq": 12, "Hkv": 2, "t": 4096, "ragged": 0, "tree": False},
        # the large serving batch
        {"name": "attn8 7B b16 t8192", "kind": "attn8", "B": 16, "R": 9, "Hq": 28, "Hkv": 4, "t": 8192, "ragged": 0, "tree": False},
        # single tokens of a ragged batch: decoding without drafts
        {"name": "attn8 7B b64 one token", "kind": "attn8", "B": 64, "R": 1, "Hq": 28, "Hkv": 4, "t": 4097, "ragged": 3000,
         "tree": False},
        # a 64-node draft tree
        {"name": "attn8 7B tree t8192", "kind": "attn8", "B": 1, "R": 65, "Hq": 28, "Hkv": 4, "t": 8192, "ragged": 0, "tree": True},
        # one long context
        {"name": "attn8 1.5B b1 t100001", "kind": "attn8", "B": 1, "R": 5, "Hq": 12, "Hkv": 2, "t": 100001, "ragged": 0,
         "tree": False},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["append8", "append8", "commit8", "gather8", "attn8", "attn8", "attn8"])
    Hkv, G = rng.choice([(2, 6), (4, 7), (2, 8), (8, 1), (8, 4), (1, 4)])
    if kind == "append8":
        B = _log(rng, 1, 64)
        n = _log(rng, 1, max(1, 16384 // B))
        t = rng.choice([0, _log(rng, 1, 16000)])
        return {"kind": kind, "B": B, "n": n, "t": t, "ragged": rng.randrange(0, n + t + 1), "Hkv": min(Hkv, 4),
                "rot": rng.choice([128, 128, 64, 32]), "pairs": rng.random() < 0.3,
                "back": min(n + t, n + _log(rng, 15, max(15, 16384 // B)))}
    if kind == "commit8":
        return {"kind": kind, "L": _log(rng, 1, 28), "B": _log(rng, 1, 16), "R": _log(rng, 1, 65), "t": _log(rng, 1, 8192),
                "ragged": rng.randrange(0, 500), "Hkv": min(Hkv, 4)}
    if kind == "gather8":
        L, B = rng.choice([1, 1, _log(rng, 2, 8)]), _log(rng, 1, 32)
        t = _log(rng, 1, max(1, 65536 // (L * B)))
        return {"kind": kind, "L": L, "B": B, "n": _log(rng, 1, t), "t": t, "ragged": rng.randrange(0, t + 1), "Hkv": min(Hkv, 4)}
    B, R = _log(rng, 1, 32), rng.choice([1, _log(rng, 2, 16), _log(rng, 2, 100)])
    t = _log(rng, 1, max(1, min(120000, 524288 // (B * Hkv), 2 * 10 ** 9 // (B * R * Hkv * G * 64))))
    return {"kind": kind, "B": B, "R": R, "Hq": Hkv * G, "Hkv": Hkv, "t": t, "ragged": rng.randrange(0, t + 1),
            "tree": rng.random() < 0.4}


def _lens(c):
    """The sequences' lengths: t, less up to `ragged` from the second sequence on (down to none)."""
    r = min(c["ragged"], c["t"])
    return [c["t"] - (b * 2654435761 % (r + 1)) for b in range(c["B"])]


def _counts(c):
    """New rows of each sequence of an append: n, less up to `ragged` from the second on (some get none)."""
    r = min(c["ragged"], c["n"])
    return [c["n"] if c["n"] == 1 else c["n"] - (b * 40503 % (r + 1)) for b in range(c["B"])]


def _pages(total):
    return (total + PAGE - 1) // PAGE


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _keys(g, *shape):
    """Rows of K: normal values, a few dims of a head larger than the others, as heads have them."""
    big = torch.ones(D, device="cuda")
    big[torch.tensor([5, 37, 101], device="cuda")] = 6.0
    return (_randn(g, *shape, D) * big).to(torch.bfloat16)


def _values(g, *shape):
    return (_randn(g, *shape, D) * 0.7).to(torch.bfloat16)


def _table(seed, B, max_pages):
    """A page table whose sequences' pages lie scattered over the pool, and a page that no sequence has."""
    p = np.random.RandomState(seed % (2 ** 32)).permutation(B * max_pages + 3)
    return torch.from_numpy(p[: B * max_pages].astype(np.int32).reshape(B, max_pages)).cuda(), int(p[-1])


def _rope(positions, rot):
    """[positions][rot] fp32: the cosines of each position's angles, then the sines (angles in 64 bits)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _tree(seed, B, R):
    r = np.random.RandomState(seed % (2 ** 32))
    p = np.full((B, R), -1, np.int32)
    for j in range(1, R):
        p[:, j] = np.maximum(0, j - 1 - r.randint(0, 8, B))
    return torch.from_numpy(p).cuda()


def _filled8(g, pages, Hkv, is_v):
    """A pool whose every position holds a row, 16 positions after 16."""
    got = []
    for p0 in range(0, pages, 256):
        x = (_values if is_v else _keys)(g, min(256, pages - p0), Hkv, PAGE).float().unflatten(2, (4, RUN))
        s = _scale(x.abs().amax((-1, -2)))
        got.append(_join8(_code(x, s[..., None, None]).flatten(2, 3), s, is_v))
    return torch.cat(got)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    bf = torch.bfloat16
    if c["kind"] == "append8":
        counts, lens = _counts(c), _lens(c)
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        rows, mp = int(off[-1]), _pages(max(l + n for l, n in zip(lens, counts)) + 1)
        H = c["Hkv"]
        # K and V are slices of the rows of a fused projection, as the layer hands them over
        qkv = torch.cat([_randn(g, rows, H, D).to(bf), _keys(g, rows, H), _values(g, rows, H)], 1)
        table, spare = _table(seed, c["B"], mp)
        P = c["B"] * mp + 3
        ends = [l + n for l, n in zip(lens, counts)]
        s.update(rows=rows, row_off=_i32(off), length=_i32(lens), table=table, spare=spare, k=qkv[:, H:2 * H], v=qkv[:, 2 * H:],
                 rope=_rope(mp * PAGE, c["rot"]), k_pool=_filled8(g, P, H, False), v_pool=_filled8(g, P, H, True),
                 runs=max((e - 1) // RUN - l // RUN + 1 for l, e in zip(lens, ends)),
                 end=_i32(ends), start=_i32([max(0, e - c["back"]) for e in ends]))
    elif c["kind"] == "commit8":
        L, B, R, H = c["L"], c["B"], c["R"], c["Hkv"]
        lens = _lens(c)
        r = np.random.RandomState(seed % (2 ** 32))
        n_acc = r.randint(0, R, B).astype(np.int32)
        path = np.full((B, R), -1, np.int32)
        for b in range(B):  # an accepted path: increasing block rows from the root on
            m = int(n_acc[b])
            path[b, 0] = 0
            path[b, 1:m + 1] = np.sort(r.permutation(R - 1)[:m]) + 1
        P = B * 3 + 3  # only the pages that the new rows reach are in the pool
        mp = _pages(c["t"] + R)
        tab = np.full((B, mp), -1, np.int32)
        perm = r.permutation(P)
        for b in range(B):
            lo = lens[b] // PAGE
            n = min(mp, lo + 3) - lo
            tab[b, lo:lo + n] = perm[3 * b:3 * b + n]
        s.update(spare=int(perm[3 * B]), length=_i32(lens), n_acc=torch.from_numpy(n_acc).cuda(), path=torch.from_numpy(path).cuda(),
                 table=torch.from_numpy(tab).cuda(), k_pool=_filled8(g, L * P, H, False).view(L, P, H, BLOCK8),
                 v_pool=_filled8(g, L * P, H, True).view(L, P, H, BLOCK8), k_blk=_keys(g, L, B, H, R), v_blk=_values(g, L, B, H, R),
                 # what is read back: the new rows, and those that may share a scale with the first of them
                 start=_i32([l // RUN * RUN for l in lens]))
    elif c["kind"] == "gather8":
        L, B, H = c["L"], c["B"], c["Hkv"]
        lens = _lens(c)
        mp = _pages(c["t"])
        table, _ = _table(seed, B, mp)
        P = B * mp + 3
        s.update(length=_i32(lens), table=table, start=_i32([max(0, (l - c["n"]) // 2) for l in lens]),
                 k_pool=_filled8(g, L * P, H, False).view(L, P, H, BLOCK8), v_pool=_filled8(g, L * P, H, True).view(L, P, H, BLOCK8))
    else:
        B, R, Hq, H = c["B"], c["R"], c["Hq"], c["Hkv"]
        mp = _pages(c["t"] + R)
        table, _ = _table(seed, B, mp)
        P = B * mp + 3
        s.update(length=_i32(_lens(c)), table=table, k_pool=_filled8(g, P, H, False), v_pool=_filled8(g, P, H, True),
                 q=_randn(g, B, R, Hq, D).to(bf), k_blk=_keys(g, B, H, R), v_blk=_values(g, B, H, R),
                 parent=_tree(seed, B, R) if c["tree"] else None)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------

def _scale(amax):
    """The smallest power of two 2^e, -120 <= e <= 119, with amax <= 448 * 2^e (fp32)."""
    bits = amax.contiguous().view(torch.int32)
    up = ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)          # 448 is 1.75 * 2^8
    e = ((bits >> 23) - 127 - 8 + up).clamp(-120, 119)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _code(x, s):
    """fp32 values -> codes (uint8); past 448 scales they are held as 448."""
    return (x / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(codes, s):
    return codes.view(torch.float8_e4m3fn).float() * s


def _places_k(device):
    """[64, 128]: where a dim of a position lies among K's codes."""
    p, d = torch.arange(PAGE, device=device)[:, None], torch.arange(D, device=device)[None, :]
    return p * D + (((d >> 4) ^ (p & 7)) << 4) + (d & 15)


def _places_v(device):
    p, d = torch.arange(PAGE, device=device)[:, None], torch.arange(D, device=device)[None, :]
    return (p >> 3) * (8 * D) + d * 8 + (p & 7)


def _join8(codes, s, is_v):
    """codes uint8 [P, H, 64, 128], scales fp32 [P, H, 4] -> uint8 [P, H, 8320]."""
    P, H = codes.shape[:2]
    out = torch.zeros(P, H, BLOCK8, dtype=torch.uint8, device=codes.device)
    out[..., (_places_v if is_v else _places_k)(codes.device).flatten()] = codes.reshape(P, H, -1)
    out[..., PAGE * D:PAGE * D + 16] = s.contiguous().view(torch.uint8).view(P, H, 16)
    return out


def _unpack8(pool, is_v):
    """uint8 [P, H, 8320] -> fp32 [P, H, 64, 128]."""
    c = pool[..., (_places_v if is_v else _places_k)(pool.device)]
    s = pool[..., PAGE * D:PAGE * D + 16].contiguous().view(torch.float32)
    return _value(c, s.repeat_interleave(RUN, -1)[..., None])


def _store8(pool, page, run, first, new, rows, is_v):
    """Rows bf16 [N, 16, H, 128], where new[N, 16] says so, into the runs (16 positions) `run`[N] of pages page[N] of a pool
    [P, H, 8320], in place; first[N]: the run's first position is among them, so that what was there before is gone."""
    H = pool.shape[1]
    x = torch.where(new[:, :, None, None], rows.float(), 0.0).transpose(1, 2)                  # [N, H, 16, 128]
    bad = ~(x.abs() < float("inf")).all(-1, keepdim=True)
    at = (page.long()[:, None], torch.arange(H, device=pool.device)[None, :])
    sc = pool.view(torch.float32)
    k = PAGE * D // 4 + run.long()[:, None]
    old = sc[at[0], at[1], k]
    amax = torch.where(bad, 0.0, x.abs()).amax((-1, -2))
    x = torch.where(bad, float("nan"), x)
    s = torch.maximum(_scale(amax), torch.where(first[:, None], 0.0, old))
    place = (_places_v if is_v else _places_k)(pool.device).view(4, RUN, D)[run.long()][:, None]  # [N, 1, 16, 128]
    at = (at[0][:, :, None, None], at[1][:, :, None, None], place)
    held = _code(_value(pool[at], old[..., None, None]), s[..., None, None])
    pool[at] = torch.where(new[:, None, :, None], _code(x, s[..., None, None]), held)
    sc[page.long()[:, None], torch.arange(H, device=pool.device)[None, :], k] = s


def _rotate(x, pos, rope, pairs):
    """bf16 [..., H, 128] rotated to its positions [...]: 32 bits, rounded once."""
    rot = rope.shape[1]
    cos, sin = rope[pos.long(), : rot // 2][..., None, :], rope[pos.long(), rot // 2:][..., None, :]
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., : rot // 2], r[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([y, z], -1).flatten(-2) if pairs else torch.cat([y, z], -1)
    return torch.cat([r, rest], -1).to(torch.bfloat16)


def _runs(length, count, n):
    """The n runs of each sequence from the one its first new position lies in: (positions [B, n, 16], which are new, index of the
    new row, whether the run's first position is new, whether any is)."""
    pos = (length // RUN * RUN)[:, None, None] + torch.arange(n * RUN, device="cuda", dtype=torch.int32).view(1, n, RUN)
    i = pos - length[:, None, None]
    new = (i >= 0) & (i < count[:, None, None])
    return pos, new, i.clamp(min=0), new[..., 0], new.any(-1)


def _plain_append8(s):
    c = s["case"]
    count = s["row_off"][1:] - s["row_off"][:-1]
    pos, new, i, first, some = _runs(s["length"], count, s["runs"])
    row = torch.where(new, s["row_off"][:-1, None, None] + i, 0).long().flatten(0, 1)
    cols = (pos[..., 0] // PAGE).clamp(max=s["table"].shape[1] - 1).long()
    page = torch.where(some, s["table"].gather(1, cols), s["spare"]).flatten()
    run = (pos[..., 0] % PAGE // RUN).flatten()
    for pool, x, is_v in ((s["k_pool"], s["k"], False), (s["v_pool"], s["v"], True)):
        r = x[row]
        if not is_v:
            r = _rotate(r, torch.where(new, pos, 0).flatten(0, 1), s["rope"], c["pairs"])
        _store8(pool, page, run, first.flatten(), new.flatten(0, 1), r, is_v)
    return [_plain_gather8(s[n], s["table"], s["start"], s["end"], c["back"], n == "v_pool") for n in ("k_pool", "v_pool")]


def _plain_gather8(pool, table, start, length, n, is_v):
    """[P, H, 8320] -> bf16 [B, H, n, 128]: positions start.. of each sequence, zeros at and past its length."""
    p = start[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    live = p < length[:, None]
    first = start // PAGE
    np_ = (n + PAGE - 1) // PAGE + 1
    cols = (first[:, None] + torch.arange(np_, device="cuda", dtype=torch.int32)).clamp(max=table.shape[1] - 1)
    B, H = table.shape[0], pool.shape[1]
    pages = table.gather(1, cols.long()).clamp(min=0).long()
    x = _unpack8(pool[pages.flatten()], is_v).view(B, np_, H, PAGE, D).transpose(1, 2).reshape(B, H, np_ * PAGE, D)
    at = (p - first[:, None] * PAGE).long()[:, None, :, None].expand(B, H, n, D)
    return torch.where(live[:, None, :, None], x.gather(2, at), 0.0).to(torch.bfloat16)


def _plain_commit8(s):
    c = s["case"]
    L, B, R, H = c["L"], c["B"], c["R"], c["Hkv"]
    n = (R + RUN - 2) // RUN + 1
    pos, new, i, first, some = _runs(s["length"], s["n_acc"] + 1, n)
    row = s["path"].gather(1, i.clamp(max=R - 1).flatten(1).long()).clamp(min=0).long()      # [B, 16 n]
    cols = (pos[..., 0] // PAGE).clamp(max=s["table"].shape[1] - 1).long()
    page = torch.where(some, s["table"].gather(1, cols), s["spare"])
    P, end = s["k_pool"].shape[1], s["length"] + s["n_acc"] + 1
    lay = torch.arange(L, device="cuda", dtype=torch.int32)[:, None, None] * P
    pages = (lay + page).flatten()
    every = lambda x: x.expand(L, *x.shape).flatten(0, 2)  # noqa: E731
    tab = (lay + s["table"].clamp(min=0)).view(L * B, -1)
    got = []
    for pool, blk, is_v in ((s["k_pool"], s["k_blk"], False), (s["v_pool"], s["v_blk"], True)):
        x = blk.gather(3, row[None, :, None, :, None].expand(L, B, H, n * RUN, D))
        x = x.view(L, B, H, n, RUN, D).permute(0, 1, 3, 4, 2, 5).reshape(L * B * n, RUN, H, D)
        flat = pool.view(L * P, *pool.shape[2:])
        _store8(flat, pages, every(pos[..., 0] % PAGE // RUN), every(first), every(new), x, is_v)
        got.append(_plain_gather8(flat, tab, s["start"].repeat(L), end.repeat(L), R + RUN - 1, is_v).view(L, B, H, -1, D))
    return got + [end]


def _plain_gather(s):
    c = s["case"]
    L, B = c["L"], c["B"]
    got = []
    for name in ("k_pool", "v_pool"):
        pool = s[name]
        tab = (torch.arange(L, device="cuda", dtype=torch.int32)[:, None, None] * pool.shape[1] + s["table"]).view(L * B, -1)
        x = _plain_gather8(pool.flatten(0, 1), tab, s["start"].repeat(L), s["length"].repeat(L), c["n"], name == "v_pool")
        got.append(x.view(L, B, *x.shape[1:]))
    return got


def _visible(parent, B, R):
    """[B, R, R] truth values: block row i is j or one of its ancestors (chain: i <= j)."""
    if parent is None:
        return torch.ones(R, R, dtype=torch.bool, device="cuda").tril().expand(B, R, R)
    eye = torch.eye(R, device="cuda")
    m = eye + (parent[:, :, None] == torch.arange(R, device="cuda", dtype=torch.int32)).float()
    for _ in range(max(1, (R - 1).bit_length())):
        m = (m @ m).clamp(max=1.0)
    return m > 0


def _plain_attn8(s):
    c = s["case"]
    B, R, Hq, H = c["B"], c["R"], c["Hq"], c["Hkv"]
    G, T = Hq // H, s["table"].shape[1] * PAGE
    rows = lambda pool, is_v: _unpack8(pool[s["table"].flatten().long()], is_v).view(B, -1, H, PAGE, D).transpose(1, 2).reshape(B, H, T, D)  # noqa: E731
    k = torch.cat([rows(s["k_pool"], False), s["k_blk"].float()], 2)
    v = torch.cat([rows(s["v_pool"], True), s["v_blk"].float()], 2)
    q = s["q"].float().view(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    z = (q @ k.transpose(-1, -2)).view(B, H, R, G, T + R) * D ** -0.5
    ctx = (torch.arange(T, device="cuda") < s["length"][:, None])[:, None, :].expand(B, R, T)
    see = torch.cat([ctx, _visible(s["parent"], B, R)], 2)
    z = z.masked_fill(~see[:, None, :, None, :], NEG)
    p = (z - z.amax(-1, keepdim=True)).exp()
    o = (p.view(B, H, R * G, T + R) @ v).view(B, H, R, G, D) / p.sum(-1, keepdim=True)
    return o.permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D).to(torch.bfloat16)


_PLAIN = {"append8": _plain_append8, "commit8": _plain_commit8, "gather8": _plain_gather, "attn8": _plain_attn8}


def _own(s):
    from speculative_decoding_verification_sv_gb300 import binding as sv
    c = s["case"]
    if c["kind"] == "append8":
        sv.kv_append_q8(s["k"], s["v"], s["row_off"], s["k_pool"], s["v_pool"], s["table"], s["length"], rope=s["rope"],
                        interleaved=c["pairs"])
        k, v = sv.kv_gather_q8(s["k_pool"][None], s["v_pool"][None], s["table"], s["start"], s["end"], c["back"])
        return [k[0], v[0]]
    if c["kind"] == "commit8":
        length = s["length"].clone()  # advanced in place
        sv.kv_commit_q8(s["k_pool"], s["v_pool"], s["table"], s["k_blk"], s["v_blk"], s["path"], s["n_acc"], length)
        k, v = sv.kv_gather_q8(s["k_pool"], s["v_pool"], s["table"], s["start"], length, c["R"] + RUN - 1)
        return [k, v, length]
    if c["kind"] == "gather8":
        return list(sv.kv_gather_q8(s["k_pool"], s["v_pool"], s["table"], s["start"], s["length"], c["n"]))
    return sv.verify_attn_q8(s["q"], s["k_pool"], s["v_pool"], s["table"], s["length"], s["k_blk"], s["v_blk"], s["parent"])


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["kind"] == "append8":
        counts, lens, H = _counts(c), _lens(c), c["Hkv"]
        rows, row = sum(counts), 2 * H * D * 2
        seen = len(set().union(*(range(l, l + n) for l, n in zip(lens, counts)))) if rows else 0
        back = sum(min(c["back"], l + n) for l, n in zip(lens, counts))
        return {"bytes": rows * row + seen * c["rot"] * 4 + 4 * (2 * c["B"] + 1) + (rows + back) * H * 256.5 + c["B"] * c["back"] * row,
                "flops": rows * H * (c["rot"] * 3 + 4 * D) + back * H * 2 * D}
    if c["kind"] == "commit8":
        L, B, R, H = c["L"], c["B"], c["R"], c["Hkv"]
        n = B * (R + 1) / 2  # a path holds one to R rows, each number as often
        w = R + RUN - 1
        return {"bytes": L * H * (n * (512 + 256.5) + (n + B * 7.5) * 256.5 + B * w * 512) + B * (R + 4) * 4, "flops": L * H * n * 8 * D}
    if c["kind"] == "gather8":
        L, B, H = c["L"], c["B"], c["Hkv"]
        got = sum(min(c["n"], l) for l in _lens(c))
        return {"bytes": L * H * (got * 256.5 + B * c["n"] * 512), "flops": L * H * got * 2 * D}
    B, R, Hq, H = c["B"], c["R"], c["Hq"], c["Hkv"]
    t = sum(_lens(c))
    return {"bytes": t * H * 256.5 + 4 * B * R * Hq * D + 4 * B * R * H * D, "flops": 4 * R * Hq * D * (t + B * (R + 1) / 2)}


# ---------------------------------------------------------------------------------------------------------------------
# exact values
# ---------------------------------------------------------------------------------------------------------------------

def _fp64(x):
    return x.detach().cpu().to(torch.float64).numpy()


def _bf16_of(x):
    """float64 -> the nearest bf16 (ties to even), as float64: 8 significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256) / 256, e)


def _e4m3_of(x):
    """float64 within +-448 -> the nearest e4m3 (ties to even): 4 significant bits, steps of 2^-9 at least."""
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    return np.rint(x / step) * step


_E4M3 = np.array([(-1.0) ** (c >> 7) * (np.ldexp(c & 7, -9) if (c >> 3) & 15 == 0 else np.ldexp(8 + (c & 7), ((c >> 3) & 15) - 10))
                  for c in range(256)])
_E4M3[[127, 255]] = np.nan


def _need(a):
    """float64 largest magnitudes -> the exponents that hold them."""
    m, e = np.frexp(a)
    return np.where(a > 0, np.clip(e - 9 + (m > 0.875), -120, 119), -120)


def _read8(blk, is_v):
    """(codes' values, exponents) of blocks (numpy uint8 [..., 8320]): float64 [..., 64, 128] and [..., 4]."""
    p, d = np.arange(64)[:, None], np.arange(128)[None, :]
    byte = p // 8 * 1024 + d * 8 + p % 8 if is_v else p * 128 + (d // 16 ^ p % 8) * 16 + d % 16
    sc = np.ascontiguousarray(blk[..., 8192:8208]).view("<f4").astype(np.float64)
    return _E4M3[blk[..., byte]], np.rint(np.log2(sc)).astype(np.int64)


def _written(val, e, rows, at):
    """Values and exponents of one run of a head ([16, 128] in units of 2^e) after float64 rows were written from place `at` on."""
    n = len(rows)
    need = int(_need(np.abs(rows).max()))
    new = need if at == 0 else max(need, int(e))
    out = _e4m3_of(np.ldexp(val, int(e) - new))
    out[at:at + n] = _e4m3_of(np.clip(np.ldexp(rows, -new), -448, 448))
    return out, new


def _turned(x, pos, rope, pairs):
    """float64 rows [n, H, 128] at positions pos[n] turned by the table's angles."""
    h = rope.shape[1] // 2
    at = np.arange(h)
    i, j = (2 * at, 2 * at + 1) if pairs else (at, at + h)
    cs, sn = rope[pos, :h][:, None], rope[pos, h:][:, None]
    y = x.copy()
    y[..., i] = x[..., i] * cs - x[..., j] * sn
    y[..., j] = x[..., i] * sn + x[..., j] * cs
    return y


def _after(blocks, rows, l, is_v, lo, hi):
    """Values at positions lo .. hi - 1 of one head after rows were written at l ..; blocks(page): the page's block."""
    out = np.zeros((hi - lo, D))
    kept = {}
    for q in range(lo // RUN * RUN, hi, RUN):
        pg = q // PAGE
        if pg not in kept:
            kept = {pg: _read8(blocks(pg), is_v)}
        val, e = kept[pg][0][q % PAGE:q % PAGE + RUN], kept[pg][1][q % PAGE // RUN]
        a, z = max(q, l), min(q + RUN, l + len(rows))
        if a < z:
            val, e = _written(val, e, rows[a - l:z - l], a - q)
        u, w = max(q, lo), min(q + RUN, hi)
        out[u - lo:w - lo] = np.ldexp(val[u - q:w - q], int(e))
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "append8":
        counts, lens = _counts(c), _lens(c)
        if sum(counts) * c["Hkv"] > 80000:
            return None
        tab, k, v, rope = s["table"].cpu().numpy(), _fp64(s["k"]), _fp64(s["v"]), _fp64(s["rope"])
        kp, vp = s["k_pool"].cpu().numpy(), s["v_pool"].cpu().numpy()
        ko = np.zeros((c["B"], c["Hkv"], c["back"], D))
        vo = np.zeros_like(ko)
        i0 = 0
        for b, (l, n) in enumerate(zip(lens, counts)):
            kr, vr = _bf16_of(_turned(k[i0:i0 + n], np.arange(l, l + n), rope, c["pairs"])), v[i0:i0 + n]
            i0 += n
            st = max(0, l + n - c["back"])
            for h in range(c["Hkv"]):
                ko[b, h, :l + n - st] = _after(lambda p: kp[tab[b, p], h], kr[:, h], l, False, st, l + n)
                vo[b, h, :l + n - st] = _after(lambda p: vp[tab[b, p], h], vr[:, h], l, True, st, l + n)
        return [ko, vo]
    if c["kind"] == "commit8":
        L, B, R, H = c["L"], c["B"], c["R"], c["Hkv"]
        lens, path, m, tab = _lens(c), s["path"].cpu().numpy(), s["n_acc"].cpu().numpy(), s["table"].cpu().numpy()
        got = []
        for pool, blk, is_v in ((s["k_pool"], s["k_blk"], False), (s["v_pool"], s["v_blk"], True)):
            x, p8 = _fp64(blk), pool.cpu().numpy()
            y = np.zeros((L, B, H, R + RUN - 1, D))
            for a in range(L):
                for b in range(B):
                    st = lens[b] // RUN * RUN
                    n = lens[b] + m[b] + 1 - st
                    for h in range(H):
                        y[a, b, h, :n] = _after(lambda p: p8[a, tab[b, p], h], x[a, b, h, path[b, :m[b] + 1]], lens[b], is_v, st, st + n)
            got.append(y)
        return got + [None]
    if c["kind"] == "gather8":
        L, B, H, n = c["L"], c["B"], c["Hkv"], c["n"]
        lens, tab, st = _lens(c), s["table"].cpu().numpy(), s["start"].cpu().numpy()
        if L * B * H * n > 400000:
            return None
        got = []
        for pool, is_v in ((s["k_pool"], False), (s["v_pool"], True)):
            p8, y = pool.cpu().numpy(), np.zeros((L, B, H, n, D))
            for a in range(L):
                for b in range(B):
                    t = min(n, lens[b] - st[b])
                    for h in range(H):
                        y[a, b, h, :t] = _after(lambda p: p8[a, tab[b, p], h], np.zeros((0, D)), 0, is_v, st[b], st[b] + t)
            got.append(y)
        return got
    B, R, Hq, H = c["B"], c["R"], c["Hq"], c["Hkv"]
    G, lens = Hq // H, _lens(c)
    if 4 * R * Hq * D * sum(lens) > 3e11:
        return None
    out = torch.zeros(B, R, Hq, D, dtype=torch.float64, device="cuda")
    value = torch.from_numpy(_E4M3).cuda()
    p, d = torch.arange(64, device="cuda")[:, None], torch.arange(128, device="cuda")[None, :]
    k_at = p * 128 + (torch.div(d, 16, rounding_mode="floor") ^ (p % 8)) * 16 + d % 16
    v_at = torch.div(p, 8, rounding_mode="floor") * 1024 + d * 8 + p % 8
    par = None if s["parent"] is None else s["parent"].cpu().numpy()
    for b in range(B):
        t = lens[b]
        pg = s["table"][b, : _pages(t)].long()
        see = torch.zeros(R, t + R, dtype=torch.bool, device="cuda")
        see[:, :t] = True
        for j in range(R):
            if par is None:
                see[j, t:t + j + 1] = True
            else:
                i = j
                while i >= 0:
                    see[j, t + i] = True
                    i = int(par[b, i])
        for h in range(H):
            kv = []
            for pool, at in ((s["k_pool"], k_at), (s["v_pool"], v_at)):
                blk = pool[pg, h]
                sc = blk[:, 8192:8208].contiguous().view(torch.float32).double()
                x = value[blk[:, at].long()].view(-1, 4, 16, D) * sc[:, :, None, None]
                kv.append(x.reshape(-1, D)[:t])
            kk, vv = torch.cat([kv[0], s["k_blk"][b, h].double()]), torch.cat([kv[1], s["v_blk"][b, h].double()])
            qq = s["q"][b, :, h * G:(h + 1) * G].double()
            z = torch.einsum("rgd,td->rgt", qq, kk) / D ** 0.5
            z = torch.where(see[:, None, :], z, torch.full((), NEG, dtype=torch.float64, device="cuda"))
            out[b, :, h * G:(h + 1) * G] = torch.einsum("rgt,td->rgd", torch.softmax(z, -1), vv)
    return out


if __name__ == "__main__":
    for one in listed() + [draw(random.Random(k)) for k in range(12)]:
        print(one, work(one))
