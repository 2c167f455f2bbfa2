"""The serving operators around the verify round: what is measured, and their plain forms.

Four groups of cases, by `kind`:
  append    rows of K and V into a paged bf16 cache, K rotated by its position on the way
  append4   the same into a cache held in 4 bits, then the cache read back as bf16 rows
  commit4   the accepted rows of a verify block of every layer into the 4-bit cache, and those rows read back
  attn4     attention of the block's rows over the 4-bit cache
  logits    repetition, frequency and presence penalties, biases and grammar masks on the block's logits

The 4-bit cache: a group of 32 head dims of one (position, head) holds a bf16 scale s with 4 significant bits and 32
codes c in 0..15 for the values (c - 8) s.  A (page, head) block is 4608 bytes: for K, codes [4 groups][64 positions]
[16 bytes], then scales [64 positions][4]; for V, codes [8 octets of positions][128 dims][4 bytes], then scales
[4 groups][64 positions].  Element e of the 8 in a 32-bit word sits at bit 4 (e >> 1) + 16 (e & 1).
"""
import random

import numpy as np
import torch

own = False

D = 128        # head dim
PAGE = 64      # positions a page
BLOCK4 = 4608  # bytes of one (page, head) of the 4-bit cache
NEG = float("-inf")


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # eight prompts of about 2048 tokens prefilled together, one layer of the 7B head layout
        {"name": "append prompts 8x2048", "kind": "append", "B": 8, "n": 2048, "t": 0, "ragged": 300, "Hkv": 4, "rot": 128,
         "pairs": False},
        # the smallest call: one token for each of 64 sequences in mid-generation, 1.5B layout, part of the dims rotated
        {"name": "append one token x64", "kind": "append", "B": 64, "n": 1, "t": 4096, "ragged": 2000, "Hkv": 2, "rot": 64,
         "pairs": True},
        # a prefill chunk of 1024 tokens behind 7168 cached ones, and the whole context read back for the chunk's attention
        {"name": "append4 chunk 4x1024", "kind": "append4", "B": 4, "n": 1024, "t": 7168, "ragged": 77, "Hkv": 4, "rot": 128,
         "pairs": False, "back": 8192},
        # one token for each of 32 sequences, and the last page's worth of each read back
        {"name": "append4 one token x32", "kind": "append4", "B": 32, "n": 1, "t": 2048, "ragged": 1500, "Hkv": 2, "rot": 128,
         "pairs": False, "back": 64},
        # the end of the headline round (28 layers, k = 4, batch 1) on a 4-bit cache
        {"name": "commit4 1.5B b1", "kind": "commit4", "L": 28, "B": 1, "R": 5, "t": 4096, "ragged": 0, "Hkv": 2},
        # the same for the 7B layout at batch 16, k = 8
        {"name": "commit4 7B b16", "kind": "commit4", "L": 28, "B": 16, "R": 9, "t": 8192, "ragged": 500, "Hkv": 4},
        # the headline round's attention
        {"name": "attn4 1.5B b1 t4096", "kind": "attn4", "B": 1, "R": 5, "Hq": 12, "Hkv": 2, "t": 4096, "ragged": 0, "tree": False},
        # the large serving batch
        {"name": "attn4 7B b16 t8192", "kind": "attn4", "B": 16, "R": 9, "Hq": 28, "Hkv": 4, "t": 8192, "ragged": 0, "tree": False},
        # a 64-node draft tree
        {"name": "attn4 7B tree t8192", "kind": "attn4", "B": 1, "R": 65, "Hq": 28, "Hkv": 4, "t": 8192, "ragged": 0, "tree": True},
        # greedy decoding of one sequence with penalties: only the argmax keys are wanted
        {"name": "logits 1.5B b1 keys", "kind": "logits", "B": 1, "R": 5, "V": 151936, "H": 4096, "bias": 0, "mask": False,
         "tree": False, "out": False},
        # greedy decoding under a grammar at batch 16, with biases
        {"name": "logits 7B b16 grammar", "kind": "logits", "B": 16, "R": 9, "V": 152064, "H": 8192, "bias": 50, "mask": True,
         "tree": False, "out": True},
        # the sampled batch: logits for the acceptance
        {"name": "logits sampled b64", "kind": "logits", "B": 64, "R": 9, "V": 151936, "H": 2048, "bias": 20, "mask": False,
         "tree": False, "out": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["append", "append4", "commit4", "attn4", "attn4", "logits", "logits"])
    Hkv, G = rng.choice([(2, 6), (4, 7), (2, 8), (8, 1), (8, 4), (1, 4)])
    if kind in ("append", "append4"):
        B = _log(rng, 1, 64)
        n = _log(rng, 1, max(1, 16384 // B))
        t = rng.choice([0, _log(rng, 1, 16000)])
        c = {"kind": kind, "B": B, "n": n, "t": t, "ragged": rng.randrange(0, n + t + 1), "Hkv": min(Hkv, 4),
             "rot": rng.choice([128, 128, 64, 32]), "pairs": rng.random() < 0.3}
        if kind == "append4":
            c["back"] = _log(rng, 1, max(1, min(n + t, 32768 // B)))
        return c
    if kind == "commit4":
        return {"kind": kind, "L": _log(rng, 1, 28), "B": _log(rng, 1, 16), "R": _log(rng, 1, 65), "t": _log(rng, 1, 8192),
                "ragged": rng.randrange(0, 500), "Hkv": min(Hkv, 4)}
    if kind == "attn4":
        B, R = _log(rng, 1, 32), rng.choice([1, _log(rng, 2, 16), _log(rng, 2, 100)])
        t = _log(rng, 1, max(1, min(120000, 524288 // (B * Hkv), 2 * 10 ** 9 // (B * R * Hkv * G * 64))))
        return {"kind": kind, "B": B, "R": R, "Hq": Hkv * G, "Hkv": Hkv, "t": t, "ragged": rng.randrange(0, t + 1),
                "tree": rng.random() < 0.4}
    B, R = _log(rng, 1, 64), rng.choice([1, _log(rng, 2, 16), _log(rng, 2, 65)])
    V = rng.choice([151936, 152064, _log(rng, 100, 160000)])
    B = max(1, min(B, 64 * 9 * 151936 // (R * V)))
    return {"kind": kind, "B": B, "R": R, "V": V, "H": _log(rng, 1, 16384), "bias": rng.choice([0, _log(rng, 1, 300)]),
            "mask": rng.random() < 0.5, "tree": rng.random() < 0.4, "out": rng.random() < 0.7}


def _lens(c, key="t"):
    """The sequences' lengths: c[key], less up to `ragged` from the second sequence on."""
    r = min(c["ragged"], c[key])
    return [c[key] - (b * 2654435761 % (r + 1)) for b in range(c["B"])]


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


def _table(seed, B, max_pages):
    """A page table whose sequences' pages lie scattered over the pool."""
    p = np.random.RandomState(seed % (2 ** 32)).permutation(B * max_pages + 3)[: B * max_pages]
    return torch.from_numpy(p.astype(np.int32).reshape(B, max_pages)).cuda()


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


def _filled4(g, pages, Hkv, is_v):
    """A pool whose every position holds a quantised row of normal values."""
    return torch.cat([_pack4(_randn(g, min(256, pages - p0), Hkv, PAGE, D).to(torch.bfloat16), is_v)
                      for p0 in range(0, pages, 256)])


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    bf = torch.bfloat16
    if c["kind"] in ("append", "append4"):
        counts, lens = _counts(c), _lens(c)
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        rows, mp = int(off[-1]), _pages(max(l + n for l, n in zip(lens, counts)) + 1)
        H = c["Hkv"]
        # K and V are slices of the rows of a fused projection, as the layer hands them over
        qkv = _randn(g, rows, 3 * H, D).to(bf)
        s.update(rows=rows, row_off=_i32(off), length=_i32(lens), table=_table(seed, c["B"], mp), k=qkv[:, H:2 * H], v=qkv[:, 2 * H:],
                 rope=_rope(mp * PAGE, c["rot"]))
        P = c["B"] * mp + 3
        if c["kind"] == "append":
            s.update(k_pool=_randn(g, P, H, PAGE, D).to(bf), v_pool=_randn(g, P, H, PAGE, D).to(bf))
        else:
            s.update(k_pool=_filled4(g, P, H, False), v_pool=_filled4(g, P, H, True))
            ends = [l + n for l, n in zip(lens, counts)]
            s.update(end=_i32(ends), start=_i32([max(0, e - c["back"]) for e in ends]))
    elif c["kind"] == "commit4":
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
                 table=torch.from_numpy(tab).cuda(), k_pool=_filled4(g, L * P, H, False).view(L, P, H, BLOCK4),
                 v_pool=_filled4(g, L * P, H, True).view(L, P, H, BLOCK4), k_blk=_randn(g, L, B, H, R, D).to(bf),
                 v_blk=_randn(g, L, B, H, R, D).to(bf))
    elif c["kind"] == "attn4":
        B, R, Hq, H = c["B"], c["R"], c["Hq"], c["Hkv"]
        lens = _lens(c)
        mp = _pages(c["t"] + R)
        P = B * mp + 3
        s.update(length=_i32(lens), table=_table(seed, B, mp), k_pool=_filled4(g, P, H, False), v_pool=_filled4(g, P, H, True),
                 q=_randn(g, B, R, Hq, D).to(bf), k_blk=_randn(g, B, H, R, D).to(bf), v_blk=_randn(g, B, H, R, D).to(bf),
                 parent=_tree(seed, B, R) if c["tree"] else None)
    else:
        B, R, V, H = c["B"], c["R"], c["V"], c["H"]
        r = np.random.RandomState(seed % (2 ** 32))
        # tokens repeat as they do in text: low ids often, high ids rarely
        some = lambda *n: np.minimum(V - 1, (V ** r.random_sample(n) - 1)).astype(np.int32)  # noqa: E731
        hl = np.array([H - (b * 37 % (H // 2 + 1)) for b in range(B)], np.int32)
        s.update(logits=_randn(g, B, R, V) * 3, tok=torch.from_numpy(some(B, R)).cuda(), parent=_tree(seed, B, R) if c["tree"] else None,
                 hist=torch.from_numpy(some(B, H)).cuda(), hist_len=torch.from_numpy(hl).cuda(), prompt_len=torch.from_numpy(hl // 3).cuda(),
                 rep=torch.from_numpy(r.uniform(1.0, 1.3, B).astype(np.float32)).cuda(),
                 freq=torch.from_numpy(r.uniform(0, 0.5, B).astype(np.float32)).cuda(),
                 pres=torch.from_numpy(r.uniform(-0.5, 1.0, B).astype(np.float32)).cuda(), bias_off=None, bias_tok=None, bias_val=None, mask=None)
        if c["bias"]:
            n = min(c["bias"], V)
            s.update(bias_off=_i32([n * b for b in range(B + 1)]),
                     bias_tok=torch.from_numpy(np.concatenate([r.permutation(V)[:n] for b in range(B)]).astype(np.int32)).cuda(),
                     bias_val=torch.from_numpy(r.uniform(-5, 5, B * n).astype(np.float32)).cuda())
        if c["mask"]:
            # a grammar's rows allow few tokens or most of them
            W = (V + 31) // 32
            w = torch.randint(-2 ** 31, 2 ** 31, (B, R, W), generator=g, device="cuda", dtype=torch.int64)
            w2 = torch.randint(-2 ** 31, 2 ** 31, (B, R, W), generator=g, device="cuda", dtype=torch.int64)
            few = (torch.arange(B * R, device="cuda").view(B, R, 1) % 3) == 0
            s["mask"] = torch.where(few, w & w2, w | w2).to(torch.int32)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------

def _quant(x):
    """bf16 [..., 128] -> (codes [..., 4, 32] int32, scales [..., 4] bf16)."""
    x = x.float().unflatten(-1, (4, 32))
    amax = x.abs().amax(-1)
    # (a division by a number would be a product with its reciprocal, off where amax is 7 times a scale)
    s = (((amax / torch.full_like(amax, 7.0)).view(torch.int32) + 0xFFFFF) & ~0xFFFFF).view(torch.float32)
    s = torch.where(amax > 0, s.clamp(2.0 ** -100, 2.0 ** 118), 0.0)
    q = torch.where(s[..., None] > 0, torch.round(x / s[..., None]), 0.0).clamp(-7, 7)
    return q.to(torch.int32) + 8, s.to(torch.bfloat16)


def _shifts(n, device):
    e = torch.arange(n, device=device) % 8
    return (4 * (e >> 1) + 16 * (e & 1)).to(torch.int32)


def _words(codes):
    """[..., 8 n] codes -> [..., n] 32-bit words."""
    return (codes << _shifts(codes.shape[-1], codes.device)).unflatten(-1, (-1, 8)).sum(-1).to(torch.int32)


def _pack4(rows, is_v):
    """bf16 [P, H, 64, 128] -> uint8 [P, H, 4608]."""
    codes, s = _quant(rows)
    P, H = rows.shape[:2]
    if is_v:
        w = _words(codes.flatten(-2).transpose(-1, -2)).transpose(-1, -2)      # [P, H, 8 octets, 128 dims]
        s = s.transpose(-1, -2)                                                # [P, H, 4, 64]
    else:
        w = _words(codes).transpose(2, 3)                                      # [P, H, 4 groups, 64, 4 words]
    return torch.cat([w.contiguous().view(torch.uint8).reshape(P, H, -1), s.contiguous().view(torch.uint8).reshape(P, H, -1)], 2)


def _unpack4(pool, is_v):
    """uint8 [P, H, 4608] -> fp32 [P, H, 64, 128]."""
    P, H = pool.shape[:2]
    w = pool[..., :4096].contiguous().view(torch.int32)
    s = pool[..., 4096:].contiguous().view(torch.bfloat16).float()
    sh = _shifts(8, pool.device)
    if is_v:
        c = ((w.view(P, H, 8, 1, 128) >> sh[:, None]) & 15).reshape(P, H, 64, 128)
        s = s.view(P, H, 4, 64).transpose(2, 3)
    else:
        c = ((w.view(P, H, 4, 64, 4, 1) >> sh) & 15).reshape(P, H, 4, 64, 32).transpose(2, 3).reshape(P, H, 64, 128)
        s = s.view(P, H, 64, 4)
    return (c - 8).float() * s.repeat_interleave(32, -1)


def _store4(pool, page, slot, rows, is_v):
    """Quantises bf16 rows [N, H, 128] into positions slot[N] of pages page[N] of a pool [P, H, 4608], in place."""
    codes, s = _quant(rows)
    N, H = rows.shape[:2]
    page, slot, h = page.long()[:, None, None], slot.long()[:, None, None], torch.arange(H, device=pool.device)[None, :, None]
    w, sc = pool.view(torch.int32), pool.view(torch.bfloat16)
    g = torch.arange(4, device=pool.device)[None, None, :]
    if is_v:
        at = (slot >> 3) * 128 + torch.arange(D, device=pool.device)[None, None, :]
        sh = _shifts(8, pool.device)[slot & 7]
        old = (w[page, h, at] >> sh) & 15
        w.index_put_((page, h, at), (codes.flatten(-2) - old) << sh, accumulate=True)
        sc[page, h, 2048 + g * PAGE + slot] = s
    else:
        at = (g * (4 * PAGE) + slot * 4)[..., None] + torch.arange(4, device=pool.device)
        w[page[..., None], h[..., None], at] = _words(codes)
        sc[page, h, 2048 + slot * 4 + g] = s


def _rotate(x, pos, rope, pairs):
    """bf16 [N, H, 128] rotated to its positions: 32 bits, rounded once."""
    rot = rope.shape[1]
    cos, sin = rope[pos.long(), : rot // 2][:, None], rope[pos.long(), rot // 2:][:, None]
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., : rot // 2], r[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([y, z], -1).flatten(-2) if pairs else torch.cat([y, z], -1)
    return torch.cat([r, rest], -1).to(torch.bfloat16)


def _places(s):
    """(position, page, slot) of each new row."""
    i = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    b = (i[:, None] >= s["row_off"][None, 1:]).sum(1)
    pos = s["length"][b] + i - s["row_off"][b]
    return pos, s["table"][b, (pos // PAGE).long()], pos % PAGE


def _plain_append(s):
    pos, page, slot = _places(s)
    h = torch.arange(s["k"].shape[1], device="cuda")[None, :]
    s["k_pool"][page.long()[:, None], h, slot.long()[:, None]] = _rotate(s["k"], pos, s["rope"], s["case"]["pairs"])
    s["v_pool"][page.long()[:, None], h, slot.long()[:, None]] = s["v"]
    return [s["k_pool"], s["v_pool"]]


def _plain_gather4(pool, table, start, length, n, is_v):
    """[P, H, 4608] -> bf16 [B, H, n, 128]: positions start.. of each sequence, zeros at and past its length."""
    p = start[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    live = p < length[:, None]
    first = start // PAGE
    np_ = (n + PAGE - 1) // PAGE + 1
    cols = (first[:, None] + torch.arange(np_, device="cuda", dtype=torch.int32)).clamp(max=table.shape[1] - 1)
    B, H = table.shape[0], pool.shape[1]
    pages = table.gather(1, cols.long()).clamp(min=0).long()
    x = _unpack4(pool[pages.flatten()], is_v).view(B, np_, H, PAGE, D).transpose(1, 2).reshape(B, H, np_ * PAGE, D)
    at = (p - first[:, None] * PAGE).long()[:, None, :, None].expand(B, H, n, D)
    return torch.where(live[:, None, :, None], x.gather(2, at), 0.0).to(torch.bfloat16)


def _plain_append4(s):
    pos, page, slot = _places(s)
    _store4(s["k_pool"], page, slot, _rotate(s["k"], pos, s["rope"], s["case"]["pairs"]), False)
    _store4(s["v_pool"], page, slot, s["v"], True)
    return [_plain_gather4(s[n], s["table"], s["start"], s["end"], s["case"]["back"], n == "v_pool") for n in ("k_pool", "v_pool")]


def _plain_commit4(s):
    c = s["case"]
    L, B, R = c["L"], c["B"], c["R"]
    j = torch.arange(R, device="cuda", dtype=torch.int32)[None, :]
    take = j <= s["n_acc"][:, None]
    rows, pos = s["path"].clamp(min=0), s["length"][:, None] + j
    # block rows that are not accepted go to a page that no sequence has
    page = torch.where(take, s["table"].gather(1, (pos // PAGE).clamp(max=s["table"].shape[1] - 1).long()), s["spare"])
    P, end = s["k_pool"].shape[1], s["length"] + s["n_acc"] + 1
    lay = torch.arange(L, device="cuda", dtype=torch.int32)[:, None, None] * P
    pages, slots = (lay + page).reshape(-1), (pos % PAGE).expand(L, B, R).reshape(-1)
    tab = (lay + s["table"].clamp(min=0)).view(L * B, -1)
    got = []
    for pool, blk, is_v in ((s["k_pool"], s["k_blk"], False), (s["v_pool"], s["v_blk"], True)):
        x = blk.gather(3, rows.long()[None, :, None, :, None].expand(*blk.shape)).transpose(2, 3)
        flat = pool.view(L * P, *pool.shape[2:])
        _store4(flat, pages, slots, x.reshape(L * B * R, *x.shape[3:]), is_v)
        got.append(_plain_gather4(flat, tab, s["length"].repeat(L), end.repeat(L), R, is_v).view(L, B, -1, R, D))
    return got + [end]


def _visible(parent, B, R):
    """[B, R, R] truth values: block row i is j or one of its ancestors (chain: i <= j)."""
    if parent is None:
        return torch.ones(R, R, dtype=torch.bool, device="cuda").tril().expand(B, R, R)
    eye = torch.eye(R, device="cuda")
    m = eye + (parent[:, :, None] == torch.arange(R, device="cuda", dtype=torch.int32)).float()
    for _ in range(max(1, (R - 1).bit_length())):
        m = (m @ m).clamp(max=1.0)
    return m > 0


def _plain_attn4(s):
    c = s["case"]
    B, R, Hq, H = c["B"], c["R"], c["Hq"], c["Hkv"]
    G, T = Hq // H, s["table"].shape[1] * PAGE
    rows = lambda pool, is_v: _unpack4(pool[s["table"].flatten().long()], is_v).view(B, -1, H, PAGE, D).transpose(1, 2).reshape(B, H, T, D)  # noqa: E731
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


def _plain_logits(s):
    c = s["case"]
    B, R, V = c["B"], c["R"], c["V"]
    l = s["logits"]
    i = torch.arange(s["hist"].shape[1], device="cuda", dtype=torch.int32)
    live, prompt = i < s["hist_len"][:, None], i < s["prompt_len"][:, None]
    base = torch.zeros(B, V, dtype=torch.int32, device="cuda").scatter_add_(1, s["hist"].long(), (live & ~prompt).int())
    seen = torch.zeros(B, V, dtype=torch.int32, device="cuda").scatter_add_(1, s["hist"].long(), (live & prompt).int()) > 0
    n = base[:, None].expand(B, R, V).contiguous()
    n.scatter_add_(2, s["tok"].long()[:, None, :].expand(B, R, R).contiguous(), _visible(s["parent"], B, R).int())
    per = lambda x: x[:, None, None]  # noqa: E731
    x = torch.where(seen[:, None] | (n > 0), torch.where(l > 0, l / per(s["rep"]), l * per(s["rep"])), l)
    x = x - per(s["freq"]) * n.float()
    x = torch.where(n > 0, x - per(s["pres"]), x)
    if s["bias_off"] is not None:
        add = torch.zeros(B, V, device="cuda")
        k = c["bias"] if c["bias"] < V else V
        add.scatter_(1, s["bias_tok"].view(B, k).long(), s["bias_val"].view(B, k))
        x = x + add[:, None]
    if s["mask"] is not None:
        bit = torch.arange(32, device="cuda", dtype=torch.int32)
        ok = ((s["mask"][..., None] >> bit) & 1).flatten(2)[..., :V] != 0
        x = x.masked_fill(~ok, NEG)
    # the largest (value, lowest column) of each slab of 128 columns, as one 64-bit key
    u = torch.where(x == 0, 0.0, x).view(torch.int32).long() & 0xFFFFFFFF
    o = torch.where(u >= 2 ** 31, 0xFFFFFFFF - u, u + 2 ** 31)
    key = ((o - 2 ** 31) << 32) + (0xFFFFFFFF - torch.arange(V, device="cuda"))
    S = (V + 127) // 128
    key = torch.nn.functional.pad(key, (0, S * 128 - V), value=-2 ** 63).view(B, R, S, 128).amax(-1) ^ (-2 ** 63)
    return [x, key] if c["out"] else [key]


_PLAIN = {"append": _plain_append, "append4": _plain_append4, "commit4": _plain_commit4, "attn4": _plain_attn4, "logits": _plain_logits}


def _own(s):
    from speculative_decoding_verification_sv_gb300 import binding as sv
    c = s["case"]
    if c["kind"] == "append":
        sv.kv_append_paged(s["k"], s["v"], s["row_off"], s["k_pool"], s["v_pool"], s["table"], s["length"], rope=s["rope"],
                           interleaved=c["pairs"])
        return [s["k_pool"], s["v_pool"]]
    if c["kind"] == "append4":
        sv.kv_append_q4(s["k"], s["v"], s["row_off"], s["k_pool"], s["v_pool"], s["table"], s["length"], rope=s["rope"],
                        interleaved=c["pairs"])
        k, v = sv.kv_gather_q4(s["k_pool"][None], s["v_pool"][None], s["table"], s["start"], s["end"], c["back"])
        return [k[0], v[0]]
    if c["kind"] == "commit4":
        length = s["length"].clone()  # advanced in place
        sv.kv_commit_q4(s["k_pool"], s["v_pool"], s["table"], s["k_blk"], s["v_blk"], s["path"], s["n_acc"], length)
        k, v = sv.kv_gather_q4(s["k_pool"], s["v_pool"], s["table"], s["length"], length, c["R"])
        return [k, v, length]
    if c["kind"] == "attn4":
        return sv.verify_attn_q4(s["q"], s["k_pool"], s["v_pool"], s["table"], s["length"], s["k_blk"], s["v_blk"], s["parent"])
    out, keys = sv.logits_process(s["logits"], tok=s["tok"], parent=s["parent"], hist=s["hist"], hist_len=s["hist_len"],
                                  prompt_len=s["prompt_len"], repetition=s["rep"], frequency=s["freq"], presence=s["pres"],
                                  bias_off=s["bias_off"], bias_tok=s["bias_tok"], bias_val=s["bias_val"], mask=s["mask"],
                                  mask_value=NEG, write_logits=c["out"], write_argmax=True)
    keys = keys.view(c["B"], c["R"], -1)
    return [out, keys] if c["out"] else [keys]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["kind"] in ("append", "append4"):
        counts, lens, H = _counts(c), _lens(c), c["Hkv"]
        rows, row = sum(counts), 2 * H * D * 2
        seen = len(set().union(*(range(l, l + n) for l, n in zip(lens, counts)))) if rows else 0
        b = rows * row + seen * c["rot"] * 4 + 4 * (2 * c["B"] + 1)
        if c["kind"] == "append":
            return {"bytes": b + rows * row, "flops": rows * H * c["rot"] * 3}
        back = sum(min(c["back"], l + n) for l, n in zip(lens, counts))
        return {"bytes": b + rows * H * 144 + back * H * 144 + c["B"] * c["back"] * row,
                "flops": rows * H * (c["rot"] * 3 + 4 * D) + back * H * 4 * D}
    if c["kind"] == "commit4":
        L, B, R, H = c["L"], c["B"], c["R"], c["Hkv"]
        n = B * (R + 1) / 2  # a path holds one to R rows, each number as often
        return {"bytes": L * H * (n * (512 + 2 * 144) + B * R * 512) + B * (R + 4) * 4, "flops": L * H * n * 8 * D}
    if c["kind"] == "attn4":
        B, R, Hq, H = c["B"], c["R"], c["Hq"], c["Hkv"]
        t = sum(_lens(c))
        return {"bytes": t * H * 144 + 4 * B * R * Hq * D + 4 * B * R * H * D, "flops": 4 * R * Hq * D * (t + B * (R + 1) / 2)}
    B, R, V = c["B"], c["R"], c["V"]
    e = B * R * V
    return {"bytes": e * (8 if c["out"] else 4) + (e / 8 if c["mask"] else 0) + B * R * ((V + 127) // 128) * 8 + B * (c["H"] + 2 * c["bias"]) * 4,
            "flops": e * 4}


# ---------------------------------------------------------------------------------------------------------------------
# exact values
# ---------------------------------------------------------------------------------------------------------------------

def _fp64(x):
    return x.detach().cpu().to(torch.float64).numpy()


def _bf16_of(x):
    """float64 -> the nearest bf16 (ties to even), as float64: 8 significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256) / 256, e)


def _held4(x):
    """The values (float64) a 4-bit cache holds for bf16 rows [..., 128]."""
    g = x.reshape(*x.shape[:-1], 4, 32)
    a = np.abs(g).max(-1, keepdims=True)
    m, e = np.frexp(a / 7)
    s = np.ldexp(np.ceil(m * 16) / 16, e)  # up to 4 significant bits
    q = np.clip(np.rint(g / np.where(s > 0, s, 1)), -7, 7)
    return (q * s).reshape(x.shape)


def _read4(blk, is_v):
    """The values (float64 [n, 64, 128]) of n blocks (numpy uint8 [n, 4608]): each one's code and scale looked up by its place."""
    sc = (np.ascontiguousarray(blk[:, 4096:]).view("<u2").astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    p, d = np.arange(64)[:, None], np.arange(128)[None, :]
    e = p % 8 if is_v else d % 8
    bit = 4 * (e // 2) + 16 * (e % 2)
    byte = (p // 8 * 512 + d * 4 if is_v else d // 32 * 1024 + p * 16 + d % 32 // 8 * 4) + bit // 8
    c = (blk[:, byte] >> (bit % 8).astype(np.uint8)) & 15
    return (c.astype(np.float64) - 8) * sc[:, d // 32 * 64 + p if is_v else p * 4 + d // 32]


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


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] in ("append", "append4"):
        counts, lens = _counts(c), _lens(c)
        tab, k, v, rope = s["table"].cpu().numpy(), _fp64(s["k"]), _fp64(s["v"]), _fp64(s["rope"])
        four = c["kind"] == "append4"
        if four:
            kp, vp = s["k_pool"].cpu().numpy(), s["v_pool"].cpu().numpy()
            ko = np.zeros((c["B"], c["Hkv"], c["back"], D))
            vo = np.zeros_like(ko)
        else:
            kp, vp = _fp64(s["k_pool"]), _fp64(s["v_pool"])
        i0 = 0
        for b, (l, n) in enumerate(zip(lens, counts)):
            pos = np.arange(l, l + n)
            kr, vr = _turned(k[i0:i0 + n], pos, rope, c["pairs"]), v[i0:i0 + n]
            i0 += n
            if not four:
                kp[tab[b, pos // PAGE], :, pos % PAGE], vp[tab[b, pos // PAGE], :, pos % PAGE] = kr, vr
                continue
            st = max(0, l + n - c["back"])
            if st < l:
                pg = tab[b, st // PAGE:_pages(l)]
                for h in range(c["Hkv"]):
                    ko[b, h, :l - st] = _read4(kp[pg, h], False).reshape(-1, D)[st % PAGE:][:l - st]
                    vo[b, h, :l - st] = _read4(vp[pg, h], True).reshape(-1, D)[st % PAGE:][:l - st]
            lo = max(st, l)
            ko[b, :, lo - st:l + n - st] = _held4(_bf16_of(kr[lo - l:])).transpose(1, 0, 2)
            vo[b, :, lo - st:l + n - st] = _held4(vr[lo - l:]).transpose(1, 0, 2)
        return [ko, vo] if four else [kp, vp]
    if c["kind"] == "commit4":
        lens, path, m = _lens(c), s["path"].cpu().numpy(), s["n_acc"].cpu().numpy()
        got = []
        for blk in (s["k_blk"], s["v_blk"]):
            x = _fp64(blk)
            y = np.zeros_like(x)
            for b in range(c["B"]):
                y[:, b, :, :m[b] + 1] = _held4(x[:, b][:, :, path[b, :m[b] + 1]])
            got.append(y)
        return got + [None]
    if c["kind"] == "attn4":
        B, R, Hq, H = c["B"], c["R"], c["Hq"], c["Hkv"]
        G, lens = Hq // H, _lens(c)
        if 4 * R * Hq * D * sum(lens) > 3e11:
            return None
        out = torch.zeros(B, R, Hq, D, dtype=torch.float64, device="cuda")
        e = torch.arange(8, device="cuda")
        sh = 4 * torch.div(e, 2, rounding_mode="floor") + 16 * (e % 2)
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
                kb, vb = s["k_pool"][pg, h], s["v_pool"][pg, h]
                n = len(pg)
                kw = kb[:, :4096].contiguous().view(torch.int32).view(n, 4, 64, 4, 1).long()
                vw = vb[:, :4096].contiguous().view(torch.int32).view(n, 8, 1, 128).long()
                ks = kb[:, 4096:].contiguous().view(torch.bfloat16).view(n, 64, 4, 1).double()
                vs = vb[:, 4096:].contiguous().view(torch.bfloat16).view(n, 4, 64).permute(0, 2, 1)[..., None].double()
                kc = torch.div(kw, 2 ** sh, rounding_mode="floor").remainder(16).double() - 8      # [n, 4, 64, 4, 8]
                vc = torch.div(vw, (2 ** sh)[:, None], rounding_mode="floor").remainder(16).double() - 8   # [n, 8, 8, 128]
                kk = (kc.permute(0, 2, 1, 3, 4).reshape(n, 64, 4, 32) * ks).reshape(n * 64, D)[:t]
                vv = (vc.reshape(n, 64, 4, 32) * vs).reshape(n * 64, D)[:t]
                kk, vv = torch.cat([kk, s["k_blk"][b, h].double()]), torch.cat([vv, s["v_blk"][b, h].double()])
                qq = s["q"][b, :, h * G:(h + 1) * G].double()
                z = torch.einsum("rgd,td->rgt", qq, kk) / D ** 0.5
                z = torch.where(see[:, None, :], z, torch.full((), NEG, dtype=torch.float64, device="cuda"))
                out[b, :, h * G:(h + 1) * G] = torch.einsum("rgt,td->rgd", torch.softmax(z, -1), vv)
        return out
    if not c["out"]:
        return None
    B, R, V = c["B"], c["R"], c["V"]
    x = s["logits"].double()
    hist, hl, pl, tok = (s[n].cpu().numpy() for n in ("hist", "hist_len", "prompt_len", "tok"))
    rep, fr, pr = (_fp64(s[n]) for n in ("rep", "freq", "pres"))
    par = None if s["parent"] is None else s["parent"].cpu().numpy()
    for b in range(B):
        before = np.bincount(hist[b, pl[b]:hl[b]], minlength=V)
        asked = np.zeros(V, bool)
        asked[hist[b, :pl[b]]] = True
        for j in range(R):
            n = before.copy()
            i = j
            while i >= 0:
                n[tok[b, i]] += 1
                i = i - 1 if par is None else int(par[b, i])
            ids = np.nonzero(asked | (n > 0))[0]
            at, cnt = torch.from_numpy(ids).cuda(), torch.from_numpy(n[ids]).cuda().double()
            y = x[b, j, at]
            y = torch.where(y > 0, y / float(rep[b]), y * float(rep[b])) - float(fr[b]) * cnt
            x[b, j, at] = y - float(pr[b]) * (cnt > 0)
        if s["bias_off"] is not None:
            o = s["bias_off"].cpu().numpy()
            x[b][:, s["bias_tok"][o[b]:o[b + 1]].long()] += s["bias_val"][o[b]:o[b + 1]].double()
    if s["mask"] is not None:
        for k in range(32):
            cols = x[..., k::32]
            cols.masked_fill_(((s["mask"][..., : cols.shape[-1]] >> k) & 1) == 0, NEG)
    return [x, None]


if __name__ == "__main__":
    for one in listed() + [draw(random.Random(k)) for k in range(12)]:
        print(one, work(one))
