"""The calls of the 8-bit cache together, as a server makes them: prompts filled in, verify
rounds with the LM head, the acceptance and the commit, eager, captured, on other streams
and threads; what the binding refuses; and where offsets pass 32 bits."""
import sys
import threading

import numpy as np
import pytest
import torch

import _serving_ref as ref
import _serving_ref8 as ref8
from test_gpu_q8 import bf, dev, i32, lost_of, random_pool, tol, units_of

pytestmark = pytest.mark.gpu

B, R, HQ, H, V, MP = 3, 4, 4, 2, 1000, 4
HID = HQ * 128


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_sv_gb300 import binding
    return binding


def ints(x):
    return x.cpu().numpy()


class Server:
    """One layer: its 8-bit cache, which starts as anything, and an LM head."""

    def __init__(self, seed):
        r = self.r = np.random.default_rng(seed)
        self.P = B * MP + 2
        self.table_n = r.permutation(self.P)[: B * MP].reshape(B, MP).astype(np.int32)
        self.table = i32(self.table_n)
        self.kp, self.vp = (dev(random_pool(r, 1, self.P, H)) for _ in range(2))
        self.length = i32([0] * B)
        self.rope = ref.rope_table(MP * 64, 128)
        self.W = bf(r.standard_normal((HID, V)) / 8).cuda()

    def inputs(self):
        q, kb, vb = (ref.bf16_round(self.r.standard_normal(s)) for s in ((B, R, HQ, 128), (B, H, R, 128), (B, H, R, 128)))
        return q, kb, vb, self.r.integers(0, V, (B, R)).astype(np.int32)

    def round(self, sv, q, kb, vb, tok, parent=None, commit=True):
        attn = sv.verify_attn_q8(q, self.kp[0], self.vp[0], self.table, self.length, kb, vb, parent)
        raw = sv.lm_head(attn.view(B * R, HID), self.W).view(B, R, V)
        acc = sv.accept_greedy(raw, tok, parent)
        if commit:
            sv.kv_commit_q8(self.kp, self.vp, self.table, kb[None], vb[None], acc[2], acc[0], self.length)
        return attn, raw, *acc


def fill(sv, s, lens):
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = ref.bf16_round(s.r.standard_normal((2, off[-1], H, 128)))
    before = [ints(p)[0] for p in (s.kp, s.vp)]
    fused = torch.cat([bf(k), bf(v)], 1).cuda()       # K and V as slices of a projection's rows
    sv.kv_append_q8(fused[:, :H], fused[:, H:], i32(off), s.kp[0], s.vp[0], s.table, s.length, rope=dev(s.rope))
    want = ref8.append(k, v, off, *before, s.table_n, [0] * B, s.rope, False, MP * 64)
    und = ref8.undefined((s.P, H, 64), s.table_n, [0] * B, lens, s.P)
    assert all(ref8.same_pool(ints(p)[0], w, und, x) for p, w, x in zip((s.kp, s.vp), want, (False, True)))
    s.length.copy_(i32(lens))


def on_gpu(q, kb, vb, tok):
    return bf(q).cuda(), bf(kb).cuda(), bf(vb).cuda(), i32(tok)


def cache_of(s, ln):
    """The cache's rows, read here by the plain form: (K, V) for each sequence."""
    pools = [ints(p)[0] for p in (s.kp, s.vp)]
    got = []
    for b in range(B):
        n = (ln[b] + 63) // 64
        got.append([ref8.get_rows(p[s.table_n[b, :n]], x).transpose(1, 0, 2, 3).reshape(H, n * 64, 128)[:, :ln[b]]
                    for p, x in zip(pools, (False, True))])
    return got


@pytest.mark.parametrize("is_tree", [False, True])
def test_a_prompt_and_verify_rounds(sv, is_tree):
    s = Server(1)
    fill(sv, s, [70, 0, 125])
    parent = np.array([[-1, 0, 0, 1], [-1, 0, 1, 2], [-1, 0, 1, 1]], np.int32) if is_tree else None
    gpar = None if parent is None else i32(parent)
    accepted = 0
    for turn in range(3):
        q, kb, vb, tok = s.inputs()
        ln, kp, vp = ints(s.length), ints(s.kp), ints(s.vp)
        # drafts that pass in part: the target's own choices, but the last row of sequence `turn`
        raw = ints(s.round(sv, *on_gpu(q, kb, vb, tok), gpar, commit=False)[1])
        for j in range(1, R):
            up = np.full(B, j - 1) if parent is None else parent[:, j]
            tok[:, j] = raw[np.arange(B), up].argmax(-1)
        tok[turn, R - 1] = (tok[turn, R - 1] + 1) % V
        ctx = cache_of(s, ln)
        attn, _, n_acc, _, path = s.round(sv, *on_gpu(q, kb, vb, tok), gpar)
        # attention over what the cache holds
        for b in range(B):
            want, wgt, big = ref.attention(q[b], *ctx[b], kb[b], vb[b], None if parent is None else parent[b:b + 1], 128 ** -0.5)
            top = 2.0 ** ref8.exponent(max(np.abs(ctx[b][1]).max(initial=0.0), 1e-30) * 2)   # (a run's scale: of all its rows, some of which are held lower)
            bound = tol(want, wgt, big, units_of(q[b], ctx[b][0], kb[b], 128 ** -0.5), ln[b] + R, lost_of(top, ctx[b][1], vb[b], HQ // H))
            assert np.all(np.abs(attn[b].double().cpu().numpy() - want) <= bound)
        accepted += int(n_acc.sum())
        # the accepted rows are in, nothing else changed
        wk, wv, wl = ref8.commit(kp, vp, s.table_n, kb[None], vb[None], ints(path), ints(n_acc), ln)
        und = ref8.undefined((s.P, H, 64), s.table_n, ln, wl, s.P)
        assert np.array_equal(ints(s.length), wl)
        assert ref8.same_pool(ints(s.kp), wk, und, False) and ref8.same_pool(ints(s.vp), wv, und, True)
        # and what is read back is what attention will see
        rows = sv.kv_gather_q8(s.kp, s.vp, s.table, i32([0] * B), s.length, MP * 64)
        for x, p, is_v in zip(rows, (wk, wv), (False, True)):
            assert np.array_equal(x.double().cpu().numpy(), ref8.gather(p, s.table_n, [0] * B, wl, MP * 64, is_v))
    assert accepted >= 3 * (R - 2)
    assert sv.get_device_error() == 0


def test_one_token_at_a_time(sv):
    """Decoding as an engine does it that has no drafts: append a token's row, then attention
    of that row alone over the cache before it; each step against the plain form."""
    s = Server(4)
    fill(sv, s, [62, 15, 0])
    ones = i32(np.arange(B + 1))
    for _ in range(5):
        q, kb, vb, _ = s.inputs()
        q, kb, vb = q[:, :1], kb[:, :, :1], vb[:, :, :1]
        ln, ctx = ints(s.length), cache_of(s, ints(s.length))
        out = sv.verify_attn_q8(bf(q).cuda(), s.kp[0], s.vp[0], s.table, s.length, bf(kb).cuda(), bf(vb).cuda())
        sv.kv_append_q8(bf(kb[:, :, 0]).cuda(), bf(vb[:, :, 0]).cuda(), ones, s.kp[0], s.vp[0], s.table, s.length)
        s.length += 1
        for b in range(B):
            want, wgt, big = ref.attention(q[b], *ctx[b], kb[b], vb[b], None, 128 ** -0.5)
            top = 2.0 ** ref8.exponent(max(np.abs(ctx[b][1]).max(initial=0.0), 1e-30) * 2)
            bound = tol(want, wgt, big, units_of(q[b], ctx[b][0], kb[b], 128 ** -0.5), ln[b] + 1, lost_of(top, ctx[b][1], vb[b], HQ // H))
            assert np.all(np.abs(out[b].double().cpu().numpy() - want) <= bound)
    assert sv.get_device_error() == 0


def test_append_and_commit_write_the_same(sv):
    """Rows put in by the append and by the commit of a block give the same bytes."""
    a, c = Server(5), Server(5)
    for s in (a, c):
        fill(sv, s, [60, 3, 124])
    _, kb, vb, _ = a.inputs()
    rows = [bf(x.transpose(0, 2, 1, 3).reshape(B * R, H, 128)).cuda() for x in (kb, vb)]
    sv.kv_append_q8(*rows, i32(np.arange(B + 1) * R), a.kp[0], a.vp[0], a.table, a.length)
    sv.kv_commit_q8(c.kp, c.vp, c.table, bf(kb).cuda()[None], bf(vb).cuda()[None], i32([list(range(R))] * B), i32([R - 1] * B), c.length)
    got = [sv.kv_gather_q8(s.kp, s.vp, s.table, i32([0] * B), c.length, MP * 64) for s in (a, c)]
    assert all(torch.equal(x, y) for x, y in zip(*got)) and ints(c.length).tolist() == [64, 7, 128]
    assert sv.get_device_error() == 0


def test_captured_rounds_replay(sv):
    """A round captured once and replayed on new inputs gives what eager calls do."""
    s, e = Server(3), Server(3)
    for x in (s, e):
        fill(sv, x, [60, 3, 124])
    static = on_gpu(*s.inputs())
    e.inputs()
    keep = [x.clone() for x in (s.kp, s.vp, s.length)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        s.round(sv, *static)      # outside the graph once: module load, first-call set-up
        for x, y in zip((s.kp, s.vp, s.length), keep):
            x.copy_(y)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs = s.round(sv, *static)
    torch.cuda.synchronize()
    for _ in range(3):
        now = on_gpu(*s.inputs())
        also = on_gpu(*e.inputs())
        for x, y in zip(static, now):
            x.copy_(y)
        g.replay()
        want = e.round(sv, *also)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
        assert torch.equal(s.length, e.length) and torch.equal(s.kp, e.kp) and torch.equal(s.vp, e.vp)
    assert sv.get_device_error() == 0


def test_captured_appends_replay(sv):
    """An append captured once follows the lengths, the offsets and the page table, which
    stay on the device."""
    s, e = Server(8), Server(8)
    n = 40
    k, v = (torch.zeros(n, H, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    off, rope, st = i32([0] * (B + 1)), dev(s.rope), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        sv.kv_append_q8(k, v, off, s.kp[0], s.vp[0], s.table, s.length, rope=rope)
    for counts in ([40, 0, 0], [1, 20, 19], [13, 13, 14], [0, 0, 1]):
        m = sum(counts)
        x, y = (bf(s.r.standard_normal((n, H, 128))).cuda() for _ in range(2))
        k.copy_(x)
        v.copy_(y)
        off.copy_(i32(np.concatenate([[0], np.cumsum(counts)])))
        g.replay()
        sv.kv_append_q8(x[:m], y[:m], off, e.kp[0], e.vp[0], e.table, e.length, rope=rope)
        torch.cuda.synchronize()
        for z in (s, e):
            z.length += i32(counts)
        assert torch.equal(s.kp, e.kp) and torch.equal(s.vp, e.vp)
    assert sv.get_device_error() == 0


def test_nothing_to_do(sv):
    """No rows to append, none to read back, sequences without new rows: nothing changes."""
    s = Server(9)
    keep = [s.kp.clone(), s.vp.clone()]
    z = torch.zeros(0, H, 128, dtype=torch.bfloat16, device="cuda")
    sv.kv_append_q8(z, z, i32([0] * (B + 1)), s.kp[0], s.vp[0], s.table, s.length)
    x = bf(s.r.standard_normal((5, H, 128))).cuda()
    sv.kv_append_q8(x, x, i32([2] * (B + 1)), s.kp[0], s.vp[0], s.table, s.length)      # rows 2 .. 2 of each
    k, v = sv.kv_gather_q8(s.kp, s.vp, s.table, s.length, s.length, 0)
    assert k.shape == v.shape == (1, B, H, 0, 128)
    k, v = sv.kv_gather_q8(s.kp, s.vp, s.table, s.length, s.length, 20)                 # empty sequences
    assert not k.any() and not v.any()
    assert torch.equal(s.kp, keep[0]) and torch.equal(s.vp, keep[1])
    assert sv.get_device_error() == 0


# ---------------------------------------------------------------------------
# streams, threads, graphs
# ---------------------------------------------------------------------------

def _split_attention(sv, seed, n):
    """n calls (their q's and results) whose pages are split over all SMs, so that each makes
    two launches with scratch between them."""
    r = np.random.default_rng(seed)
    P, t = 300, 19100
    mk = lambda *s: bf(r.standard_normal(s)).cuda()  # noqa: E731
    rest = (*(dev(random_pool(r, P, H)) for _ in range(2)), i32([list(range(P))]), i32([t]), mk(1, H, R, 128), mk(1, H, R, 128))
    assert sv.verify_attn_q8_workspace(1, R, HQ, H, 128, P * 64) > 0
    qs = [mk(1, R, HQ, 128) for _ in range(n)]
    want = [sv.verify_attn_q8(q, *rest) for q in qs]
    torch.cuda.synchronize()
    return qs, rest, want


def test_two_graphs_at_once(sv):
    """Two captured attentions share no scratch: replayed together on two streams beside an
    eager one, each gives its own result."""
    qs, rest, want = _split_attention(sv, 5, 3)
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in qs]
    for q, st in zip(qs[:2], streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(sv.verify_attn_q8(q, *rest))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(50):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager = sv.verify_attn_q8(qs[2], *rest, stream=streams[2])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[2])


def test_two_threads_at_once(sv):
    """Two threads, each on its own stream, make rounds at the same time."""
    def work(seed, got):
        with torch.cuda.stream(torch.cuda.Stream()):
            s = Server(seed)
            fill(sv, s, [60, 3, 124])
            for _ in range(5):
                got.append([x.clone() for x in s.round(sv, *on_gpu(*s.inputs()))])
            got.append([s.length.clone(), s.kp.clone(), s.vp.clone()])
            torch.cuda.current_stream().synchronize()
    alone, together = [[], []], [[], []]
    for i in range(2):
        work(10 + i, alone[i])
    th = [threading.Thread(target=work, args=(10 + i, together[i])) for i in range(2)]
    for t in th:
        t.start()
    for t in th:
        t.join()
    for i in range(2):
        assert len(together[i]) == 6
        for x, y in zip(alone[i], together[i]):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
    assert sv.get_device_error() == 0


def test_two_threads_on_one_stream(sv):
    """Threads that share a stream come between each other's launches: each call's scratch
    is its own."""
    qs, rest, want = _split_attention(sv, 12, 4)
    start, differ = threading.Barrier(len(qs)), [None] * len(qs)
    outs = [[torch.empty_like(want[0]) for _ in range(500)] for _ in qs]

    def work(i):
        start.wait()
        for o in outs[i]:
            sv.verify_attn_q8(qs[i], *rest, out=o)
        differ[i] = (torch.stack(outs[i]) != want[i]).flatten(1).any(1).sum()
    th = [threading.Thread(target=work, args=(i,)) for i in range(len(qs))]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)      # (threads that wait for the interpreter get it soon)
    for t in th:
        t.start()
    for t in th:
        t.join()
    sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert [int(d) for d in differ] == [0] * len(qs)
    assert sv.get_device_error() == 0


def test_scratch_is_given_back(sv):
    qs, rest, want = _split_attention(sv, 13, 1)
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        with torch.cuda.stream(torch.cuda.Stream()):
            out = sv.verify_attn_q8(qs[0], *rest)
            torch.cuda.current_stream().synchronize()
            assert torch.equal(out, want[0])
            del out
            torch.cuda.current_stream().synchronize()
    assert torch.cuda.memory_allocated() == before


def test_a_stream_given(sv):
    """Every call enqueues on the stream it is given, outputs and scratch included."""
    st = torch.cuda.Stream()
    a, b = Server(6), Server(6)
    got = []
    for s, stream in ((a, None), (b, st)):
        q, kb, vb, _ = on_gpu(*s.inputs())
        off = i32([0, 3, 3, 9])
        k, v = (bf(x).cuda() for x in s.r.standard_normal((2, 9, H, 128)))
        n_acc, path = i32([1, 0, 3]), i32([[0, 1, 2, 3]] * B)
        torch.cuda.synchronize()
        sv.kv_append_q8(k, v, off, s.kp[0], s.vp[0], s.table, s.length, stream=stream)
        attn = sv.verify_attn_q8(q, s.kp[0], s.vp[0], s.table, i32([3, 0, 6]), kb, vb, stream=stream)
        sv.kv_commit_q8(s.kp, s.vp, s.table, kb[None], vb[None], path, n_acc, s.length, stream=stream)
        rows = sv.kv_gather_q8(s.kp, s.vp, s.table, i32([0] * B), s.length, 8, stream=stream)
        (stream or torch.cuda.current_stream()).synchronize()
        got.append([s.kp, s.vp, attn, s.length, *rows])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_cache_ready_sees_what_came_before_the_last_kernel(sv):
    """cache_ready allows reading the cache under the preceding kernel, not under the one
    before that: a commit, an unrelated attention, then one over the committed cache."""
    r = np.random.default_rng(9)
    layers, b, n, mp = 28, 8, 9, 8
    P = b * mp
    table = i32(np.arange(P).reshape(b, mp))
    pools = [dev(random_pool(r, layers, P, H)) for _ in range(2)]
    keep = [p.clone() for p in pools]
    blk = [torch.randn(layers, b, H, n, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    mk = lambda *s: bf(r.standard_normal(s)).cuda()  # noqa: E731
    q, kb, vb = mk(b, R, HQ, 128), mk(b, H, R, 128), mk(b, H, R, 128)
    other = [dev(random_pool(r, 2, H)) for _ in range(2)]
    small = (mk(1, R, HQ, 128), *other, i32([[0, 1]]), i32([100]), mk(1, H, R, 128), mk(1, H, R, 128))
    length, start = i32([100 + 30 * i for i in range(b)]), i32([100 + 30 * i for i in range(b)])
    path, n_acc = i32([list(range(n))] * b), i32([n - 1] * b)

    def chain(ready, sync):
        sv.kv_commit_q8(*pools, table, *blk, path, n_acc, length)
        sync()
        sv.verify_attn_q8(*small)
        sync()
        return sv.verify_attn_q8(q, pools[0][-1], pools[1][-1], table, length, kb, vb, cache_ready=ready)

    def reset():
        length.copy_(start)
        for p, k in zip(pools, keep):
            p.copy_(k)
    want = chain(False, torch.cuda.synchronize)
    reset()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        got = chain(True, lambda: None)
    for _ in range(30):
        reset()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert sv.get_device_error() == 0


def test_outputs_are_ordinary_tensors(sv):
    r = np.random.default_rng(11)
    kp, vp = (dev(random_pool(r, 1, 2, H)) for _ in range(2))
    want = sv.kv_gather_q8(kp, vp, i32([[0, 1]]), i32([0]), i32([100]), 70)
    for mode in (torch.inference_mode, torch.no_grad, torch.enable_grad):
        with mode():
            k, v = sv.kv_gather_q8(kp, vp, i32([[0, 1]]), i32([0]), i32([100]), 70)
            assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and k.is_contiguous() and v.is_contiguous()
            k.view(-1)[0] = 5.0
            v.mul_(2)
            assert torch.equal(v, want[1] * 2) and k[0, 0, 0, 0, 0] == 5
            assert not k.requires_grad and k.dtype == torch.bfloat16
            del k
            assert torch.equal(v, want[1] * 2)
            out = sv.verify_attn_q8(bf(r.standard_normal((1, R, HQ, 128))).cuda(), kp[0], vp[0], i32([[0, 1]]), i32([100]),
                                    bf(r.standard_normal((1, H, R, 128))).cuda(), bf(r.standard_normal((1, H, R, 128))).cuda())
            out.add_(1)


# ---------------------------------------------------------------------------
# refusals of the binding
# ---------------------------------------------------------------------------

def _calls(sv):
    """Every call with its arguments by name (all in order)."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    n, u8, f32, nb = torch.int32, torch.uint8, torch.float32, sv.KV_Q8_BYTES
    base = dict(page_table=z(B, MP, d=n), length=z(B, d=n))
    pools = lambda *s: dict(k_pool=z(*s, d=u8), v_pool=z(*s, d=u8))  # noqa: E731
    return {
        "kv_append_q8": (sv.kv_append_q8, dict(k=z(5, H, 128), v=z(5, H, 128), row_off=z(B + 1, d=n), rope=z(256, 128, d=f32),
                                               **pools(9, H, nb), **base)),
        "kv_commit_q8": (sv.kv_commit_q8, dict(pools(2, 9, H, nb), k_blk=z(2, B, H, R, 128), v_blk=z(2, B, H, R, 128),
                                               path=z(B, R, d=n), n_acc=z(B, d=n), page_table=torch.arange(B * MP, dtype=n, device="cuda").view(B, MP) % 9,
                                               length=z(B, d=n))),
        "kv_gather_q8": (sv.kv_gather_q8, dict(pools(2, 9, H, nb), start=z(B, d=n), n=7, k_out=z(2, B, H, 7, 128),
                                               v_out=z(2, B, H, 7, 128), **base)),
        "verify_attn_q8": (sv.verify_attn_q8, dict(q=z(B, R, HQ, 128), k_blk=z(B, H, R, 128), v_blk=z(B, H, R, 128),
                                                   parent=torch.tensor([[-1, 0, 1, 2]] * B, dtype=n, device="cuda"),
                                                   out=z(B, R, HQ, 128), **pools(9, H, nb), **base)),
    }


@pytest.mark.parametrize("name", ["kv_append_q8", "kv_commit_q8", "kv_gather_q8", "verify_attn_q8"])
def test_every_tensor_is_checked(sv, name):
    f, a = _calls(sv)[name]
    f(**a)
    keep = {k: v.clone() for k, v in a.items() if torch.is_tensor(v)}
    for k, v in a.items():
        if not torch.is_tensor(v):
            continue
        with pytest.raises(TypeError):
            f(**{**a, k: v.to(torch.float16 if v.dtype != torch.float16 else torch.float32)})
        with pytest.raises(TypeError):
            f(**{**a, k: v.tolist()})
        with pytest.raises(ValueError):
            f(**{**a, k: v.cpu()})
        with pytest.raises(ValueError):
            f(**{**a, k: v[None]})
        apart = torch.stack([v, v], -1)[..., 0]      # the same values, every other element
        with pytest.raises(ValueError):
            f(**{**a, k: apart})
        if k not in ("rope", "page_table"):          # (these set their own width)
            with pytest.raises((ValueError, sv.SVError)):
                f(**{**a, k: torch.cat([v, v], -1)})
    torch.cuda.synchronize()
    assert all(torch.equal(v, a[k]) for k, v in keep.items())
    assert sv.get_device_error() == 0


def test_other_refusals_of_the_binding(sv):
    mp = 300     # long enough that the pages are split over all SMs: the partials need scratch
    need = sv.verify_attn_q8_workspace(1, R, HQ, H, 128, mp * 64)
    assert need > 0
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    pool = torch.zeros(9, H, sv.KV_Q8_BYTES, dtype=torch.uint8, device="cuda")
    a = (z(1, R, HQ, 128), pool, pool.clone(), i32([[0] * mp]), i32([0]), z(1, H, R, 128), z(1, H, R, 128))
    with pytest.raises(ValueError):
        sv.verify_attn_q8(*a, ws=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        sv.verify_attn_q8(*a, ws=torch.empty(need, dtype=torch.uint8))
    sv.verify_attn_q8(*a, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    f, a = _calls(sv)["kv_gather_q8"]
    with pytest.raises(ValueError):
        f(**{**a, "n": -1})
    with pytest.raises(TypeError):
        f(**{**a, "n": 2.5})
    with pytest.raises(ValueError):      # pools of the 4-bit cache
        f(**{**a, "k_pool": torch.zeros(2, 9, H, sv.KV_Q4_BYTES, dtype=torch.uint8, device="cuda")})
    with pytest.raises(sv.SVError):      # R past 128
        z = torch.zeros(1, 1, 1, 129, 128, dtype=torch.bfloat16, device="cuda")
        p = torch.zeros(1, 2, 1, sv.KV_Q8_BYTES, dtype=torch.uint8, device="cuda")
        sv.kv_commit_q8(p, p.clone(), i32([[0, 1]]), z, z, i32([[0] * 129]), i32([0]), i32([0]))


# ---------------------------------------------------------------------------
# past 32 bits
# ---------------------------------------------------------------------------

def test_cache_offsets_past_32_bits(sv):
    """The last pages of pools of 5.3 GB: the same results as in small pools."""
    pages, Hb = 80000, 8
    r = np.random.default_rng(7)
    t, n = 150, 40
    q, kb, vb = (bf(r.standard_normal(s)).cuda() for s in ((1, R, 16, 128), (1, Hb, R, 128), (1, Hb, R, 128)))
    k, v = (bf(x).cuda() for x in r.standard_normal((2, n, Hb, 128)))
    small = [dev(random_pool(r, 4, Hb)) for _ in range(2)]
    got = []
    for P in (4, pages):
        kp, vp = (torch.zeros(P, Hb, sv.KV_Q8_BYTES, dtype=torch.uint8, device="cuda") for _ in range(2))
        kp[-4:], vp[-4:] = small[0], small[1]
        table, length = i32([[P - 3, P - 1, P - 4, P - 2]]), i32([t])
        sv.kv_append_q8(k, v, i32([0, n]), kp, vp, table, length)
        length += n
        out = sv.verify_attn_q8(q, kp, vp, table, length, kb, vb)
        sv.kv_commit_q8(kp[None], vp[None], table, kb[None], vb[None], i32([[0, 1, 2, 3]]), i32([3]), length)
        rows = sv.kv_gather_q8(kp[None], vp[None], table, i32([0]), length, 256)
        got.append([out, *rows, kp[-4:].clone(), vp[-4:].clone(), length])
        if P == pages:
            assert not kp[:-4].any() and not vp[:-4].any()
        del kp, vp
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert sv.get_device_error() == 0


def test_rows_read_back_past_32_bits(sv):
    """A window whose bf16 rows pass 2^32 bytes: every layer like the first, which is read alone."""
    r = np.random.default_rng(8)
    L, P, Hb, n = 600, 32, 8, 2048
    pool = dev(random_pool(r, 1, P, Hb)).expand(L, -1, -1, -1).contiguous()
    table, start, length = i32([list(range(P)), list(range(P))[::-1]]), i32([0, 5]), i32([2048, 2000])
    k, v = sv.kv_gather_q8(pool, pool, table, start, length, n)
    assert k.numel() * 2 > 2 ** 32
    one = sv.kv_gather_q8(pool[:1], pool[:1], table, start, length, n)
    for x, y in zip((k, v), one):
        assert all(torch.equal(x[i], y[0]) for i in (0, 1, 127, 511, L - 1))
    assert sv.get_device_error() == 0
