"""The cache and logits calls together, as a server makes them: prompts filled in,
verify rounds over the 4-bit cache with the sampling controls and the acceptance,
eager, captured and on other streams; and where offsets pass 32 bits."""
import sys
import threading

import numpy as np
import pytest
import torch

import _serving_ref as ref
from test_gpu_q4 import bf, i32, random_pool, tol

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
    """One layer: its 4-bit cache, an LM head and the controls of three sequences."""

    def __init__(self, seed=0):
        r = self.r = np.random.default_rng(seed)
        self.P = B * MP + 2
        self.table_n = r.permutation(self.P)[: B * MP].reshape(B, MP).astype(np.int32)
        self.table = i32(self.table_n)
        self.kp, self.vp = (torch.from_numpy(random_pool(r, 1, self.P, H, is_v=x)).cuda() for x in (False, True))
        self.length = i32([0] * B)
        self.rope = ref.rope_table(MP * 64, 128)
        self.W = bf(r.standard_normal((HID, V)) / 8).cuda()
        self.hist_n = r.integers(0, V, (B, 64)).astype(np.int32)
        self.hist = i32(self.hist_n)
        self.hist_len = i32([0] * B)
        self.controls_n = dict(prompt_len=np.array([3, 0, 9], np.int32), repetition=np.array([1.2, 1.0, 1.5], np.float32),
                               frequency=np.array([0.3, 0.0, 0.1], np.float32), presence=np.array([0.2, 0.4, 0.0], np.float32))
        self.controls = {k: torch.from_numpy(v).cuda() for k, v in self.controls_n.items()}
        self.mask_n = r.integers(-2 ** 31, 2 ** 31, (B, R, (V + 31) // 32)).astype(np.int32)
        self.mask = torch.from_numpy(self.mask_n).cuda()

    def inputs(self):
        r = self.r
        q, kb, vb = (ref.bf16_round(r.standard_normal(s)) for s in ((B, R, HQ, 128), (B, H, R, 128), (B, H, R, 128)))
        return q, kb, vb, r.integers(0, V, (B, R)).astype(np.int32)

    def round(self, sv, q, kb, vb, tok, parent=None, commit=True):
        """One verify round; every step is one of the library's calls."""
        attn = sv.verify_attn_q4(q, self.kp[0], self.vp[0], self.table, self.length, kb, vb, parent)
        raw = sv.lm_head(attn.view(B * R, HID), self.W).view(B, R, V)
        out, keys = sv.logits_process(raw, tok=tok, parent=parent, hist=self.hist, hist_len=self.hist_len, mask=self.mask,
                                      write_argmax=True, **self.controls)
        acc = sv.accept_greedy_commit(keys, tok, V, parent)
        if commit:
            sv.kv_commit_q4(self.kp, self.vp, self.table, kb[None], vb[None], acc[2], acc[0], self.length)
        return attn, raw, out, keys, *acc


def fill(sv, s, lens):
    """Prompts of ragged lengths: into the cache and the history."""
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = ref.bf16_round(s.r.standard_normal((2, off[-1], H, 128)))
    before = [ints(p)[0] for p in (s.kp, s.vp)]
    fused = torch.cat([bf(k), bf(v)], 1).cuda()       # K and V as slices of a projection's rows
    sv.kv_append_q4(fused[:, :H], fused[:, H:], i32(off), s.kp[0], s.vp[0], s.table, s.length, rope=torch.from_numpy(s.rope).cuda())
    want = ref.append_q4(k, v, off, *before, s.table_n, [0] * B, s.rope, False, MP * 64)
    assert all(np.array_equal(ints(p)[0], w) for p, w in zip((s.kp, s.vp), want))
    s.length.copy_(i32(lens))
    s.hist_len.copy_(i32([min(n, 64) for n in lens]))


def on_gpu(q, kb, vb, tok):
    return bf(q).cuda(), bf(kb).cuda(), bf(vb).cuda(), i32(tok)


@pytest.mark.parametrize("is_tree", [False, True])
def test_a_prompt_and_verify_rounds(sv, is_tree):
    s = Server(1)
    lens = [70, 0, 125]
    fill(sv, s, lens)
    parent = np.array([[-1, 0, 0, 1], [-1, 0, 1, 2], [-1, 0, 1, 1]], np.int32) if is_tree else None
    gpar = None if parent is None else i32(parent)
    accepted = 0
    for turn in range(3):
        q, kb, vb, tok = s.inputs()
        ln, hl = ints(s.length), ints(s.hist_len)
        kp, vp = ints(s.kp), ints(s.vp)
        controls = dict(hist=s.hist_n, hist_len=hl, mask=s.mask_n, **s.controls_n)
        # drafts that pass in part: the target's own choices, but the last row of sequence `turn`
        raw = ints(s.round(sv, *on_gpu(q, kb, vb, tok), gpar, commit=False)[1])
        for j in range(1, R):
            y = ref.logits(raw, tok=tok, parent=parent, **controls)
            up = np.full(B, j - 1) if parent is None else parent[:, j]
            tok[:, j] = y[np.arange(B), up].argmax(-1)
        tok[turn, R - 1] = (tok[turn, R - 1] + 1) % V
        attn, raw, out, keys, n_acc, out_tok, path = s.round(sv, *on_gpu(q, kb, vb, tok), gpar)
        # attention over what the cache holds
        ctx = [ref.gather_q4(p, s.table_n, [0] * B, ln, MP * 64, x)[0] for p, x in ((kp, False), (vp, True))]
        for b in range(B):
            want, wgt, big = ref.attention(q[b], ctx[0][b, :, :ln[b]], ctx[1][b, :, :ln[b]], kb[b], vb[b],
                                           None if parent is None else parent[b:b + 1], 128 ** -0.5)
            assert np.all(np.abs(attn[b].double().cpu().numpy() - want) <= tol(want, wgt, big, ln[b] + R))
        # the controls, bit for bit, and the keys of what they leave
        y = ref.logits(ints(raw), tok=tok, parent=parent, **controls)
        assert np.array_equal(ints(out), y)
        assert np.array_equal(ints(keys), ref.argmax_keys(y.reshape(B * R, V)))
        # greedy acceptance, as over the logits themselves
        again = sv.accept_greedy(out, i32(tok), gpar)
        assert all(torch.equal(x, z) for x, z in zip((n_acc, out_tok, path), again))
        accepted += int(n_acc.sum())
        # the accepted rows are in, nothing else changed
        wk, wv, wl = ref.commit_q4(kp, vp, s.table_n, kb[None], vb[None], ints(path), ints(n_acc), ln)
        assert np.array_equal(ints(s.kp), wk) and np.array_equal(ints(s.vp), wv) and np.array_equal(ints(s.length), wl)
    assert accepted >= 3 * (R - 2)
    assert sv.get_device_error() == 0


def test_bf16_prompt_then_paged_verify(sv):
    """The bf16 cache filled by rows is the one that verify_attn_paged reads and
    kv_commit_paged goes on from: as if the rows had been committed."""
    r = np.random.default_rng(2)
    lens, P = [70, 1, 125], B * MP + 2
    table = i32(r.permutation(P)[: B * MP].reshape(B, MP))
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = (bf(x).cuda() for x in r.standard_normal((2, off[-1], H, 128)))
    pools = [torch.zeros(1, P, H, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    length = i32([0] * B)
    sv.kv_append_paged(k, v, i32(off), pools[0][0], pools[1][0], table, length)
    # the same rows through the commit, a block of at most 64 at a time
    done = np.zeros(B, np.int64)
    other = i32([0] * B)
    while (done < lens).any():
        n = np.minimum(64, lens - done)
        blk = torch.zeros(2, 1, B, H, 64, 128, dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            for w, x in enumerate((k, v)):
                blk[w, 0, b, :, :n[b]] = x[off[b] + done[b]: off[b] + done[b] + n[b]].transpose(0, 1)
        path = i32([list(range(64))] * B)
        keep = other.clone()
        sv.kv_commit_paged(pools[2], pools[3], table, blk[0].contiguous(), blk[1].contiguous(), path,
                           i32(np.maximum(n - 1, 0)), other)
        other.copy_(torch.where(i32(n) > 0, other, keep))      # a sequence that is done takes a row too many: not counted
        done += n
    length.copy_(i32(lens))
    assert torch.equal(other, length)
    mk = lambda *s: bf(r.standard_normal(s)).cuda()  # noqa: E731
    q, kb, vb = mk(B, R, HQ, 128), mk(B, H, R, 128), mk(B, H, R, 128)
    one = sv.verify_attn_paged(q, pools[0][0], pools[1][0], table, length, kb, vb)
    two = sv.verify_attn_paged(q, pools[2][0], pools[3][0], table, length, kb, vb)
    assert torch.equal(one, two)
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
    for turn in range(3):
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


def test_two_graphs_at_once(sv):
    """Two captured attentions share no scratch: replayed together on two streams
    beside an eager one, each gives its own result."""
    r = np.random.default_rng(5)
    P, t, n = 260, 16600, 3      # (long enough that the pages are split over all SMs)
    kp, vp = (torch.from_numpy(random_pool(r, P, H, is_v=x)).cuda() for x in (False, True))
    table, length = i32([list(range(P))]), i32([t])
    mk = lambda *s: bf(r.standard_normal(s)).cuda()  # noqa: E731
    qs, kb, vb = [mk(1, R, HQ, 128) for _ in range(n)], mk(1, H, R, 128), mk(1, H, R, 128)
    assert sv.verify_attn_q4_workspace(1, R, HQ, H, 128, P * 64) > 0
    want = [sv.verify_attn_q4(q, kp, vp, table, length, kb, vb) for q in qs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(n)]
    for q, st in zip(qs[:2], streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(sv.verify_attn_q4(q, kp, vp, table, length, kb, vb))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(50):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager = sv.verify_attn_q4(qs[2], kp, vp, table, length, kb, vb, stream=streams[2])
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


def _split_attention(sv, seed, n):
    """n calls (their q's and results) whose pages are split over all SMs, so that
    each makes two launches with scratch between them."""
    r = np.random.default_rng(seed)
    P, t = 260, 16600
    kp, vp = (torch.from_numpy(random_pool(r, P, H, is_v=x)).cuda() for x in (False, True))
    mk = lambda *s: bf(r.standard_normal(s)).cuda()  # noqa: E731
    rest = (kp, vp, i32([list(range(P))]), i32([t]), mk(1, H, R, 128), mk(1, H, R, 128))
    assert sv.verify_attn_q4_workspace(1, R, HQ, H, 128, P * 64) > 0
    qs = [mk(1, R, HQ, 128) for _ in range(n)]
    want = [sv.verify_attn_q4(q, *rest) for q in qs]
    torch.cuda.synchronize()
    return qs, rest, want


def test_two_threads_on_one_stream(sv):
    """Threads that share a stream (torch's default one) come between each other's
    launches: each call's scratch is its own."""
    qs, rest, want = _split_attention(sv, 12, 4)
    start, differ = threading.Barrier(len(qs)), [None] * len(qs)
    outs = [[torch.empty_like(want[0]) for _ in range(1500)] for _ in qs]

    def work(i):
        start.wait()
        for o in outs[i]:
            sv.verify_attn_q4(qs[i], *rest, out=o)
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
    """What a call took for its scratch is free again afterwards, on every stream."""
    qs, rest, want = _split_attention(sv, 13, 1)
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        with torch.cuda.stream(torch.cuda.Stream()):
            out = sv.verify_attn_q4(qs[0], *rest)
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
        q, kb, vb, tok = on_gpu(*s.inputs())
        off = i32([0, 3, 3, 9])
        k, v = (bf(x).cuda() for x in s.r.standard_normal((2, 9, H, 128)))
        pool = torch.zeros(2, s.P, H, 64, 128, dtype=torch.bfloat16, device="cuda")
        raw = torch.randn(B, R, V, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
        n_acc, path = i32([1, 0, 3]), i32([[0, 1, 2, 3]] * B)
        torch.cuda.synchronize()
        sv.kv_append_paged(k, v, off, pool[0], pool[1], s.table, s.length, stream=stream)
        sv.kv_append_q4(k, v, off, s.kp[0], s.vp[0], s.table, s.length, stream=stream)
        attn = sv.verify_attn_q4(q, s.kp[0], s.vp[0], s.table, s.length, kb, vb, stream=stream)
        out, keys = sv.logits_process(raw, tok=tok, hist=s.hist, hist_len=s.hist_len, write_argmax=True, stream=stream)
        sv.kv_commit_q4(s.kp, s.vp, s.table, kb[None], vb[None], path, n_acc, s.length, stream=stream)
        rows = sv.kv_gather_q4(s.kp, s.vp, s.table, i32([0] * B), s.length, 8, stream=stream)
        (stream or torch.cuda.current_stream()).synchronize()
        got.append([pool, s.kp, s.vp, attn, out, keys, s.length, *rows])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_cache_ready_sees_what_came_before_the_last_kernel(sv):
    """cache_ready allows reading the cache under the preceding kernel, not under
    the one before that: a commit, an unrelated attention, then one over the
    committed cache."""
    r = np.random.default_rng(9)
    layers, b, n, mp = 28, 8, 9, 8
    P = b * mp
    table = i32(np.arange(P).reshape(b, mp))
    pools = [torch.from_numpy(random_pool(r, layers, P, H, is_v=x)).cuda() for x in (False, True)]
    keep = [p.clone() for p in pools]
    blk = [torch.randn(layers, b, H, n, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    mk = lambda *s: bf(r.standard_normal(s)).cuda()  # noqa: E731
    q, kb, vb = mk(b, R, HQ, 128), mk(b, H, R, 128), mk(b, H, R, 128)
    other = [torch.from_numpy(random_pool(r, 2, H, is_v=x)).cuda() for x in (False, True)]
    small = (mk(1, R, HQ, 128), *other, i32([[0, 1]]), i32([100]), mk(1, H, R, 128), mk(1, H, R, 128))
    length, start = i32([100 + 30 * i for i in range(b)]), i32([100 + 30 * i for i in range(b)])
    path, n_acc = i32([list(range(n))] * b), i32([n - 1] * b)

    def chain(ready, sync):
        sv.kv_commit_q4(*pools, table, *blk, path, n_acc, length)
        sync()
        sv.verify_attn_q4(*small)
        sync()
        return sv.verify_attn_q4(q, pools[0][-1], pools[1][-1], table, length, kb, vb, cache_ready=ready)

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
    """Under inference mode and outside, the outputs can be written, viewed and
    dropped one by one."""
    r = np.random.default_rng(11)
    kp, vp = (torch.from_numpy(random_pool(r, 1, 2, H, is_v=x)).cuda() for x in (False, True))
    want = sv.kv_gather_q4(kp, vp, i32([[0, 1]]), i32([0]), i32([100]), 70)
    for mode in (torch.inference_mode, torch.no_grad, torch.enable_grad):
        with mode():
            k, v = sv.kv_gather_q4(kp, vp, i32([[0, 1]]), i32([0]), i32([100]), 70)
            assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and k.is_contiguous() and v.is_contiguous()
            k.view(-1)[0] = 5.0
            v.mul_(2)
            assert torch.equal(v, want[1] * 2) and k[0, 0, 0, 0, 0] == 5
            assert not k.requires_grad and k.dtype == torch.bfloat16
            del k
            assert torch.equal(v, want[1] * 2)
            out = sv.verify_attn_q4(bf(r.standard_normal((1, R, HQ, 128))).cuda(), kp[0], vp[0], i32([[0, 1]]), i32([100]),
                                    bf(r.standard_normal((1, H, R, 128))).cuda(), bf(r.standard_normal((1, H, R, 128))).cuda())
            out.add_(1)


# ---------------------------------------------------------------------------
# refusals of the binding
# ---------------------------------------------------------------------------

def _calls(sv):
    """Every call with its arguments by name (all in order)."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    n, u8, f32 = torch.int32, torch.uint8, torch.float32
    base = dict(page_table=z(B, MP, d=n), length=z(B, d=n))
    pools = lambda *s: dict(k_pool=z(*s, d=u8), v_pool=z(*s, d=u8))  # noqa: E731
    rows = dict(k=z(5, H, 128), v=z(5, H, 128), row_off=z(B + 1, d=n), rope=z(256, 128, d=f32))
    return {
        "kv_append_paged": (sv.kv_append_paged, dict(rows, k_pool=z(9, H, 64, 128), v_pool=z(9, H, 64, 128), **base)),
        "kv_append_q4": (sv.kv_append_q4, dict(rows, **pools(9, H, 4608), **base)),
        "kv_commit_q4": (sv.kv_commit_q4, dict(pools(2, 9, H, 4608), k_blk=z(2, B, H, R, 128), v_blk=z(2, B, H, R, 128),
                                               path=z(B, R, d=n), n_acc=z(B, d=n), **base)),
        "kv_gather_q4": (sv.kv_gather_q4, dict(pools(2, 9, H, 4608), start=z(B, d=n), n=7, k_out=z(2, B, H, 7, 128),
                                               v_out=z(2, B, H, 7, 128), **base)),
        "verify_attn_q4": (sv.verify_attn_q4, dict(q=z(B, R, HQ, 128), k_blk=z(B, H, R, 128), v_blk=z(B, H, R, 128),
                                                   parent=torch.tensor([[-1, 0, 1, 2]] * B, dtype=n, device="cuda"),
                                                   out=z(B, R, HQ, 128), **pools(9, H, 4608), **base)),
        "logits_process": (sv.logits_process, dict(
            logits=z(B, R, V, d=f32), tok=z(B, R, d=n), hist=z(B, 8, d=n), hist_len=z(B, d=n), prompt_len=z(B, d=n),
            repetition=z(B, d=f32) + 1, frequency=z(B, d=f32), presence=z(B, d=f32), bias_off=z(B + 1, d=n), bias_tok=z(5, d=n),
            bias_val=z(5, d=f32), mask=z(B, R, 32, d=n), out=z(B, R, V, d=f32), argmax=z(B * R, 8, d=torch.int64))),
    }


@pytest.mark.parametrize("name", ["kv_append_paged", "kv_append_q4", "kv_commit_q4", "kv_gather_q4", "verify_attn_q4",
                                  "logits_process"])
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
        if v.shape != torch.Size([1]):
            with pytest.raises(ValueError):
                f(**{**a, k: apart})
        if k not in ("bias_tok", "bias_val", "hist", "rope", "page_table"):     # (these set their own width)
            wider = torch.cat([v, v], -1)
            with pytest.raises((ValueError, sv.SVError)):
                f(**{**a, k: wider})
    torch.cuda.synchronize()
    assert all(torch.equal(v, a[k]) for k, v in keep.items())
    assert sv.get_device_error() == 0


def test_other_refusals_of_the_binding(sv):
    c = _calls(sv)
    f, a = c["logits_process"]
    with pytest.raises(ValueError):
        f(**{**a, "hist_len": None})
    with pytest.raises(ValueError):
        f(**{**a, "bias_val": None})
    b = 100      # more units than clusters: the partials need scratch
    need = sv.verify_attn_q4_workspace(b, R, HQ, H, 128, 64)
    assert need > 0
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    pool = torch.zeros(9, H, 4608, dtype=torch.uint8, device="cuda")
    a = (z(b, R, HQ, 128), pool, pool.clone(), i32([[0]] * b), i32([0] * b), z(b, H, R, 128), z(b, H, R, 128))
    with pytest.raises(ValueError):
        sv.verify_attn_q4(*a, ws=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        sv.verify_attn_q4(*a, ws=torch.empty(need, dtype=torch.uint8))
    sv.verify_attn_q4(*a, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    f, a = c["kv_gather_q4"]
    with pytest.raises(ValueError):
        f(**{**a, "n": -1})
    with pytest.raises(TypeError):
        f(**{**a, "n": 2.5})
    with pytest.raises(sv.SVError):      # R past 128
        z = torch.zeros(1, 1, 1, 129, 128, dtype=torch.bfloat16, device="cuda")
        p = torch.zeros(1, 2, 1, 4608, dtype=torch.uint8, device="cuda")
        sv.kv_commit_q4(p, p.clone(), i32([[0, 1]]), z, z, i32([[0] * 129]), i32([0]), i32([0]))


# ---------------------------------------------------------------------------
# past 32 bits
# ---------------------------------------------------------------------------

def test_cache_offsets_past_32_bits(sv):
    """The last pages of pools of 5.5 GB (4 bits) and 10 GB (bf16): the same
    results as in small pools."""
    pages, Hb = 150000, 8
    r = np.random.default_rng(7)
    t, n = 150, 40
    q, kb, vb = (bf(r.standard_normal(s)).cuda() for s in ((1, R, 16, 128), (1, Hb, R, 128), (1, Hb, R, 128)))
    k, v = (bf(x).cuda() for x in r.standard_normal((2, n, Hb, 128)))
    small = [torch.from_numpy(random_pool(r, 4, Hb, is_v=x)).cuda() for x in (False, True)]
    got = []
    for P in (4, pages):
        kp, vp = (torch.zeros(P, Hb, 4608, dtype=torch.uint8, device="cuda") for _ in range(2))
        kp[-4:], vp[-4:] = small[0], small[1]
        table, length = i32([[P - 3, P - 1, P - 4, P - 2]]), i32([t])
        sv.kv_append_q4(k, v, i32([0, n]), kp, vp, table, length)
        length += n
        out = sv.verify_attn_q4(q, kp, vp, table, length, kb, vb)
        sv.kv_commit_q4(kp[None], vp[None], table, kb[None], vb[None], i32([[0, 1, 2, 3]]), i32([3]), length)
        rows = sv.kv_gather_q4(kp[None], vp[None], table, i32([0]), length, 256)
        got.append([out, *rows, kp[-4:].clone(), vp[-4:].clone(), length])
        if P == pages:
            assert not kp[:-4].any() and not vp[:-4].any()
        del kp, vp
    assert all(torch.equal(x, y) for x, y in zip(*got))
    got = []
    for P in (4, pages // 2):
        kp, vp = (torch.zeros(P, Hb, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        sv.kv_append_paged(k, v, i32([0, n]), kp, vp, i32([[P - 3, P - 1, P - 4, P - 2]]), i32([t]))
        got.append([kp[-4:].clone(), vp[-4:].clone()])
        if P == pages // 2:
            assert not kp[:-4].any() and not vp[:-4].any()
        del kp, vp
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert sv.get_device_error() == 0


def test_logits_past_32_bits(sv):
    """64 x 128 rows of 300000: 2.4e9 logits, processed in place; the last
    sequence is what it is alone."""
    b, rows, vocab = 64, 128, 300000
    x = torch.empty(b, rows, vocab, device="cuda")
    g = torch.Generator("cuda").manual_seed(3)
    for i in range(0, b, 8):
        x[i:i + 8].normal_(generator=g)
    hist = torch.randint(0, vocab, (b, 300), generator=g, device="cuda").to(torch.int32)
    tok = torch.randint(0, vocab, (b, rows), generator=g, device="cuda").to(torch.int32)
    hl = i32([300] * b)
    rep, freq = (torch.full((b,), v, device="cuda") for v in (1.3, 0.2))
    alone = sv.logits_process(x[-1:].clone(), tok=tok[-1:], hist=hist[-1:], hist_len=hl[-1:], repetition=rep[-1:],
                              frequency=freq[-1:], write_argmax=True)
    first = sv.logits_process(x[:1].clone(), tok=tok[:1], hist=hist[:1], hist_len=hl[:1], repetition=rep[:1],
                              frequency=freq[:1], write_argmax=True)
    out, keys = sv.logits_process(x, tok=tok, hist=hist, hist_len=hl, repetition=rep, frequency=freq, out=x, write_argmax=True)
    assert out.data_ptr() == x.data_ptr()
    keys = keys.view(b, rows, -1)
    for i, want in ((0, first), (-1, alone)):
        assert torch.equal(x[i], want[0][0]) and torch.equal(keys[i], want[1].view(rows, -1))
    assert sv.get_device_error() == 0
