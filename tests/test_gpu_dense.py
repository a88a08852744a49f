"""The dense cache operators on a B200 against their definitions in 64 bits.

Tolerances.  A score is c <q', k'> of rotated rows, |q'| = |q|, |k'| = |k|; A = c max|q| max|k|
bounds every |score| (Cauchy).  bf16 rounds by at most 2^-8 of a value (half a step), 2^-8/sqrt 3 of
its power of two rms; what a first rounding leaves is rounded again, so two parts are off by 2^-16.
 * fp32 output and the rows kernel: a score's operands are two parts each and the product of the
   two small parts is dropped: three errors of at most 2^-16 of |q' k'|, of independent sign over the
   128 terms, so that a score is off by 2^-16 A with ease (the bound 3 * 2^-16 A would need all of
   them to agree).  A weight e^s / sum e^s moves by at most twice that, relative, and a probability's
   own two parts add 2^-16: |out - exact| <= (2 * 2^-16 A + 2^-16) max|v|.  Over an output's tokens
   the errors are independent as well: their 2-norm stays under 2^-16 of the output's.
 * bf16 output: one rounding of the output and, in the chunk kernel, one of each probability: both
   are 2^-8/sqrt 3 rms of a value's power of two, 1.7e-3 of the value's norm; rotated rows in fp16
   (half a step 2^-11) add 2^-11 sigma to a score of spread sigma <= 2.  Together 2.6e-3; 2^-7 is
   allowed.
 * weights (fp32): each is a sum of softmax weights of two-part scores:
   |w - exact| <= (2 * 2^-16 A + 2^-16) w, and 2^-16 in the norm as above.
"""

import numpy as np
import pytest
import torch

import dense_reference as F
import hierarchical_sparse_attention_build_b200 as R
from test_gpu_paged import paginate

pytestmark = pytest.mark.gpu

BASE = 1.0e6


def params(H, G, **kw):
    return R.params(**{**dict(num_kv_heads=H, num_q_heads=H * G, branching=8, top_k=4, rope_base=BASE), **kw})


class Case:
    """A cache (contiguous or paged) with garbage past every sequence's tokens, and queries."""

    def __init__(self, B, H, G, L, n, seed, page=0, lens=None, spare=0, scale=1.0, garbage=float("nan"), **kw):
        g = torch.Generator().manual_seed(seed)
        cap = L + spare
        if page:
            cap = -(-cap // page) * page
        self.B, self.H, self.G, self.L, self.n, self.cap = B, H, G, L, n, cap
        self.k = (torch.randn(B, H, cap, 128, generator=g) * (0.5 + 1.5 * torch.rand(1, H, 1, 128, generator=g))).bfloat16()
        self.v = torch.randn(B, H, cap, 128, generator=g).bfloat16()
        self.q = (scale * torch.randn(B, n, H * G, 128, generator=g)).bfloat16()
        self.lens = lens if lens is not None else [L] * B
        for b, m in enumerate(self.lens):
            self.k[b, :, m:] = garbage
            self.v[b, :, m:] = garbage
        self.p = params(H, G, **kw)
        self.page = page
        seq = torch.tensor(self.lens, dtype=torch.int64).cuda() if lens is not None else None
        if page:
            kp, vp, self.table = paginate(self.k, self.v, page, seed)
            self.cache = R.TokenCache(self.p, kp, vp, L, seq_len=seq, page_table=self.table)
        else:
            self.cache = R.TokenCache(self.p, self.k.cuda(), self.v.cuda(), L, seq_len=seq)
        self.ws = R.DenseWorkspace(self.p, B, cap, "cuda")
        self.qd = self.q.cuda()

    def attend(self, fp32=True, view=None):
        out = torch.full(self.q.shape, 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        R.dense_attend(self.p, self.cache, self.qd, out, self.ws, view)
        R.check_device_errors(self.ws)
        return out

    def want(self, causal=False, own=False, **kw):
        return F.attend(self.q, self.k, self.v, self.lens, self.G, BASE, causal=causal, own=own, **kw)

    def bound(self):
        L = max(self.lens)
        k = torch.nan_to_num(self.k[:, :, :L].double(), 0, 0, 0)
        v = torch.nan_to_num(self.v[:, :, :L].double(), 0, 0, 0)
        A = self.q.double().norm(dim=-1).max() * k.norm(dim=-1).max() * 128 ** -0.5
        return float((2 * 2.0 ** -16 * A + 2.0 ** -16) * v.abs().max())


def check(got, want, fp32, bound):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    rel = float((got - want).norm() / want.norm().clamp_min(1e-30))
    if fp32:
        assert float((got - want).abs().max()) <= bound, (float((got - want).abs().max()), bound)
        assert rel <= 2.0 ** -16, rel
    else:
        assert rel <= 2.0 ** -7, rel
    assert not got[(want == 0).all(-1)].any()  # a query that sees nothing


SHAPES = [  # B, H, G, L, n, page, lens, view
    (1, 1, 1, 1, 1, 0, None, {}),
    (1, 2, 4, 2, 1, 0, None, {}),
    (2, 1, 8, 17, 1, 0, None, {}),
    (1, 2, 4, 63, 3, 0, None, dict(causal=True, own=True)),
    (1, 2, 4, 64, 3, 0, None, dict(causal=True)),
    (3, 2, 2, 65, 5, 16, [65, 1, 3], dict(causal=True, own=True)),
    (4, 2, 4, 200, 1, 32, [0, 200, 33, 64], {}),
    (1, 1, 1, 300, 300, 0, None, dict(causal=True)),
    (1, 1, 8, 257, 257, 1, None, dict(causal=True, own=True)),
    (2, 3, 4, 1000, 7, 64, [1000, 130], dict(causal=True, own=True)),
    (2, 2, 4, 5000, 1, 0, None, {}),
    (1, 1, 4, 4096, 16, 0, None, {}),
    (2, 2, 1, 3001, 33, 256, [1500, 3001], dict(causal=True)),
    (1, 8, 4, 700, 129, 0, None, dict(causal=True, own=True)),
    (1, 1, 8, 1025, 70, 8, None, dict(causal=True, own=True)),
    # windows: shorter and longer than the cache, sinks inside and outside of them
    (1, 2, 4, 100, 1, 0, None, dict(sinks=4, window=16)),
    (1, 2, 4, 100, 1, 0, None, dict(sinks=4, window=1)),
    (1, 1, 4, 100, 1, 0, None, dict(sinks=0, window=33)),
    (1, 1, 4, 100, 1, 0, None, dict(sinks=100, window=5)),
    (1, 1, 4, 100, 1, 0, None, dict(sinks=17, window=200)),
    (2, 2, 2, 400, 9, 16, [400, 12], dict(sinks=3, window=50, causal=True, own=True)),
    (2, 2, 2, 400, 9, 16, [5, 400], dict(sinks=3, window=50, causal=True, own=True, token_positions=True)),
    (1, 2, 8, 600, 300, 0, None, dict(sinks=20, window=100, causal=True)),
    (1, 2, 4, 2000, 150, 64, None, dict(sinks=70, window=333, causal=True, own=True)),
    (1, 1, 2, 900, 900, 0, None, dict(sinks=2, window=64, causal=True, own=True)),
    (3, 1, 4, 3000, 1, 0, [3000, 200, 70], dict(sinks=64, window=128)),
]


def split_view(view):
    ref = dict(view)
    causal, own = ref.pop("causal", False), ref.pop("own", False)
    v = R.View(sinks=ref.get("sinks", 0), window=ref.get("window", 0), causal=causal, own_token=own,
               token_positions=ref.get("token_positions", False))
    return v, dict(causal=causal, own=own, **ref)


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
def test_attend(shape):
    B, H, G, L, n, page, lens, view = shape
    c = Case(B, H, G, L, n, seed=L * 31 + n, page=page, lens=lens, spare=5)
    v, ref = split_view(view)
    want = c.want(**ref)
    for fp32, kernel in ((True, R.DENSE_AUTO), (False, R.DENSE_AUTO), (False, R.DENSE_ROWS), (False, R.DENSE_CHUNK)):
        v.kernel = kernel
        check(c.attend(fp32, v), want, fp32, c.bound())


def test_same_call_gives_the_same_bits():
    c = Case(2, 2, 4, 3000, 3, seed=5)
    for fp32, kernel in ((True, R.DENSE_ROWS), (False, R.DENSE_ROWS), (False, R.DENSE_CHUNK)):
        v = R.View(causal=True, own_token=True, kernel=kernel)
        first = c.attend(fp32, v)
        for _ in range(3):
            assert torch.equal(first, c.attend(fp32, v))


@pytest.mark.parametrize("view", [dict(causal=True, own=True), dict(causal=True, own=True, sinks=3, window=20)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.0e38])
@pytest.mark.parametrize("n", [6, 150])
def test_hidden_tokens_do_not_reach_a_query(view, bad, n):
    """Tokens some queries of a tile see and others do not hold NaN, infinities or huge numbers:
    the queries that do not see them are what they are without: bit for bit in the rows kernel;
    the chunk kernel (bf16 outputs of long chunks) hands such a tile to the rows kernel, so its
    queries meet the definition within the bf16 bound."""
    L = 400
    c = Case(1, 2, 4, L, n, seed=11)
    v, ref = split_view(view)
    runs = ((True, R.DENSE_ROWS), (False, R.DENSE_ROWS), (False, R.DENSE_CHUNK))

    def attend(fp32, kernel):
        v.kernel = kernel
        return c.attend(fp32, v)

    plain = {r: attend(*r) for r in runs}
    want = c.want(**ref)
    hit = L - n // 2  # a token in the middle of the chunk
    old = L - n - 10  # one before it, that a window leaves behind part way through the chunk
    spots = [hit] + ([old] if "window" in view else [])
    for t in spots:
        c.cache.k_tok[0, :, t] = bad
        c.cache.v_tok[0, :, t] = bad
    blind = [i for i, p in enumerate(F.positions(L, n, True, True))
             if not any(t < p and ("window" not in view or t >= p - 20) for t in spots)]
    for r in runs:
        got = attend(*r)
        if r[1] == R.DENSE_ROWS:
            assert torch.equal(got[0, blind], plain[r][0, blind])
        else:
            check(got[:, blind], want[:, blind], False, 0.0)
        if bad != bad:
            assert torch.isnan(got[0, n // 2 + 1]).any()


def test_a_hidden_value_is_ignored_even_where_its_weight_would_be_zero():
    """Infinite values alone (finite keys): a masked key's weight is zero, and zero times infinity
    must not appear."""
    L, n = 300, 140
    for G, fp32, kernel in ((1, True, R.DENSE_ROWS), (4, False, R.DENSE_CHUNK), (8, False, R.DENSE_CHUNK)):
        c = Case(1, 1, G, L, n, seed=12)
        v = R.View(causal=True, own_token=True, kernel=kernel)
        plain = c.attend(fp32, v)
        c.cache.v_tok[0, :, L - 3] = float("inf")
        got = c.attend(fp32, v)
        if fp32:
            assert torch.equal(got[0, :n - 3], plain[0, :n - 3])
        else:  # the chunk kernel's tile is computed again by the rows kernel
            check(got[:, :n - 3], c.want(causal=True, own=True)[:, :n - 3], False, 0.0)
        assert not torch.isfinite(got[0, n - 3:]).any()


def test_equals_the_sparse_calls_that_keep_everything():
    """top_k = all makes the tree attention dense RoPE attention over the same tokens."""
    g = torch.Generator().manual_seed(3)
    H, G, L, n = 2, 4, 900, 20
    k, v = (torch.randn(1, H, L + n, 128, generator=g).bfloat16().cuda() for _ in range(2))
    kn, vn = (torch.randn(1, n, H, 128, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(1, n, H * G, 128, generator=g).bfloat16().cuda()
    p = params(H, G, top_k=R.TOPK_ALL)
    pooler = torch.eye(128).cuda()
    tree = R.RecsaTree(p, k, v, pooler, L)
    R.build_tree(p, tree)
    ws, dws = R.Workspace(p, L + n, "cuda"), R.DenseWorkspace(p, 1, L + n, "cuda")
    a, b = (torch.empty(1, n, H * G, 128, device="cuda") for _ in range(2))
    R.decode(p, tree, q, a, ws)
    R.dense_attend(p, tree, q, b, dws)
    assert float((a - b).norm() / a.norm()) <= 2.0 ** -16
    R.prefill_chunk(p, tree, kn, vn, q, a, ws)
    twin = R.RecsaTree(p, k.clone(), v.clone(), pooler, L)
    R.build_tree(p, twin)
    R.dense_prefill_chunk(p, twin, kn, vn, q, b, dws)
    assert float((a - b).norm() / a.norm()) <= 2.0 ** -16
    assert twin.length == tree.length == L + n
    assert torch.equal(twin.k_tok, tree.k_tok) and torch.equal(twin.v_tok, tree.v_tok)
    for l in range(1, tree.levels + 1):  # the tree kept up to date as recsa_prefill_chunk keeps it
        n_l = -(-(L + n) // 8 ** l)
        for x, y in zip(tree.level_rows(l), twin.level_rows(l)):
            assert torch.equal(x[:, :, :n_l], y[:, :, :n_l])
    R.check_device_errors(dws)


@pytest.mark.parametrize("page,lens", [(0, None), (16, None), (0, [50, 0, 33]), (32, [50, 7, 0])])
def test_prefill_chunk_appends_then_attends(page, lens):
    B, H, G, L, n = 3, 2, 4, 50, 40
    c = Case(B, H, G, L, n, seed=21, page=page, lens=lens, spare=n + 3)
    g = torch.Generator().manual_seed(22)
    kn, vn = (torch.randn(B, n, H, 128, generator=g).bfloat16() for _ in range(2))
    out = torch.empty(B, n, H * G, 128, device="cuda")
    R.dense_prefill_chunk(c.p, c.cache, kn.cuda(), vn.cuda(), c.qd, out, c.ws, R.View(own_token=True))
    R.check_device_errors(c.ws)
    old = list(c.lens)
    for b in range(B):
        c.k[b, :, old[b]:old[b] + n] = kn[b].transpose(0, 1)
        c.v[b, :, old[b]:old[b] + n] = vn[b].transpose(0, 1)
    c.lens = [m + n for m in old]
    assert c.cache.length == L + n
    if lens is not None:
        assert c.cache.seq_len.tolist() == c.lens
    check(out, c.want(causal=True, own=True), True, c.bound())
    got = F.tokens(c.cache.k_tok.cpu(), c.table, page) if page else c.cache.k_tok.cpu()
    for b in range(B):
        assert torch.equal(got[b, :, :c.lens[b]], c.k[b, :, :c.lens[b]])


@pytest.mark.parametrize("view", [R.View(), R.View(sinks=2, window=30)])
def test_decode_steps_and_their_graph(view):
    """Steps called one by one and replayed from one captured graph: the same bits, and the formula."""
    B, H, G, steps = 3, 2, 4, 6
    g = torch.Generator().manual_seed(31)
    new = [[torch.randn(B, 1, x, 128, generator=g).bfloat16() for x in (H, H, H * G)] for _ in range(steps)]
    got = []
    for graph in (False, True):
        c = Case(B, H, G, 90, 1, seed=30, page=16, lens=[90, 0, 41], spare=10)
        bufs = [x.cuda() for x in new[0]]
        out = torch.empty(B, 1, H * G, 128, device="cuda")

        def step():
            R.dense_decode_step(c.p, c.cache, *bufs, out, c.ws, view)

        if graph:
            start = c.cache.seq_len.clone()
            rows = [x.clone() for x in (c.cache.k_tok, c.cache.v_tok)]
            cg = torch.cuda.CUDAGraph()
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step()
            torch.cuda.current_stream().wait_stream(s)
            c.cache.seq_len.copy_(start)
            c.cache.k_tok.copy_(rows[0])
            c.cache.v_tok.copy_(rows[1])
            with torch.cuda.graph(cg):
                step()
        outs = []
        for x in new:
            for dst, src in zip(bufs, x):
                dst.copy_(src)
            cg.replay() if graph else step()
            outs.append(out.clone())
        R.check_device_errors(c.ws)
        got.append(outs)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert c.cache.seq_len.tolist() == [96, 6, 47]
    for i, x in enumerate(new):
        for b in range(B):
            t = [90, 0, 41][b] + i
            c.k[b, :, t], c.v[b, :, t] = x[0][b, 0], x[1][b, 0]
        c.lens = [m + i + 1 for m in (90, 0, 41)]
        c.q = x[2]
        check(got[0][i], c.want(sinks=view.sinks, window=view.window), True, c.bound())


def test_captured_calls_replay():
    """A chunk, the weights of many and of few rows, and an eviction captured once: replays give the
    eager calls' bits on new inputs, also after eager calls on the same workspace."""
    B, H, G, L, n, keep = 2, 2, 4, 700, 90, 200
    c = Case(B, H, G, L, n, seed=37, lens=[700, 350])
    into = R.TokenCache(c.p, *(torch.zeros(B, H, keep, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)), 0,
                        seq_len=torch.zeros(B, dtype=torch.int64, device="cuda"))
    view, few = R.View(causal=True, own_token=True, kernel=R.DENSE_CHUNK), R.View(causal=True)
    out = torch.empty_like(c.qd)
    q1 = c.qd[:, -2:].contiguous()
    w, w1 = (torch.zeros(B, H, c.cap, device="cuda") for _ in range(2))
    kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")

    def calls():
        R.dense_attend(c.p, c.cache, c.qd, out, c.ws, view)
        R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, view, accumulate=False)
        R.accumulate_weights(c.p, c.cache, q1, w1, c.ws, few, accumulate=False)
        R.evict(c.p, c.cache, w, keep, kept, into=into, sinks=2, recent=8)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        c.qd.normal_()
        q1.copy_(c.qd[:, -2:])
        c.cache.seq_len.copy_(torch.randint(1, L, (B,)))
        c.cache.k_tok.normal_()
        results = []
        for run in (graph.replay, calls):
            for t in (out, w, w1, kept, into.k_tok, into.seq_len):
                t.zero_()
            run()
            results.append([t.clone() for t in (out, w, w1, kept, into.k_tok, into.v_tok, into.seq_len)])
        assert all(torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())) for a, b in zip(*results))
    R.check_device_errors(c.ws)


def test_a_full_sequence_is_flagged_and_kept():
    c = Case(2, 1, 2, 32, 1, seed=33, lens=[32, 10])
    before = c.cache.k_tok.clone()
    x = [torch.randn(2, 1, h, 128).bfloat16().cuda() for h in (1, 1, 2)]
    out = torch.empty(2, 1, 2, 128, device="cuda")
    R.dense_decode_step(c.p, c.cache, *x, out, c.ws)
    with pytest.raises(R.RecsaError) as e:
        R.check_device_errors(c.ws)
    assert e.value.code == 6
    assert c.cache.seq_len.tolist() == [32, 11]
    assert torch.equal(torch.nan_to_num(c.cache.k_tok[0]), torch.nan_to_num(before[0]))
    c.k[1, :, 10], c.v[1, :, 10] = x[0][1, 0].cpu(), x[1][1, 0].cpu()
    c.lens, c.q = [32, 11], x[2].cpu()
    check(out, c.want(), True, c.bound())
    R.check_device_errors(c.ws)


def test_bad_lengths_pages_and_workspaces_are_flagged():
    c = Case(2, 1, 4, 60, 1, seed=34, page=16, lens=[60, 20], garbage=0.0)
    c.cache.seq_len.copy_(torch.tensor([999, -5]))
    c.attend_out = torch.empty(c.q.shape, device="cuda")
    R.dense_attend(c.p, c.cache, c.qd, c.attend_out, c.ws)
    with pytest.raises(R.RecsaError) as e:
        R.check_device_errors(c.ws)
    assert e.value.code == 6
    c.lens = [60, 0]  # clamped
    c.cache.seq_len.copy_(torch.tensor([60, 20]))
    R.check_device_errors(c.ws)
    c.cache.page_table[0, 1] = 10_000
    for f in (lambda: R.dense_attend(c.p, c.cache, c.qd, c.attend_out, c.ws),
              lambda: R.accumulate_weights(c.p, c.cache, c.qd, torch.zeros(2, 1, c.cap, device="cuda"), c.ws)):
        f()
        with pytest.raises(R.RecsaError) as e:
            R.check_device_errors(c.ws)
        assert e.value.code == 6
    # the tokens of the missing page are skipped: sequence 0 sees [0, 16) and [32, 60)
    w = F.weights_of(c.q[0, 0].double(), c.k[0, 0, :60].double(), 60, BASE, 128 ** -0.5)
    w[:, 16:32] = 0
    want = (w / w.sum(-1, keepdim=True)) @ c.v[0, 0, :60].double()
    assert float((c.attend_out[0, 0].double().cpu() - want).abs().max()) <= c.bound()
    raw = R.DenseWorkspace(c.p, 2, c.cap, "cuda")
    raw.buf.zero_()
    R.dense_attend(c.p, c.cache, c.qd, c.attend_out, raw)
    with pytest.raises(R.RecsaError) as e:
        R.check_device_errors(raw)
    assert e.value.code == 6


def test_another_stream_and_two_workspaces():
    c = Case(2, 2, 4, 2000, 2, seed=35)
    ws2 = R.DenseWorkspace(c.p, 2, c.cap, "cuda")
    want = c.attend()
    torch.cuda.synchronize()
    outs = [torch.empty_like(want) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, o, w in zip(streams, outs, (c.ws, ws2)):
            R.dense_attend(c.p, c.cache, c.qd, o, w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("B,H,G,L,n,page,lens,view", [
    (5, 8, 4, 9000, 1, 16, [9000, 17, 0, 4000, 8999], {}),  # long enough for the steps to be dealt out
    (3, 16, 2, 9000, 4, 0, [300, 9000, 2], dict(causal=True, own=True)),
    (40, 8, 8, 1200, 1, 64, [1200 - 29 * i for i in range(40)], {}),
    (5, 8, 4, 9000, 1, 0, [9000, 17, 0, 4000, 8999], dict(sinks=20, window=6000)),
])
def test_uneven_sequences(B, H, G, L, n, page, lens, view):
    c = Case(B, H, G, L, n, seed=L + B, page=page, lens=lens, spare=5)
    v, ref = split_view(view)
    check(c.attend(True, v), c.want(**ref), True, c.bound())
    if not view.get("window"):
        got = torch.zeros(B, H, c.cap, device="cuda")
        R.accumulate_weights(c.p, c.cache, c.qd, got, c.ws, v, accumulate=False)
        want = c.want(want_weights=True, **ref)
        assert float((got.double().cpu() - want).norm() / want.norm()) <= 2.0 ** -16


def test_far_rows_and_far_positions():
    """Rows past 2^31 elements of the cache; positions where an fp32 angle would be worthless."""
    H, G, cap, L = 8, 4, 1 << 20, (1 << 20) - 3
    p = params(H, G)
    k, v = (torch.zeros(3, H, cap, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(40)
    k[2, 5:].normal_(generator=g)
    v[2, 5:].normal_(generator=g)
    q = torch.randn(3, 1, H * G, 128, generator=g, device="cuda").bfloat16()
    cache = R.TokenCache(p, k, v, L)
    ws = R.DenseWorkspace(p, 3, cap, "cuda")
    for view, ref in ((R.View(), {}), (R.View(sinks=4, window=500), dict(sinks=4, window=500)),
                      (R.View(sinks=4, window=500, token_positions=True),
                       dict(sinks=4, window=500, token_positions=True))):
        out = torch.empty(3, 1, H * G, 128, device="cuda")
        R.dense_attend(p, cache, q, out, ws, view)
        R.check_device_errors(ws)
        for h in (5, 7):
            want = F.attend(q[2:, :, h * G:(h + 1) * G], k[2:, h:h + 1], v[2:, h:h + 1], [L], G, BASE, **ref)
            got = out[2:, :, h * G:(h + 1) * G].double()
            assert float((got - want).norm() / want.norm()) <= 2.0 ** -16, (ref, h)


@pytest.mark.parametrize("case", [
    # many items dealt out evenly, several blocks an item, whole items only, ragged and paged
    dict(B=1, H=1, G=4, L=9000, n=64, view=dict(causal=True, own=True)),
    dict(B=1, H=2, G=8, L=5000, n=100, view=dict(causal=True, own=True)),
    dict(B=3, H=2, G=4, L=2100, n=65, lens=[2100, 64, 700], page=16, view=dict(causal=True, own=True)),
    dict(B=3, H=1, G=1, L=700, n=512, lens=[0, 700, 513], view=dict(causal=True)),
    dict(B=2, H=4, G=4, L=4000, n=300, page=1, view=dict(causal=True, own=True)),
    dict(B=1, H=8, G=4, L=1500, n=1400, view=dict(causal=True, own=True)),
    dict(B=1, H=2, G=4, L=3000, n=700, view=dict(causal=True, own=True, sinks=200, window=500)),
    dict(B=2, H=2, G=2, L=3000, n=400, lens=[3000, 130], view=dict(causal=True, own=True, sinks=4, window=128)),
    dict(B=4, H=8, G=4, L=900, n=200, view=dict(causal=True, own=True, sinks=130, window=1)),
    dict(B=2, H=2, G=4, L=600, n=64, view={}),  # many independent queries at the end of the cache
], ids=str)
def test_chunks(case):
    lens = case.get("lens")
    c = Case(case["B"], case["H"], case["G"], case["L"], case["n"], seed=case["L"] + case["n"], page=case.get("page", 0),
             lens=lens, spare=3)
    v, ref = split_view(case["view"])
    v.kernel = R.DENSE_CHUNK
    got = c.attend(False, v)
    check(got, c.want(**ref), False, 0.0)
    for _ in range(2):
        assert torch.equal(got, c.attend(False, v))


def test_empty_caches():
    c = Case(2, 2, 4, 1, 3, seed=80, spare=40)
    c.cache.length = 0
    for fp32, kernel in ((True, R.DENSE_ROWS), (False, R.DENSE_ROWS), (False, R.DENSE_CHUNK)):
        for view in (R.View(kernel=kernel), R.View(causal=True, own_token=True, kernel=kernel)):
            assert not c.attend(fp32, view).any()
    w = torch.full((2, 2, c.cap), 3.0, device="cuda")
    R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws)
    kept = torch.zeros(2, 2, 5, dtype=torch.int32, device="cuda")
    R.evict(c.p, c.cache, w, 5, kept)
    R.check_device_errors(c.ws)
    assert (w == 3.0).all() and (kept == -1).all() and c.cache.length == 0


def test_more_queries_than_the_images_hold():
    """A short cache's workspace holds the rotated rows of a few items at a time."""
    c = Case(1, 1, 8, 128, 700, seed=81)
    check(c.attend(False, R.View(kernel=R.DENSE_CHUNK)), c.want(), False, 0.0)
    want = c.want(want_weights=True)
    w = torch.full((1, 1, c.cap), 0.5, device="cuda")
    for acc in (False, True):
        R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, accumulate=acc)
        assert float((w.double().cpu() / (1 + acc) - want).norm() / want.norm()) <= 2.0 ** -16


def test_more_heads_than_the_images_hold():
    """Long caches whose heads' rotated keys do not fit the workspace together: heads in turn."""
    H, G, L, n = 8, 4, 180001, 80
    p = params(H, G)
    g = torch.Generator(device="cuda").manual_seed(82)
    k, v = (torch.empty(1, H, L, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    q = torch.empty(1, n, H * G, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    cache, ws = R.TokenCache(p, k, v, L), R.DenseWorkspace(p, 1, L, "cuda")
    assert ws.nbytes < 8 * L * 256 + (50 << 20)
    view = R.View(causal=True, own_token=True, kernel=R.DENSE_CHUNK)
    out = torch.empty_like(q)
    R.dense_attend(p, cache, q, out, ws, view)
    w = torch.zeros(1, H, L, device="cuda")
    R.accumulate_weights(p, cache, q[:, -8:].contiguous(), w, ws, view)
    R.check_device_errors(ws)
    for h in (0, 3, 6, 7):
        one = dict(q=q[:, -8:, h * G:(h + 1) * G], k=k[:, h:h + 1], v=v[:, h:h + 1], lens=[L], G=G, base=BASE, causal=True,
                   own=True)
        check(out[:, -8:, h * G:(h + 1) * G], F.attend(**one).cpu(), False, 0.0)
        want = F.attend(want_weights=True, **one)
        assert float((w[:, h:h + 1].double() - want).norm() / want.norm()) <= 2.0 ** -16


def test_chunk_rows_beyond_half_precision():
    """Keys or queries larger than fp16 holds: the tile is computed by the rows kernel."""
    for big_q in (False, True):
        c = Case(1, 2, 4, 500, 80, seed=70)
        c.softmax = 2.0 ** -17  # keeps the scores of such rows in the softmax's range
        c.p = params(2, 4, softmax_scale=c.softmax)
        if big_q:
            c.q[:, 5:9] *= 2.0 ** 24
            c.qd = c.q.cuda()
        else:
            c.k[:, :, 100:140] *= 2.0 ** 17
            c.cache.k_tok.copy_(c.k)
        got = c.attend(False, R.View(causal=True, own_token=True, kernel=R.DENSE_CHUNK))
        check(got, c.want(causal=True, own=True, scale=c.softmax), False, 0.0)


# ---------------------------------------------------------------------------- weights


@pytest.mark.parametrize("B,H,G,L,n,page,lens,view", [
    (1, 1, 1, 1, 1, 0, None, {}),
    (2, 2, 4, 100, 1, 16, [100, 0], {}),
    (2, 2, 4, 700, 3, 0, None, dict(causal=True, own=True)),
    (1, 1, 8, 300, 70, 8, None, dict(causal=True)),
    (3, 2, 2, 65, 80, 0, [65, 10, 33], dict(causal=True, own=True)),
    (1, 8, 4, 2500, 64, 64, None, dict(causal=True, own=True)),
    (2, 1, 4, 5000, 2, 0, None, {}),
    (2, 2, 1, 777, 1, 64, [777, 5], {}),
    (1, 2, 2, 6000, 600, 0, None, dict(causal=True, own=True)),
    (3, 2, 8, 900, 33, 16, [900, 0, 20], dict(causal=True, own=True)),
    (1, 1, 1, 200, 9, 0, None, {}),
])
def test_weights(B, H, G, L, n, page, lens, view):
    c = Case(B, H, G, L, n, seed=L + n, page=page, lens=lens, spare=7)
    v, ref = split_view(view)
    want = F.attend(c.q, c.k, c.v, c.lens, G, BASE, want_weights=True, **ref)
    w = torch.full((B, H, c.cap), 3.0, device="cuda")
    R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, v, accumulate=False)
    R.check_device_errors(c.ws)
    A = c.bound() / float(torch.nan_to_num(c.v[:, :, :max(c.lens)].double(), 0, 0, 0).abs().max())
    got = w.double().cpu()
    for b, m in enumerate(c.lens):
        assert (got[b, :, m:] == 3.0).all()
        d = (got[b, :, :m] - want[b, :, :m]).abs()
        assert (d <= A * want[b, :, :m] + 1e-30).all(), float((d / want[b, :, :m].clamp_min(1e-30)).max())
        if m:
            assert float(d.norm() / want[b, :, :m].norm().clamp_min(1e-30)) <= 2.0 ** -16
    twice = w.clone()
    R.accumulate_weights(c.p, c.cache, c.qd, twice, c.ws, v, accumulate=True)
    for b, m in enumerate(c.lens):
        assert torch.equal(twice[b, :, :m], w[b, :, :m] + w[b, :, :m])
        assert (twice[b, :, m:] == 3.0).all()


@pytest.mark.parametrize("B,G,L,n,lens", [
    (1, 2, 4097, 2, None),  # the last token is seen by no query and opens a step of its own
    (2, 1, 33, 8, [33, 1]),
    (2, 4, 16, 1, [1, 16]),
    (1, 4, 385, 20, None),  # the same in the kernel for more rows
])
def test_weights_of_tokens_no_query_sees(B, G, L, n, lens):
    """Without its own token a chunk's last one is seen by none: its weight is 0, whatever an
    earlier call left in the workspace."""
    c = Case(B, 2, G, L, n, seed=90, lens=lens)
    c.ws.buf[1 << 20:] = 0x41
    w = torch.full((B, 2, c.cap), 3.0, device="cuda")
    R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, R.View(causal=True), accumulate=False)
    R.check_device_errors(c.ws)
    want = c.want(causal=True, want_weights=True)
    for b, m in enumerate(c.lens):
        got = w[b, :, :m].double().cpu()
        assert (got[:, m - 1] == 0).all()
        assert float((got - want[b, :, :m]).norm()) <= 2.0 ** -16 * max(float(want[b, :, :m].norm()), 1.0)


# ---------------------------------------------------------------------------- eviction


def long_tail(shape, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.empty(shape).exponential_(1.0, generator=g) ** 3
    return torch.where(w < 0.02, torch.zeros_like(w), w)


EVICT = [  # B, H, L, keep, sinks, recent, page, lens
    (1, 1, 10, 4, 0, 0, 0, None),
    (1, 1, 10, 1, 0, 0, 0, None),
    (2, 2, 100, 64, 4, 16, 16, [100, 64]),
    (2, 2, 300, 33, 33, 0, 0, [300, 20]),
    (2, 2, 300, 33, 1, 32, 8, [300, 0]),
    (1, 3, 2051, 1024, 4, 64, 0, None),
    (2, 1, 9000, 5000, 4, 100, 64, [8999, 9000]),
    (1, 2, 40000, 39999, 4, 100, 0, None),
    (1, 2, 40000, 300, 0, 0, 256, None),
]


@pytest.mark.parametrize("mode", ["in_place", "into", "into_paged"])
@pytest.mark.parametrize("shape", EVICT, ids=[f"{i}" for i in range(len(EVICT))])
def test_evict(shape, mode):
    B, H, L, keep, sinks, recent, page, lens = shape
    c = Case(B, H, 2, L, 1, seed=L + keep, page=page, lens=lens, spare=5, garbage=9.0)
    w0 = long_tail((B, H, c.cap), seed=keep)
    w0[:, :, L // 2:] *= -1.0 if L == 300 else 1.0  # negative weights order too
    w0[:, :, 3] = float("nan")
    w0[:, :, 5] = float("inf")
    w0[:, :, 6] = -float("inf")
    w = w0.cuda()
    kept = torch.full((B, H, keep), 77, dtype=torch.int32, device="cuda")
    before = [F.tokens(x.cpu(), c.table, page) if page else x.cpu().clone() for x in (c.cache.k_tok, c.cache.v_tok)]
    if mode == "in_place":
        to, tw, tcap = None, w, c.cap
        R.evict(c.p, c.cache, w, keep, kept, into_weights=w, sinks=sinks, recent=recent)
        got_cache = c.cache
        after = [F.tokens(x.cpu(), c.table, page) if page else x.cpu() for x in (c.cache.k_tok, c.cache.v_tok)]
    else:
        tcap = -(-(keep + 3) // 16) * 16
        seq = torch.full((B,), -1, dtype=torch.int64, device="cuda") if lens is not None or mode == "into_paged" else None
        rows = [torch.full((B, H, tcap, 128), 5.0, dtype=torch.bfloat16) for _ in range(2)]
        if mode == "into":
            to = R.TokenCache(c.p, rows[0].cuda(), rows[1].cuda(), 0, seq_len=seq)
        else:
            kp, vp, table = paginate(rows[0], rows[1], 16, seed=1)
            to = R.TokenCache(c.p, kp, vp, 0, seq_len=seq, page_table=table)
        tw = torch.full((B, H, tcap), -1.0, device="cuda")
        R.evict(c.p, c.cache, w, keep, kept, into=to, into_weights=tw, sinks=sinks, recent=recent)
        got_cache = to
        after = [x.cpu() if mode == "into" else F.tokens(x.cpu(), table, 16) for x in (to.k_tok, to.v_tok)]
        now = [F.tokens(x.cpu(), c.table, page) if page else x.cpu() for x in (c.cache.k_tok, c.cache.v_tok)]
        assert all(torch.equal(x, y) for x, y in zip(now, before)) and c.cache.length == L
    torch.cuda.synchronize()
    assert got_cache.length == min(L, keep)
    if got_cache.seq_len is not None:
        assert got_cache.seq_len.tolist() == [min(m, keep) for m in c.lens]
    bits = lambda x: x.view(torch.int32)  # noqa: E731  (NaN weights compare by their bits)
    for b, m in enumerate(c.lens):
        for h in range(H):
            want = F.evict(w0[b, h], m, keep, sinks, recent)
            n = len(want)
            assert kept[b, h].tolist() == want + [-1] * (keep - n)
            for x, y in zip(after, before):
                assert torch.equal(x[b, h, :n], y[b, h, want])
            assert torch.equal(bits(tw[b, h, :n].cpu()), bits(w0[b, h, want]))
            if mode == "in_place":  # slots past the kept rows are left as they were
                for x, y in zip(after, before):
                    assert torch.equal(x[b, h, n:], y[b, h, n:])
            else:
                assert (tw[b, h, n:] == -1.0).all() and all((x[b, h, n:] == 5.0).all() for x in after)


def test_evict_ties_go_to_the_lower_slots():
    for L in (500, 20000):
        c = Case(1, 2, 1, L, 1, seed=1)
        w = torch.zeros(1, 2, c.cap, device="cuda")
        w[:, 1, ::3] = 1.0
        kept = torch.empty(1, 2, 100, dtype=torch.int32, device="cuda")
        R.evict(c.p, c.cache, w, 100, kept, sinks=2, recent=10)
        tail = list(range(L - 10, L))
        assert kept[0, 0].tolist() == list(range(90)) + tail
        assert kept[0, 1].tolist() == F.evict(w[0, 1].cpu(), L, 100, 2, 10)


def test_evict_rebuilds_the_tree():
    """A cache with a tree: after the eviction the tree is the one built over the kept tokens."""
    B, H, L, keep = 2, 2, 700, 300
    for lens in (None, [700, 120]):
        c = Case(B, H, 2, L, 1, seed=50, lens=lens, garbage=0.0)
        pooler = torch.randn(128, 128, generator=torch.Generator().manual_seed(51)).cuda()
        seq = torch.tensor(lens).cuda() if lens else None
        tree = R.RecsaTree(c.p, c.cache.k_tok, c.cache.v_tok, pooler, L, seq_len=seq)
        R.build_tree(c.p, tree)
        kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
        R.evict(c.p, tree, long_tail((B, H, L), 52).cuda(), keep, kept, sinks=4, recent=20)
        twin = R.RecsaTree(c.p, tree.k_tok, tree.v_tok, pooler, keep, seq_len=seq)
        R.build_tree(c.p, twin)
        for b in range(B):
            n = keep if not lens else min(lens[b], keep)
            l = 1
            while n > 8:
                n = -(-n // 8)
                for x, y in zip(tree.level_rows(l), twin.level_rows(l)):
                    assert torch.equal(x[b, :, :n], y[b, :, :n])
                l += 1


# ---------------------------------------------------------------------------- together


@pytest.mark.parametrize("page,lens", [(0, None), (16, [256, 40, 200])])
def test_prompt_weigh_evict_decode(page, lens):
    """A serving loop: a chunk of the prompt, its last queries' weights, the eviction, decode steps
    that add their own weights, a second eviction in place, a windowed step."""
    B, H, G, L, n, keep = 3, 2, 4, 256, 48, 128
    c = Case(B, H, G, L, n, seed=60, page=page, lens=lens, spare=n + 8)
    if lens is None:
        c.cache.seq_len = None
    g = torch.Generator().manual_seed(61)
    kn, vn = (torch.randn(B, n, H, 128, generator=g).bfloat16() for _ in range(2))
    out = torch.empty(B, n, H * G, 128, device="cuda")
    view = R.View(causal=True, own_token=True)
    R.dense_prefill_chunk(c.p, c.cache, kn.cuda(), vn.cuda(), c.qd, out, c.ws, view)
    for b in range(B):
        m = c.lens[b]
        c.k[b, :, m:m + n], c.v[b, :, m:m + n] = kn[b].transpose(0, 1), vn[b].transpose(0, 1)
    c.lens = [m + n for m in c.lens]
    check(out, c.want(causal=True, own=True), True, c.bound())
    w = torch.zeros(B, H, c.cap, device="cuda")
    R.accumulate_weights(c.p, c.cache, c.qd[:, -16:].contiguous(), w, c.ws, view)
    kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
    w0 = w.cpu().clone()
    R.evict(c.p, c.cache, w, keep, kept, into_weights=w, sinks=4, recent=32)
    k2, v2 = torch.zeros_like(c.k), torch.zeros_like(c.v)
    for b in range(B):
        for h in range(H):
            idx = F.evict(w0[b, h], c.lens[b], keep, 4, 32)
            assert kept[b, h].tolist()[:len(idx)] == idx
            k2[b, h, :len(idx)], v2[b, h, :len(idx)] = c.k[b, h, idx], c.v[b, h, idx]
    c.k, c.v, c.lens = k2, v2, [min(m, keep) for m in c.lens]
    for step in range(3):
        x = [torch.randn(B, 1, h, 128, generator=g).bfloat16() for h in (H, H, H * G)]
        o = torch.empty(B, 1, H * G, 128, device="cuda")
        sv = R.View(sinks=4, window=60) if step == 2 else R.View()
        if lens is not None:
            R.dense_decode_step(c.p, c.cache, *(t.cuda() for t in x), o, c.ws, sv)
            c.cache.length += 1
        else:
            sv.own_token = 1
            R.dense_prefill_chunk(c.p, c.cache, *(t.cuda() for t in x), o, c.ws, sv)
        for b in range(B):
            c.k[b, :, c.lens[b]], c.v[b, :, c.lens[b]] = x[0][b, 0], x[1][b, 0]
        c.lens = [m + 1 for m in c.lens]
        c.q = x[2]
        check(o, c.want(sinks=sv.sinks, window=sv.window), True, c.bound())
        if step < 2:
            R.accumulate_weights(c.p, c.cache, x[2].cuda(), w, c.ws)
    R.check_device_errors(c.ws)
    total = w.double().sum(-1).cpu()
    assert torch.isfinite(total).all()
