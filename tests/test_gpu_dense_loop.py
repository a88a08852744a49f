"""Serving loops over a bounded cache: append, attend, weigh, evict, again and again, with the
rows and the weights of every slot carried along in 64 bits beside the library's.

Tolerances.  Outputs as in test_gpu_dense.py.  A call's weights are off by at most 2^-16 of their
norm; after k calls the errors' norms add up to at most 2^-16 sqrt(k) of the sum's norm, since the
weights are not negative (|a + b|^2 >= |a|^2 + |b|^2); the fp32 adds put 2^-24 a call on top.
"""

import math

import pytest
import torch

import dense_reference as F
import hierarchical_sparse_attention_build_b200 as R
from test_gpu_dense import Case, check, params
from test_gpu_dense_layers import layer
from test_gpu_paged import paginate

pytestmark = pytest.mark.gpu

VIEW = R.View(causal=True, at_token=True)


class Loop:
    """A Case whose rows, lengths and weights (`want`, 64 bits) follow the calls."""

    def __init__(self, B, H, G, cap, page, uneven, seed):
        self.c = c = Case(B, H, G, 1, 1, seed=seed, page=page, lens=[0] * B if uneven else None, spare=cap - 1)
        c.cache.length, c.lens = 0, [0] * B
        self.gen = torch.Generator().manual_seed(seed)
        self.w = torch.zeros(B, H, c.cap, device="cuda")
        self.want = torch.zeros(B, H, c.cap, dtype=torch.float64)
        self.calls = 0

    def append(self, n):
        """n tokens on the cache and their queries' outputs compared; the queries are returned."""
        c = self.c
        k, v = (torch.randn(c.B, n, c.H, 128, generator=self.gen).bfloat16() for _ in range(2))
        q = torch.randn(c.B, n, c.H * c.G, 128, generator=self.gen).bfloat16()
        out = torch.empty(q.shape, device="cuda")
        R.dense_prefill_chunk(c.p, c.cache, k.cuda(), v.cuda(), q.cuda(), out, c.ws, VIEW)
        for b, m in enumerate(c.lens):
            c.k[b, :, m:m + n], c.v[b, :, m:m + n] = k[b].transpose(0, 1), v[b].transpose(0, 1)
        first, c.lens, c.q = list(c.lens), [m + n for m in c.lens], q
        check(out, layer(c, q, first), True, c.bound())
        return q

    def weigh(self, q):
        c, n = self.c, q.shape[1]
        R.accumulate_weights(c.p, c.cache, q.cuda(), self.w, c.ws, VIEW)
        self.want += layer(c, q, [m - n for m in c.lens], weights=True)
        self.calls += 1
        self.compare()

    def compare(self):
        got = self.w.double().cpu()
        assert float((got - self.want).norm() / self.want.norm()) <= math.sqrt(self.calls) * (2.0 ** -16 + 2.0 ** -24)
        for b, m in enumerate(self.c.lens):
            assert (got[b, :, m:] == 0).all()  # no weight where there is no token

    def evict(self, keep, sinks, recent, into=None, into_weights=None):
        c = self.c
        kept = torch.empty(c.B, c.H, keep, dtype=torch.int32, device="cuda")
        w0 = self.w.cpu()
        tw = self.w if into is None else into_weights
        R.evict(c.p, c.cache, self.w, keep, kept, into=into, into_weights=tw, sinks=sinks, recent=recent)
        R.check_device_errors(c.ws)
        k, v, want = torch.zeros_like(c.k), torch.zeros_like(c.v), torch.zeros_like(self.want)
        for b in range(c.B):
            for h in range(c.H):
                idx = F.evict(w0[b, h], c.lens[b], keep, sinks, recent)
                m = len(idx)
                assert kept[b, h].tolist() == idx + [-1] * (keep - m)
                k[b, h, :m], v[b, h, :m], want[b, h, :m] = c.k[b, h, idx], c.v[b, h, idx], self.want[b, h, idx]
        c.k, c.v, self.want = k, v, want
        c.lens = [min(m, keep) for m in c.lens]
        self.w = tw
        if into is not None:
            c.cache = into
        self.compare()


@pytest.mark.parametrize("page,uneven", [(0, False), (16, True)])
def test_weights_follow_their_tokens_in_place(page, uneven):
    """Prompt, weights, eviction, tokens over the slots given up, weights, a second eviction."""
    s = Loop(2, 2, 4, 200, page, uneven, seed=7)
    if uneven:  # one sequence is far shorter: the first eviction leaves it whole
        s.append(20)
        s.c.cache.seq_len[1] = 0
        s.c.lens[1] = 0
    s.weigh(s.append(100)[:, -16:].contiguous())
    s.evict(110 if uneven else 60, 4, 16)
    for _ in range(3):
        for _ in range(20):
            q = s.append(1)
        s.weigh(q)
    s.evict(60, 4, 8)
    s.weigh(s.append(2))


def test_weights_follow_their_tokens_between_two_caches():
    """Two caches and two weight buffers used in turn, the receiving buffer cleared before each call."""
    s = Loop(2, 2, 4, 200, 0, True, seed=8)
    c = s.c
    kp, vp, table = paginate(torch.zeros_like(c.k[:, :, :160]), torch.zeros_like(c.v[:, :, :160]), 32, seed=9)
    other = R.TokenCache(c.p, kp, vp, 0, seq_len=torch.zeros(2, dtype=torch.int64, device="cuda"), page_table=table)
    spare = torch.zeros(2, 2, 160, device="cuda")
    s.weigh(s.append(150)[:, -9:].contiguous())
    full_k, full_w, first = c.cap, s.w, c.cache
    for to, tw, cap in ((other, spare, 160), (first, full_w, full_k)):
        tw.zero_()
        if cap < c.k.shape[2]:
            c.k, c.v, s.want = c.k[:, :, :cap].contiguous(), c.v[:, :, :cap].contiguous(), s.want
            pad = 0
        else:
            pad = cap - c.k.shape[2]
        s.want = s.want[:, :, :cap].contiguous() if not pad else torch.nn.functional.pad(s.want, (0, pad))
        if pad:
            c.k, c.v = (torch.nn.functional.pad(x, (0, 0, 0, pad)) for x in (c.k, c.v))
        s.evict(70, 4, 10, into=to, into_weights=tw)
        c.cap = cap
        s.weigh(s.append(60)[:, -2:].contiguous())


def test_a_bounded_decode_step_in_one_graph():
    """Append, attend, weigh and evict in place, captured once: replays give the eager steps' bits,
    for sequences that reach the bound at different steps."""
    B, H, G, keep, steps = 3, 2, 4, 40, 12
    g = torch.Generator().manual_seed(12)
    new = [[torch.randn(B, 1, h, 128, generator=g).bfloat16() for h in (H, H, H * G)] for _ in range(steps)]
    results = []
    for graph in (False, True):
        c = Case(B, H, G, 64, 1, seed=11, page=16, lens=[38, 3, 40], garbage=0.0)
        c.cache.length = 64  # the bound of every step
        w = torch.zeros(B, H, c.cap, device="cuda")
        kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
        bufs = [x.cuda() for x in new[0]]
        out = torch.empty(B, 1, H * G, 128, device="cuda")

        def step():
            c.cache.length = 64
            R.dense_decode_step(c.p, c.cache, *bufs, out, c.ws, VIEW)
            R.accumulate_weights(c.p, c.cache, bufs[2], w, c.ws, VIEW)
            R.evict(c.p, c.cache, w, keep, kept, into_weights=w, sinks=2, recent=8)

        if graph:
            state = (c.cache.seq_len, c.cache.k_tok, c.cache.v_tok, w)
            before = [x.clone() for x in state]
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step()
            torch.cuda.current_stream().wait_stream(s)
            for x, y in zip(state, before):
                x.copy_(y)
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg):
                step()
        seen = []
        for x in new:
            for dst, src in zip(bufs, x):
                dst.copy_(src)
            cg.replay() if graph else step()
            seen.append([t.clone() for t in (out, kept, w, c.cache.seq_len)])
        R.check_device_errors(c.ws)
        assert c.cache.seq_len.tolist() == [40, 15, 40] and c.cache.length == keep
        results.append(seen + [[c.cache.k_tok, c.cache.v_tok]])
    for a, b in zip(*results):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_large_batch_of_uneven_sequences():
    """More sequences than have their steps dealt out to the blocks, and one fewer."""
    for B in (257, 256):
        H, G, L = 1, 4, 2000
        lens = [(37 * b) % (L + 1) for b in range(B)]
        lens[5] = L
        p = params(H, G)
        gen = torch.Generator(device="cuda").manual_seed(B)
        k, v = (torch.empty(B, H, L, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
        q = torch.empty(B, 1, H * G, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        cache, ws = R.TokenCache(p, k, v, L, seq_len=torch.tensor(lens, device="cuda")), R.DenseWorkspace(p, B, L, "cuda")
        out, w = torch.empty(q.shape, device="cuda"), torch.zeros(B, H, L, device="cuda")
        R.dense_attend(p, cache, q, out, ws)
        R.accumulate_weights(p, cache, q, w, ws)
        R.check_device_errors(ws)
        want = F.attend(q, k, v, lens, G)
        assert float((out.double() - want).norm() / want.norm()) <= 2.0 ** -16
        want = F.attend(q, k, v, lens, G, want_weights=True)
        assert float((w.double() - want).norm() / want.norm()) <= 2.0 ** -16
