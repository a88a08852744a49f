"""Lengths and page-table entries out of range: what the calls still do, and that they say so.

The bad values are ones that the kernels' own checks turn into an error (nothing out of range is
dereferenced); tolerances are test_gpu_dense.py's.
"""

import pytest
import torch

import dense_reference as F
import hierarchical_sparse_attention_build_b200 as R
from test_gpu_dense import Case, check
from test_gpu_paged import paginate

pytestmark = pytest.mark.gpu


def flagged(ws):
    """The error word is set, and reading it cleared it."""
    with pytest.raises(R.RecsaError) as e:
        R.check_device_errors(ws)
    assert e.value.code == 6
    R.check_device_errors(ws)


def receiver(c, cap, page=0):
    rows = [torch.full((c.B, c.H, cap, 128), 5.0, dtype=torch.bfloat16) for _ in range(2)]
    seq = torch.zeros(c.B, dtype=torch.int64, device="cuda")
    if not page:
        return R.TokenCache(c.p, rows[0].cuda(), rows[1].cuda(), 0, seq_len=seq), None
    kp, vp, table = paginate(*rows, page, seed=1)
    return R.TokenCache(c.p, kp, vp, 0, seq_len=seq, page_table=table), table


def contents(cache, table, page):
    return [F.tokens(x.cpu(), table, page) if page else x.cpu().clone() for x in (cache.k_tok, cache.v_tok)]


@pytest.mark.parametrize("into", [False, True])
def test_evict_flags_lengths_out_of_range(into):
    B, H, L, keep = 3, 2, 60, 20
    c = Case(B, H, 2, L, 1, seed=1, lens=[60, 20, 41], garbage=0.0)
    c.cache.seq_len.copy_(torch.tensor([999, -5, 41]))
    w = torch.rand(B, H, c.cap, generator=torch.Generator().manual_seed(2)).cuda()
    w0 = w.cpu().clone()
    kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
    to = receiver(c, 32)[0] if into else None
    R.evict(c.p, c.cache, w, keep, kept, into=to, sinks=2, recent=4)
    flagged(c.ws)
    got = (to or c.cache)
    assert got.seq_len.tolist() == [20, 0, 20]  # clamped to 60 and 0
    rows = contents(got, None, 0)
    for b, m in enumerate((60, 0, 41)):
        for h in range(H):
            idx = F.evict(w0[b, h], m, keep, 2, 4)
            assert kept[b, h].tolist() == idx + [-1] * (keep - len(idx))
            assert torch.equal(rows[0][b, h, :len(idx)], c.k[b, h, idx])
            assert torch.equal(rows[1][b, h, :len(idx)], c.v[b, h, idx])


@pytest.mark.parametrize("into", [False, True])
def test_evict_from_a_missing_page(into):
    """Rows of a page outside the pool arrive as zeros, not as what the slot held before."""
    B, H, L, keep, page = 2, 2, 160, 60, 16
    c = Case(B, H, 2, L, 1, seed=3, page=page, lens=[160, 130])
    table = c.table.clone()
    w = torch.rand(B, H, c.cap, generator=torch.Generator().manual_seed(4)).cuda()
    w[:, :, 96:112] = 2.0  # the slots of the missing page are kept
    kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
    c.cache.page_table[0, 6] = 10_000
    w0 = w.cpu().clone()
    to = receiver(c, 64)[0] if into else None
    R.evict(c.p, c.cache, w, keep, kept, into=to, sinks=2, recent=4)
    flagged(c.ws)
    rows = contents(to, None, 0) if into else contents(c.cache, table, page)
    for b in range(B):
        for h in range(H):
            idx = F.evict(w0[b, h], c.lens[b], keep, 2, 4)
            assert kept[b, h].tolist() == idx and set(range(96, 112)) <= set(idx)
            for x, y in zip(rows, (c.k, c.v)):
                want = y[b, h, idx].clone()
                if b == 0:
                    want[[96 <= i < 112 for i in idx]] = 0
                assert torch.equal(x[b, h, :keep], want)


def test_evict_to_a_missing_page():
    """Rows that would go to a page outside the pool are not written; the others are."""
    B, H, L, keep, page = 2, 1, 200, 60, 16
    c = Case(B, H, 2, L, 1, seed=5)
    w = torch.rand(B, H, c.cap, generator=torch.Generator().manual_seed(6)).cuda()
    kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
    to, table = receiver(c, 64, page)
    table = table.clone()
    to.page_table[1, 2] = -3
    R.evict(c.p, c.cache, w, keep, kept, into=to)
    flagged(c.ws)
    rows = contents(to, table, page)
    for b in range(B):
        idx = F.evict(w[b, 0].cpu(), L, keep, 0, 0)
        for x, y in zip(rows, (c.k, c.v)):
            want = y[b, 0, idx].clone()
            if b == 1:
                want[32:48] = 5.0
            assert torch.equal(x[b, 0, :keep], want)


def test_a_clean_eviction_flags_nothing():
    c = Case(2, 2, 2, 100, 1, seed=7, page=16, lens=[100, 0])
    kept = torch.empty(2, 2, 30, dtype=torch.int32, device="cuda")
    R.evict(c.p, c.cache, torch.rand(2, 2, c.cap, device="cuda"), 30, kept)
    R.check_device_errors(c.ws)


@pytest.mark.parametrize("with_tree", [False, True])
@pytest.mark.parametrize("bad", [55, -4, 999])
def test_prefill_flags_lengths_out_of_range(with_tree, bad):
    """A length the cache's bound excludes - one that the advanced bound would admit, too - gets no
    tokens and is flagged, with a tree over the cache and without."""
    B, H, G, L, n = 2, 1, 4, 50, 12
    c = Case(B, H, G, L, n, seed=11, lens=[50, 33], spare=20, garbage=0.0)
    cache = c.cache
    if with_tree:
        cache = R.RecsaTree(c.p, c.cache.k_tok, c.cache.v_tok, torch.eye(128).cuda(), L, seq_len=c.cache.seq_len)
        R.build_tree(c.p, cache)
    cache.seq_len[0] = bad
    before = cache.k_tok.clone()
    new = [torch.randn(B, n, h, 128).bfloat16().cuda() for h in (H, H)]
    out = torch.empty(B, n, H * G, 128, device="cuda")
    R.dense_prefill_chunk(c.p, cache, *new, c.qd, out, c.ws, R.View(causal=True, own_token=True))
    flagged(c.ws)
    assert cache.seq_len.tolist() == [bad, 33 + n] and cache.length == L + n
    assert torch.equal(cache.k_tok[0], before[0])
    c.k[1, :, 33:45], c.v[1, :, 33:45] = (x[1].transpose(0, 1).cpu() for x in new)
    c.lens = [62, 45]
    check(out[1:], c.want(causal=True, own=True)[1:], True, c.bound())


@pytest.mark.parametrize("with_tree,uneven,n", [(False, False, 3), (True, False, 3), (True, False, 100), (True, True, 3)])
def test_prefill_flags_a_missing_page_that_no_query_reads(with_tree, uneven, n):
    """The chunk's last token alone lies on the missing page, and without its own token no query
    sees it: the append flags it."""
    page, L = 16, 160 - n + 1
    c = Case(1, 1, 4, L, n, seed=12, page=page, lens=[L] if uneven else None, spare=n + 8, garbage=0.0)
    cache = c.cache
    if with_tree:
        cache = R.RecsaTree(c.p, c.cache.k_tok, c.cache.v_tok, torch.eye(128).cuda(), L, seq_len=c.cache.seq_len,
                            page_table=c.table)
        R.build_tree(c.p, cache)
    R.check_device_errors(c.ws)
    c.table[0, 10] = 10_000
    new = [torch.randn(1, n, 1, 128).bfloat16().cuda() for _ in range(2)]
    out = torch.empty(1, n, 4, 128, device="cuda")
    R.dense_prefill_chunk(c.p, cache, *new, c.qd, out, c.ws)
    flagged(c.ws)
    c.k[0, 0, L:L + n], c.v[0, 0, L:L + n] = new[0][0, :, 0].cpu(), new[1][0, :, 0].cpu()
    c.lens = [L + n]
    check(out, c.want(causal=True), True, c.bound())


def test_neighbouring_buffers_are_accepted():
    """Queries and output, weights and kept slots side by side in one allocation; two page pools
    interleaved page by page, whose ranges overlap and whose rows do not."""
    B, H, G, L, keep, page = 1, 2, 2, 64, 20, 16
    c = Case(B, H, G, L, 1, seed=13)
    want = c.attend(False)
    both = torch.empty(2, *c.qd.shape, dtype=torch.bfloat16, device="cuda")
    both[0] = c.qd
    R.dense_attend(c.p, c.cache, both[0], both[1], c.ws)
    assert torch.equal(both[1], want)
    w = torch.rand(3, B, H, L, device="cuda")
    kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
    w0 = w[0].cpu()
    R.evict(c.p, c.cache, w[0], keep, kept, into_weights=w[1])
    for h in range(H):
        idx = F.evict(w0[0, h], L, keep, 0, 0)
        assert kept[0, h].tolist() == idx and torch.equal(w[1, 0, h, :keep].cpu(), w0[0, h, idx])
    # pages 0, 2, 4, ... of one pool hold K, the others V
    pool = torch.zeros(10, H, page, 128, dtype=torch.bfloat16, device="cuda")
    k, v = pool[:9], pool[1:]
    table = torch.tensor([[0, 4, 2, 6]], dtype=torch.int32, device="cuda")
    d = Case(B, H, G, L, 1, seed=14)
    for i, pg in enumerate(table[0].tolist()):
        k[pg], v[pg] = (x[0, :, i * page:(i + 1) * page].cuda() for x in (d.k, d.v))
    cache = R.TokenCache(d.p, k, v, L, page_table=table)
    out = torch.empty(B, 1, H * G, 128, device="cuda")
    R.dense_attend(d.p, cache, d.qd, out, d.ws)
    check(out, d.want(), True, d.bound())
    R.evict(d.p, cache, w[2], keep, kept)
    R.check_device_errors(d.ws)
    for h in range(H):
        idx = F.evict(w[2, 0, h].cpu(), L, keep, 0, 0)
        got = torch.cat([k[pg, h] for pg in (0, 4)])[:keep].cpu(), torch.cat([v[pg, h] for pg in (0, 4)])[:keep].cpu()
        assert torch.equal(got[0], d.k[0, h, idx]) and torch.equal(got[1], d.v[0, h, idx])
