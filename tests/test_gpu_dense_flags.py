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
