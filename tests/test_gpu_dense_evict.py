"""Eviction's order and sizes.  Selections are compared exactly (the weights are given)."""

import pytest
import torch

import dense_reference as F
import hierarchical_sparse_attention_build_b200 as R
from test_gpu_dense import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,keep", [(200, 60), (20000, 700)])
def test_zeros_of_either_sign_tie(L, keep):
    c = Case(1, 2, 1, L, 1, seed=1)
    g = torch.Generator().manual_seed(2)
    w = torch.where(torch.rand(1, 2, L, generator=g) < 0.5, 0.0, -0.0)
    w[:, :, 7::91] = 1.0
    w[:, :, 9::83] = -1.0
    kept = torch.empty(1, 2, keep, dtype=torch.int32, device="cuda")
    before = w.cuda()
    moved = before.clone()
    R.evict(c.p, c.cache, moved, keep, kept, into_weights=moved, sinks=3, recent=5)
    for h in range(2):
        idx = F.evict(w[0, h], L, keep, 3, 5)
        assert kept[0, h].tolist() == idx
        assert torch.equal(moved[0, h, :keep].view(torch.int32), before[0, h, idx].view(torch.int32))


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("L,keep,sinks,recent,page", [
    (70_001, 20_000, 4, 64, 0),       # a thread holds up to 32 keys
    (131_072, 131_071, 0, 0, 0),
    (131_073, 9, 3, 3, 0),            # keys read again each time
    (150_000, 100_000, 0, 1000, 256),
    (1_048_579, 4096, 4, 256, 0),
])
def test_long_caches(L, keep, sinks, recent, page, into):
    H = 2
    g = torch.Generator().manual_seed(L)
    p = R.params(num_kv_heads=H, num_q_heads=2 * H, branching=8, top_k=4)
    cap = -(-L // page) * page if page else L + 3
    rows = torch.arange(cap, dtype=torch.int32).view(1, 1, cap, 1).expand(1, H, cap, 64).contiguous()
    k = rows.cuda().view(torch.bfloat16).view(1, H, cap, 128)  # a slot's number in every word of its row
    v = k.flip(1).contiguous()
    if page:
        table = torch.randperm(cap // page, generator=g).to(torch.int32).view(1, -1).cuda()
        pool = [torch.empty(cap // page, H, page, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for x, y in zip(pool, (k, v)):
            x[table[0].long()] = y.view(H, cap // page, page, 128).transpose(0, 1)
        cache = R.TokenCache(p, *pool, L, page_table=table)
    else:
        cache = R.TokenCache(p, k.clone(), v.clone(), L)
    w = torch.empty(1, H, cap).exponential_(1.0, generator=g) ** 3
    w = (w * 64).round() / 64  # many ties
    kept = torch.empty(1, H, keep, dtype=torch.int32, device="cuda")
    moved = w.cuda()
    to = None
    if into:
        to = R.TokenCache(p, *(torch.empty(1, H, keep, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)), 0)
        tw = torch.empty(1, H, keep, device="cuda")
    R.evict(p, cache, moved, keep, kept, into=to, into_weights=tw if into else moved, sinks=sinks, recent=recent)
    ws = R.DenseWorkspace(p, 1, 64, "cuda")
    R.check_device_errors(ws)
    got = to or cache
    for h in range(H):
        idx = F.evict(w[0, h], L, keep, sinks, recent)
        assert kept[0, h].tolist() == idx
        at = torch.tensor(idx, device="cuda")
        assert torch.equal((tw if into else moved)[0, h, :keep].cpu(), w[0, h, idx])
        for x in (got.k_tok, got.v_tok):
            if got.page_table is not None:
                x = x[got.page_table[0].long(), h].reshape(-1, 128)
            else:
                x = x[0, h]
            assert torch.equal(x[:keep].contiguous().view(torch.int32), at.int()[:, None].expand(keep, 64))
        if not into:
            assert not moved[0, h, keep:L].any()
