"""The dense cache operators over long caches.  Tolerances are test_gpu_dense.py's."""

import pytest
import torch

import dense_reference as F
import hierarchical_sparse_attention_build_b200 as R
from test_gpu_dense import BASE, params
from test_gpu_paged import paginate

pytestmark = pytest.mark.gpu


def normal(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


@pytest.mark.parametrize("L,lens,n,page,causal", [
    (700_000, None, 3, 0, True),           # just past what the workspace's images hold at once
    (1_000_003, [1_000_003, 655_361, 9], 3, 0, True),
    (1_310_720, None, 40, 256, True),      # two tiles of query rows, keys in three slices
    (655_361, None, 5, 0, False),
])
def test_weights_of_many_rows_over_long_caches(L, lens, n, page, causal):
    """More than 8 query rows a KV group, and a head whose rotated keys do not fit the workspace."""
    H, G = 1, 4
    B = len(lens) if lens else 1
    p = params(H, G)
    cap = -(-L // page) * page if page else L
    k = normal(B, H, cap, 128, seed=L)
    q = normal(B, n, H * G, 128, seed=n)
    seq = torch.tensor(lens, device="cuda") if lens else None
    if page:
        kp, vp, table = paginate(k, k[:, :, :1].expand_as(k), page, seed=2)
        cache = R.TokenCache(p, kp, vp, L, seq_len=seq, page_table=table)
    else:
        cache = R.TokenCache(p, k, k, L, seq_len=seq)
    ws = R.DenseWorkspace(p, B, cap, "cuda")
    view = R.View(causal=causal, own_token=causal)
    w = torch.full((B, H, cap), 3.0, device="cuda")
    R.accumulate_weights(p, cache, q, w, ws, view, accumulate=False)
    R.check_device_errors(ws)
    want = torch.zeros(B, H, cap, dtype=torch.float64, device="cuda")
    for b in range(B):
        m = lens[b] if lens else L
        kr = F.rotate(k[b, 0, :m].double(), torch.arange(m, device="cuda"), BASE)
        for i, at in enumerate(F.positions(m, n, causal, causal)):
            if at > 0:
                s = 128 ** -0.5 * F.rotate(q[b, i].double(), at, BASE) @ kr[:at].T
                want[b, 0, :at] += torch.softmax(s, -1).sum(0)
        got = w[b, 0, :m].double()
        assert float((got - want[b, 0, :m]).norm() / want[b, 0, :m].norm()) <= 2.0 ** -16
        assert (w[b, :, m:] == 3.0).all()
    again = w.clone()
    R.accumulate_weights(p, cache, q, again, ws, view)
    for b in range(B):
        m = lens[b] if lens else L
        assert torch.equal(again[b, :, :m], w[b, :, :m] + w[b, :, :m]) and (again[b, :, m:] == 3.0).all()


def test_a_larger_workspace_buffer_is_used():
    p, L = params(1, 4), 300_000
    need = R.dense_workspace_size(p, 1, L)
    buf = torch.empty(need + (256 << 20), dtype=torch.uint8, device="cuda")
    ws = R.DenseWorkspace(p, 1, L, "cuda", buffer=buf)
    assert ws.nbytes == buf.numel()
    k, q = normal(1, 1, L, 128, seed=1), normal(1, 4, 4, 128, seed=2)
    cache = R.TokenCache(p, k, k, L)
    got = []
    for each in (ws, R.DenseWorkspace(p, 1, L, "cuda")):
        w = torch.zeros(1, 1, L, device="cuda")
        R.accumulate_weights(p, cache, q, w, each)
        R.check_device_errors(each)
        got.append(w)
    assert torch.equal(*got)
