"""The dense cache operators' accuracy on sharp scores, and launches of many items.

Tolerances.  test_gpu_dense.py's bounds, and for scores of spread sigma (standard normal rows, q
scaled by sigma / 1.5: the keys' heads have magnitudes up to 2) their norms: a rounding of relative
size r is off by r / sqrt 3 rms, so with errors of independent sign over a score's terms
 * two parts: three errors of 2^-16 / sqrt 3 move a score by at most 2^-16 sigma rms and an output by
   as much of its norm, the probabilities' parts by 2^-16: (1 + sigma) 2^-16;
 * chunk kernel: two fp16 roundings, 2^-11 sqrt(2/3) sigma; a bf16 one of each weight and of the
   output, 2^-8 / sqrt 3 of a power of two each (1.7e-3 of the norm): the root of their squares, and a quarter.
"""

import math

import pytest
import torch

import dense_reference as F
import hierarchical_sparse_attention_build_b200 as R
from test_gpu_dense import BASE, Case, check, params, split_view

pytestmark = pytest.mark.gpu


def rel(got, want):
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("sigma", [1.0, 5.0, 20.0])
@pytest.mark.parametrize("L,n,view", [(3000, 1, {}), (900, 4, dict(causal=True, own=True)),
                                      (700, 150, dict(causal=True, own=True)),
                                      (700, 150, dict(causal=True, own=True, sinks=4, window=100))])
def test_sharp_scores(L, n, view, sigma):
    c = Case(1, 2, 4, L, n, seed=L + n, scale=sigma / 1.5)
    v, ref = split_view(view)
    want = c.want(**ref)
    bf16 = 2.0 ** -8 / math.sqrt(3.0)
    for fp32, kernel in ((True, R.DENSE_ROWS), (False, R.DENSE_ROWS), (False, R.DENSE_CHUNK)):
        v.kernel = kernel
        got = c.attend(fp32, v).double().cpu()
        rows = (got - want).norm(dim=-1) / want.norm(dim=-1)
        print(f"sigma {sigma} n {n} window {v.window} fp32 {fp32} kernel {kernel}: norm {rel(got, want):.2e} "
              f"worst row {float(rows.max()):.2e}")
        if kernel == R.DENSE_CHUNK:
            assert rel(got, want) <= 1.25 * math.hypot(bf16, bf16, 2.0 ** -11 * math.sqrt(2.0 / 3.0) * sigma)
        elif fp32:
            assert float((got - want).abs().max()) <= c.bound()
            assert rel(got, want) <= (1 + sigma) * 2.0 ** -16
        else:
            assert rel(got, want) <= 1.25 * math.hypot(bf16, (1 + sigma) * 2.0 ** -16)
    if not view.get("window"):
        w = torch.zeros(1, 2, c.cap, device="cuda")
        R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, v)
        assert rel(w.double().cpu(), c.want(want_weights=True, **ref)) <= (1 + sigma) * 2.0 ** -16


def test_queries_beyond_half_precision():
    """Rotated, scaled queries larger than fp16 holds (and keys below its range): the chunk kernel
    hands the tile to the rows kernel."""
    c = Case(1, 2, 4, 500, 64, seed=70)
    scale = 2.0 ** -17
    c.p = params(2, 4, softmax_scale=scale)
    c.q = (c.q.float() * 2.0 ** 34).bfloat16()
    c.k = (c.k.float() * 2.0 ** -20).bfloat16()
    assert float(c.q.abs().max()) * scale * math.log2(math.e) > 4 * 65504
    c.qd = c.q.cuda()
    c.cache.k_tok.copy_(c.k)
    got = c.attend(False, R.View(causal=True, own_token=True, kernel=R.DENSE_CHUNK))
    check(got, c.want(causal=True, own=True, scale=scale), False, 0.0)


def causal_rows(q, k, v, L):
    """Queries q [n][G][128] of the last n tokens over k, v [L][128], own tokens seen (64 bits)."""
    n = q.shape[0]
    p = torch.arange(L - n + 1, L + 1, device=q.device)
    s = 128 ** -0.5 * F.rotate(q.double(), p[:, None], BASE) @ F.rotate(k.double(), torch.arange(L, device=q.device), BASE).T
    seen = torch.arange(L, device=q.device) < p[:, None]
    w = torch.softmax(torch.where(seen[:, None], s, -math.inf), -1)
    return w @ v.double()


@pytest.mark.parametrize("kernel", [R.DENSE_CHUNK, R.DENSE_ROWS])
def test_more_items_than_the_workspace_lists(kernel):
    """Above 4096 work items: none is shared among blocks, and two items share a mark.  A value that
    only the last query of the last head sees is infinite, so that its tile is marked."""
    B, H, G, L, n = 64, 8, 8, 300, 300
    p = params(H, G)
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.empty(B, H, L, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    q = torch.empty(B, n, H * G, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    v[B - 1, H - 1, L - 1] = math.inf
    cache, ws, out = R.TokenCache(p, k, v, L), R.DenseWorkspace(p, B, L, "cuda"), torch.empty_like(q)
    for _ in range(2):  # a second call finds the marks cleared
        out.fill_(7.0)
        R.dense_attend(p, cache, q, out, ws, R.View(causal=True, own_token=True, kernel=kernel))
        R.check_device_errors(ws)
        for b, h in ((0, 0), (13, 1), (12, 6), (40, 5), (B - 1, H - 2), (B - 1, H - 1)):
            rows = slice(h * G, (h + 1) * G)
            got, m = out[b, :, rows].double(), n
            if (b, h) == (B - 1, H - 1):
                assert torch.isposinf(got[n - 1]).all()
                m = n - 1
            want = causal_rows(q[b, :m, rows], k[b, h, :L - n + m], v[b, h, :L - n + m], L - n + m)
            assert torch.isfinite(got[:m]).all() and rel(got[:m], want) <= 2.0 ** -7
        assert torch.isfinite(out[:B - 1]).all()


@pytest.mark.parametrize("kernel,fp32,n", [(R.DENSE_ROWS, True, 40), (R.DENSE_ROWS, False, 1), (R.DENSE_CHUNK, False, 40)])
def test_attention_skips_a_missing_page(kernel, fp32, n):
    L, page = 500, 16
    c = Case(2, 2, 4, L, n, seed=71, page=page, garbage=0.0)
    c.table[1, 9] = -1
    view = R.View(causal=True, own_token=True, kernel=kernel)
    out = torch.full(c.q.shape, 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    R.dense_attend(c.p, c.cache, c.qd, out, c.ws, view)
    with pytest.raises(R.RecsaError) as e:
        R.check_device_errors(c.ws)
    assert e.value.code == 6
    check(out, masked(c, 1, 144, 160)[0], fp32, c.bound())


def masked(c, bad, t0, t1):
    """Outputs and weights of causal queries (own tokens seen) with tokens [t0, t1) of sequence `bad` missing."""
    out = torch.zeros(c.q.shape, dtype=torch.float64)
    got = torch.zeros(c.B, c.H, c.cap, dtype=torch.float64)
    for b in range(c.B):
        L = c.lens[b]
        for i, p in enumerate(F.positions(L, c.n, True, True)):
            for h in range(c.H):
                rows = slice(h * c.G, (h + 1) * c.G)
                w = F.weights_of(c.q[b, i, rows].double(), c.k[b, h, :L].double(), p, BASE, 128 ** -0.5)
                if b == bad:
                    w[:, t0:t1] = 0
                    w = w / w.sum(-1, keepdim=True)
                out[b, i, rows] = w @ c.v[b, h, :L].double()
                got[b, h, :L] += w.sum(0)
    return out, got


@pytest.mark.parametrize("n", [2, 40])
def test_weights_of_a_missing_page_are_zero(n):
    """Both kernels: at most 8 query rows a KV group, and more."""
    L, page = 500, 16
    c = Case(2, 2, 4, L, n, seed=72, page=page, garbage=0.0)
    c.table[0, 3] = 10_000
    w = torch.full((2, 2, c.cap), 3.0, device="cuda")
    R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, R.View(causal=True, own_token=True), accumulate=False)
    with pytest.raises(R.RecsaError) as e:
        R.check_device_errors(c.ws)
    assert e.value.code == 6
    got, want = w[:, :, :L].double().cpu(), masked(c, 0, 48, 64)[1][:, :, :L]
    assert not got[0, :, 48:64].any() and (w[:, :, L:] == 3.0).all()
    assert rel(got, want) <= 2.0 ** -16


def test_attention_over_clamped_lengths():
    c = Case(2, 2, 4, 60, 1, seed=73, lens=[60, 20], garbage=0.0)
    c.cache.seq_len.copy_(torch.tensor([999, -5]))
    for fp32, kernel in ((True, R.DENSE_ROWS), (False, R.DENSE_CHUNK)):
        out = torch.full(c.q.shape, 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        R.dense_attend(c.p, c.cache, c.qd, out, c.ws, R.View(kernel=kernel))
        with pytest.raises(R.RecsaError) as e:
            R.check_device_errors(c.ws)
        assert e.value.code == 6
        c.lens = [60, 0]
        check(out, c.want(), fp32, c.bound())
