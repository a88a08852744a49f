"""fp32 outputs of the dense cache operators to fp32's own accuracy.

Tolerances, in the norm, for scores of spread sigma: rotated rows are two fp16 parts (11 bits each;
what they leave and the product of the two second parts are 2^-22 of an operand each, of
independent sign over a score's terms) of values rotated in fp32 (an angle good to 2 pi 2^-26, two
rounded products and a rounded sum on either side): less than 2^-21 sigma rms on a score.  exp2 is good
to 2^-22, weights in three bf16 parts to 2^-26, and sums are joined in rounded fp32 adds: 2^-21
for all of them.  Together (1 + sigma) 2^-21.
"""

import pytest
import torch

import dense_reference as F
import hierarchical_sparse_attention_build_b200 as R
from test_gpu_dense import BASE, Case, params, split_view
from test_gpu_dense_scores import rel

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sigma", [0.1, 1.0, 5.0])
@pytest.mark.parametrize("B,H,G,L,n,page,lens,view", [
    (1, 2, 4, 4096, 16, 0, None, {}),
    (2, 2, 4, 3000, 1, 0, None, {}),
    (3, 2, 2, 900, 5, 32, [900, 1, 333], dict(causal=True, own=True)),
    (2, 1, 8, 700, 40, 0, None, dict(causal=True, own=True, sinks=3, window=200)),
    (5, 8, 4, 9000, 1, 16, [9000, 17, 0, 4000, 8999], {}),  # steps dealt out to the blocks
    (3, 8, 4, 9000, 3, 0, [300, 9000, 2], dict(causal=True)),
])
def test_outputs(B, H, G, L, n, page, lens, view, sigma):
    c = Case(B, H, G, L, n, seed=L + n, page=page, lens=lens, scale=sigma / 1.5)
    v, ref = split_view(view)
    assert rel(c.attend(True, v).double().cpu(), c.want(**ref)) <= (1 + sigma) * 2.0 ** -21


@pytest.mark.parametrize("sigma", [0.1, 1.0, 5.0])
@pytest.mark.parametrize("B,H,G,L,n,lens", [(2, 2, 4, 5000, 1, None), (2, 2, 1, 3000, 8, [3000, 77]), (1, 2, 8, 700, 1, None),
                                            (5, 8, 4, 9000, 2, [9000, 17, 0, 4000, 8999])])
def test_weights_of_few_rows(B, H, G, L, n, lens, sigma):
    c = Case(B, H, G, L, n, seed=L + n, lens=lens, scale=sigma / 1.5)
    w = torch.zeros(B, H, c.cap, device="cuda")
    R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, R.View(causal=n > 1, own_token=n > 1))
    R.check_device_errors(c.ws)
    want = c.want(want_weights=True, causal=n > 1, own=n > 1)
    assert rel(w.double().cpu(), want) <= (1 + sigma) * 2.0 ** -21


@pytest.mark.parametrize("kscale,qscale", [(2.0 ** 11, 2.0 ** -11), (2.0 ** 20, 2.0 ** -20), (2.0 ** -20, 2.0 ** 20),
                                           (2.0 ** 100, 2.0 ** -100), (2.0 ** -100, 2.0 ** 100)])
@pytest.mark.parametrize("n", [1, 5])
def test_rows_beyond_the_parts_range(kscale, qscale, n):
    """Keys or queries whose parts fp16 does not hold: such rows are computed in fp32 (or lie so far
    below that range that a product with the other side's would be as if they were beyond it)."""
    c = Case(2, 2, 4, 700, n, seed=91, page=16, lens=[700, 90])
    c.k = (c.k.float() * kscale).bfloat16()
    c.q = (c.q.float() * qscale).bfloat16()
    pool = c.cache.k_tok
    pool.copy_((pool.float() * kscale).bfloat16())
    c.qd = c.q.cuda()
    view, ref = R.View(causal=True, own_token=True), dict(causal=True, own=True)
    assert rel(c.attend(True, view).double().cpu(), c.want(**ref)) <= 4 * 2.0 ** -21
    w = torch.full((2, 2, c.cap), 3.0, device="cuda")
    if n == 1:
        R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, view, accumulate=False)
        R.check_device_errors(c.ws)
        want = c.want(want_weights=True, **ref)
        for b, m in enumerate(c.lens):
            assert rel(w[b, :, :m].double().cpu(), want[b, :, :m]) <= 4 * 2.0 ** -21


def test_one_key_beyond_the_parts_range():
    """A single key beyond fp16 among ordinary ones, seen by some rows only, with a score like theirs."""
    c = Case(1, 1, 4, 300, 2, seed=92)
    c.k[0, 0, 299] = 0
    c.k[0, 0, 299, 63] = 2.0 ** 17
    c.q[..., 63] = 2.0 ** -14
    c.cache.k_tok.copy_(c.k)
    c.qd = c.q.cuda()
    view, ref = R.View(causal=True, own_token=True), dict(causal=True, own=True)
    assert rel(c.attend(True, view).double().cpu(), c.want(**ref)) <= 4 * 2.0 ** -21
    w = torch.zeros(1, 1, c.cap, device="cuda")
    R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, view)
    assert rel(w.double().cpu(), c.want(want_weights=True, **ref)) <= 4 * 2.0 ** -21


@pytest.mark.parametrize("sigma", [0.1, 1.0, 5.0])
@pytest.mark.parametrize("B,H,G,L,n,page,lens", [(1, 2, 4, 4000, 3, 0, None), (2, 1, 8, 900, 40, 16, [900, 100]),
                                                 (1, 1, 1, 3000, 200, 0, None), (3, 2, 2, 200, 9, 0, [200, 0, 5])])
def test_weights_of_many_rows(B, H, G, L, n, page, lens, sigma):
    c = Case(B, H, G, L, n, seed=L + n, page=page, lens=lens, scale=sigma / 1.5)
    for own in (True, False):
        w = torch.zeros(B, H, c.cap, device="cuda")
        R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, R.View(causal=True, own_token=own))
        R.check_device_errors(c.ws)
        want = c.want(want_weights=True, causal=True, own=own)
        assert rel(w.double().cpu(), want) <= (1 + sigma) * 2.0 ** -21


def test_weights_of_a_head_beyond_the_parts_range():
    """One head's keys exceed fp16, another's queries do: those come from two bf16 parts (2^-16 each
    of scores of spread 2: 3 * 2^-16), the others keep theirs, in this call and the next."""
    H, G, L, n = 4, 4, 700, 12
    c = Case(1, H, G, L, n, seed=93)
    c.k[:, 1] = (c.k[:, 1].float() * 2.0 ** 20).bfloat16()
    c.q[:, :, G:2 * G] = (c.q[:, :, G:2 * G].float() * 2.0 ** -20).bfloat16()
    c.k[:, 3] = (c.k[:, 3].float() * 2.0 ** -20).bfloat16()
    c.q[:, :, 3 * G:] = (c.q[:, :, 3 * G:].float() * 2.0 ** 20).bfloat16()
    c.cache.k_tok.copy_(c.k)
    view = R.View(causal=True, own_token=True)
    plain = Case(1, H, G, L, n, seed=93)
    want = plain.want(want_weights=True, causal=True, own=True)  # powers of two cancel
    for case, wide in ((c, (1, 3)), (plain, ()), (c, (1, 3))):
        w = torch.zeros(1, H, c.cap, device="cuda")
        R.accumulate_weights(c.p, case.cache, case.q.cuda(), w, c.ws, view)
        R.check_device_errors(c.ws)
        for h in range(H):
            assert rel(w[0, h].double().cpu(), want[0, h]) <= (3 * 2.0 ** -16 if h in wide else 3 * 2.0 ** -21)


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 3.0e38])
@pytest.mark.parametrize("n", [2, 40])
def test_weights_beside_a_key_that_some_queries_do_not_see(bad, n):
    """A key beyond every range among the chunk's tokens: the queries before it weigh as without it."""
    c = Case(1, 1, 4, 500, n, seed=94)
    hit = 500 - n // 2
    c.cache.k_tok[0, :, hit] = bad
    view = R.View(causal=True)
    few = n - n // 2  # the first queries alone: none sees the key (own tokens hidden)
    q = c.q[:, :few].cuda().contiguous()
    c.cache.length = 500 - n // 2
    w = torch.zeros(1, 1, c.cap, device="cuda")
    R.accumulate_weights(c.p, c.cache, q, w, c.ws, view)
    c.lens, c.q = [500 - n // 2], c.q[:, :few]
    want = c.want(causal=True, want_weights=True)
    assert rel(w.double().cpu(), want) <= 3 * 2.0 ** -21
    # the same queries and one that sees every token but its own: only hidden from the rest, finite
    c.cache.length = hit + 1
    w = torch.zeros(1, 1, c.cap, device="cuda")
    R.accumulate_weights(c.p, c.cache, torch.cat([q, q[:, :1]], 1), w, c.ws, view)
    R.check_device_errors(c.ws)
    assert torch.isfinite(w).all() and (w[0, 0, hit] == 0)
