"""The dense cache operators on values and scores at the edges of their types.

Tolerances.  test_gpu_dense.py's, and for rows whose scores are set exactly (`staircase`): queries
and keys lie in dimension 63 alone, which position t turns by t * base^(-126/128) < 5.1e-4 of a
radian over 400 tokens, so that products of at most 66 keep their value to 66 (1 - cos) < 1e-5 and
every operand its fp16 rounding (at most 2^-11 of the 5.1e-4 that lie in dimension 127): a weight
is off by less than 2^-14.  What is left is the roundings of weights and outputs: 2 * 2^-16 in the
rows kernel's parts, 2 * 2^-8 (bf16, half a step each) in the chunk kernel and of bf16 outputs.
"""

import math

import pytest
import torch

import hierarchical_sparse_attention_build_b200 as R
from test_gpu_dense import Case, check, params, split_view

pytestmark = pytest.mark.gpu

RUNS = [(True, R.DENSE_ROWS), (False, R.DENSE_ROWS), (False, R.DENSE_CHUNK)]


def upload(c):
    c.cache.k_tok.copy_(c.k)
    c.cache.v_tok.copy_(c.v)
    c.qd = c.q.cuda()


@pytest.mark.parametrize("n,view", [(1, {}), (6, dict(causal=True, own=True)), (150, dict(causal=True, own=True)),
                                    (6, dict(causal=True, own=True, sinks=3, window=50)), (1, dict(sinks=20, window=30))])
@pytest.mark.parametrize("L", [400, 3000])
def test_infinities_that_every_query_sees(n, view, L):
    """A weighted mean with an infinite value is that infinity wherever the token lies: all queries
    of a tile see it here, so no mask sends its step to a path of its own."""
    c = Case(1, 2, 4, L, n, seed=n)
    v, ref = split_view(view)
    t = L - n - 20
    c.v[0, :, t, :10] = math.inf
    c.v[0, :, t, 10:20] = -math.inf
    c.v[0, :, t, 20] = math.inf
    c.v[0, :, t - 3, 20] = -math.inf
    c.v[0, 1, t, 30] = math.nan
    upload(c)
    want = c.want(**ref)
    assert torch.isinf(want[..., :20]).all() and torch.isnan(want[..., 20]).all()
    off = ~torch.isfinite(want)
    for fp32, kernel in RUNS:
        v.kernel = kernel
        got = c.attend(fp32, v).double().cpu()
        assert torch.equal(torch.nan_to_num(got[off], nan=5.0), torch.nan_to_num(want[off], nan=5.0))
        check(got.masked_fill(off, 0.0), want.masked_fill(off, 0.0), fp32, c.bound())


def staircase(n, steps, seed, values=1.0, L=400):
    """A case whose scores, in powers of two, are `steps`[t] for every query row (the others' are 0)."""
    c = Case(1, 2, 4, L, n, seed=seed)
    c.softmax = math.log(2.0)
    c.p = params(2, 4, softmax_scale=c.softmax)
    c.q.zero_()
    c.q[..., 63] = 8.0
    c.k.zero_()
    for t, s in steps.items():
        c.k[0, :, t, 63] = s / 8.0
    c.v = (c.v.float() * values).bfloat16()
    upload(c)
    return c


STAIRS = [
    {40: 60.0, 200: 65.0},                          # 2^60 held against a maximum of 2^0, then 2^-5 of the new one
    {1: 64.0, 33: 65.0, 34: 64.0, 399 - 150: 66.0},  # weights of 2^64, then just past it
    {100: 64.0, 101: 64.0, 230: 65.0, 231: 130.0},
    {0: 64.0, 16: 130.0, 64: 129.0, 128: 128.0},
    {t: 0.5 * t for t in range(250)},               # grows from step to step
]


def spread(c, fp32, kernel, view):
    """Largest error against the largest value, and what its roundings allow."""
    view.kernel = kernel
    got = c.attend(fp32, view).double().cpu()
    want = c.want(causal=bool(view.causal), own=bool(view.own_token), scale=c.softmax)
    assert torch.isfinite(got).all()
    top = float(c.v[:, :, :c.L].double().abs().max())
    allowed = 2.0 ** -14 + 2 * 2.0 ** -16 + (0.0 if fp32 else 2.0 ** -8) + (2.0 ** -8 if kernel == R.DENSE_CHUNK else 0.0)
    return float((got - want).abs().max()) / top, allowed


@pytest.mark.parametrize("n", [1, 3, 150])
@pytest.mark.parametrize("steps", STAIRS, ids=range(len(STAIRS)))
def test_maxima_that_lag(steps, n):
    """Scores that outgrow the maximum a row started with, by less and by more than 2^64: what was
    summed before weighs in the output with the right factor."""
    c = staircase(n, steps, seed=1)
    for fp32, kernel in RUNS:
        off, allowed = spread(c, fp32, kernel, R.View(causal=n > 1, own_token=n > 1))
        assert off <= allowed, (off, allowed)


@pytest.mark.parametrize("n", [1, 3, 150])
@pytest.mark.parametrize("values", [2.0 ** 70, 2.0 ** 100, 2.0 ** 125])
def test_large_finite_values(values, n):
    """Means of large values are finite, also where their sums under lagging maxima would not be."""
    for steps in (STAIRS[0], STAIRS[2], STAIRS[4], {}):
        c = staircase(n, steps, seed=2, values=1.0)
        c.v = (c.v.float().clamp(-1.9, 1.9) * values).bfloat16()
        upload(c)
        for fp32, kernel in RUNS:
            off, allowed = spread(c, fp32, kernel, R.View(causal=n > 1, own_token=n > 1))
            assert off <= allowed, (steps, fp32, kernel, off, allowed)


def test_the_largest_value_everywhere():
    top = float(torch.finfo(torch.bfloat16).max)
    for L in (17, 5000):
        c = Case(2, 2, 4, L, 1, seed=3)
        c.v[:] = top
        c.v[..., ::2] *= -1
        upload(c)
        for fp32, kernel in RUNS:
            got = c.attend(fp32, R.View(kernel=kernel)).double().cpu()
            want = torch.where(torch.arange(128) % 2 == 0, -top, top).double()
            # weights and their sum: parts of 2^-16, fp32 sums of up to 5000 terms
            assert float((got / want - 1).abs().max()) <= (2.0 ** -15 if fp32 else 2.0 ** -8)
