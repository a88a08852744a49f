"""The dense cache operators as a causal RoPE model's dense and windowed layers call them.

The expected values come from the layer's textbook form, token by token: the query of token i
sits at position i and sees the tokens j <= i at their positions j, with a window the last
`window` of them and the first `sinks`, renumbered 0, 1, ... when the sinks are scored by rank.
Tolerances are test_gpu_dense.py's.
"""

import pytest
import torch

import hierarchical_sparse_attention_build_b200 as R
from test_gpu_dense import BASE, Case, check

pytestmark = pytest.mark.gpu


def turn(x, pos):
    """Rows x [m][128] (fp64) as 64 complex pairs turned by their positions pos [m]."""
    z = torch.complex(x[:, :64], x[:, 64:])
    freq = torch.tensor([BASE ** (-2.0 * i / 128) for i in range(64)], dtype=torch.float64)
    a = pos.double()[:, None] * freq
    return z * torch.polar(torch.ones_like(a), a)


def token_weights(q, k, i, window=0, sinks=0, token_positions=False):
    """(tokens, weights [rows][tokens]) of the query rows q [rows][128] of token i over k [> i][128]."""
    see = torch.arange(i + 1)
    at = see
    if window:
        see = see[(see < sinks) | (see > i - window)]
        at = see if token_positions else torch.arange(len(see))
    kz = turn(k[see].double(), at)
    qz = turn(q.double(), at[-1:].expand(q.shape[0]))
    s = (qz @ kz.conj().T).real * 128 ** -0.5
    return see, torch.softmax(s, dim=-1)


def layer(c, q, first, weights=False, **view):
    """The queries q [B][n][Hq][128] of tokens first[b], first[b] + 1, ... of a Case's caches."""
    out = torch.zeros(q.shape, dtype=torch.float64)
    got = torch.zeros(c.B, c.H, c.cap, dtype=torch.float64)
    for b in range(c.B):
        for n in range(q.shape[1]):
            for h in range(c.H):
                rows = slice(h * c.G, (h + 1) * c.G)
                see, w = token_weights(q[b, n, rows], c.k[b, h], first[b] + n, **view)
                out[b, n, rows] = w @ c.v[b, h, see].double()
                got[b, h, see] += w.sum(0)
    return got if weights else out


VIEWS = [{}, dict(window=60), dict(window=60, sinks=5), dict(window=60, sinks=5, token_positions=True),
         dict(window=400, sinks=3)]


@pytest.mark.parametrize("view", VIEWS, ids=str)
@pytest.mark.parametrize("n,page,lens", [(1, 0, None), (3, 16, [300, 3]), (90, 0, None), (90, 64, [300, 100])])
def test_chunk_queries_sit_at_their_tokens(view, n, page, lens):
    c = Case(2, 2, 4, 300, n, seed=n, page=page, lens=lens, spare=4)
    want = layer(c, c.q, [m - n for m in c.lens], **view)
    for fp32, kernel in ((True, R.DENSE_AUTO), (False, R.DENSE_ROWS), (False, R.DENSE_CHUNK)):
        got = c.attend(fp32, R.View(causal=True, at_token=True, kernel=kernel, **view))
        check(got, want, fp32, c.bound())


@pytest.mark.parametrize("view", VIEWS, ids=str)
def test_a_layers_prompt_and_decode_steps(view):
    """A prompt in two chunks, then decode steps: the outputs of one causal pass over all tokens."""
    B, H, G, n = 2, 2, 4, 100
    c = Case(B, H, G, 1, n, seed=3, lens=[0, 0], spare=2 * n + 7)
    c.cache.length = 0
    g = torch.Generator().manual_seed(4)
    v = R.View(at_token=True, **view)
    for m in (n, n, 1, 1, 1):
        k, val = (torch.randn(B, m, H, 128, generator=g).bfloat16() for _ in range(2))
        q = torch.randn(B, m, H * G, 128, generator=g).bfloat16()
        at = c.lens[0]
        c.k[:, :, at:at + m], c.v[:, :, at:at + m] = k.transpose(1, 2), val.transpose(1, 2)
        out = torch.empty(B, m, H * G, 128, device="cuda")
        new = [x.cuda() for x in (k, val, q)]
        if m == 1:
            R.dense_decode_step(c.p, c.cache, *new, out, c.ws, v)
            c.cache.length += 1
        else:
            R.dense_prefill_chunk(c.p, c.cache, *new, out, c.ws, v)
        R.check_device_errors(c.ws)
        c.lens = [at + m] * B
        c.q = q
        check(out, layer(c, q, [at] * B, **view), True, c.bound())
        if m == 1:  # the last token's query, asked for again without an append
            R.dense_attend(c.p, c.cache, new[2], out, c.ws, v)
            check(out, layer(c, q, [at] * B, **view), True, c.bound())


@pytest.mark.parametrize("n,lens", [(1, None), (2, [300, 40]), (70, None), (70, [300, 90])])
def test_weights_of_a_layer(n, lens):
    """Both kernels: at most 8 query rows a KV group, and more."""
    c = Case(2, 2, 4, 300, n, seed=n + 50, lens=lens, spare=3)
    want = layer(c, c.q, [m - n for m in c.lens], weights=True)
    for causal in (True, False) if n == 1 else (True,):
        w = torch.zeros(2, 2, c.cap, device="cuda")
        R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, R.View(causal=causal, at_token=True))
        R.check_device_errors(c.ws)
        assert float((w.double().cpu() - want).norm() / want.norm()) <= 2.0 ** -16
