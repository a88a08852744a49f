"""Buffers of a dense call that may not overlap (host checks: nothing is launched, no GPU needed)."""

import ctypes

import pytest

import hierarchical_sparse_attention_build_b200 as R
from test_dense_host import FAKE, INVALID, P, T, call, evict, refused

Q_BYTES = 2 * 8 * 256  # batch 2, 8 query heads: one query
CACHE = 2 * 2 * 256 * 256  # batch 2, 2 KV heads, 256 slots
FAR = 1 << 32


def overlaps(*args):
    refused(INVALID, *args)
    assert "overlaps" in R.last_error(), R.last_error()


@pytest.mark.parametrize("op,n", [("attend", 3), ("prefill", 3), ("step", 1)])
def test_out_over_q(op, n):
    t = T(seq_len=FAKE)
    q = FAKE + FAR
    for out in (q, q + 16, q + n * Q_BYTES - 16, q - 16, q - 2 * n * Q_BYTES + 16):  # (fp32 output: twice q's bytes)
        overlaps(*call(op, t=t, n=n, q=q, out=out))


def test_weights_over_q():
    q = FAKE + FAR
    for w in (q, q + 3 * Q_BYTES - 16, q - 2 * 2 * 256 * 4 + 16):
        overlaps(*call("weights", q=q, out=w))


def other(at, **kw):
    return T(**{**dict(k_tok=at, v_tok=at + CACHE, length=0), **kw})


def test_evict_over_itself():
    tree = T(k_tok=FAKE + FAR, v_tok=FAKE + 2 * FAR)
    base = dict(t=tree, w=FAKE, kept=FAKE + (1 << 20))
    # K and V rows in one place; a receiving cache that begins or ends inside the other's rows
    overlaps(*evict(t=T(), w=FAKE + FAR, kept=FAKE + 2 * FAR))
    overlaps(*evict(into=other(FAKE + 3 * FAR, v_tok=FAKE + 3 * FAR + 16), **base))
    for at in (FAKE + FAR + 16, FAKE + FAR - CACHE + 16, FAKE + 2 * FAR + CACHE - 16, FAKE + FAR - 2 * CACHE + 256):
        overlaps(*evict(into=other(at), **base))
    # weights and kept slots
    into = other(FAKE + 3 * FAR)
    wbytes, kbytes = 2 * 2 * 256 * 4, 2 * 2 * 32 * 4
    for iw in (FAKE + 16, FAKE - wbytes + 16):
        overlaps(*evict(iw=iw, **base))
        overlaps(*evict(into=into, iw=iw, **base))
    for kept in (FAKE, FAKE + wbytes - 16, FAKE - kbytes + 16):
        overlaps(*evict(t=tree, w=FAKE, kept=kept))
    overlaps(*evict(t=tree, w=FAKE, kept=FAKE + 2 * wbytes, iw=FAKE + 2 * wbytes + kbytes - 16))
    assert ctypes.sizeof(R.View) == 24
