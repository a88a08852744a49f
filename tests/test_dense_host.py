"""Refusals of the dense cache operators (host checks: nothing is launched, no GPU needed)."""

import ctypes
import os
import re

import pytest
import torch

import hierarchical_sparse_attention_build_b200 as R

lib = R.raw_library()
INVALID, UNSUPPORTED, WS_SMALL, CAPACITY = 1, 2, 3, 4
FAKE = 0x7F0000000000  # aligned, never dereferenced
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "recsa_dense.h")


def P(**kw):
    return R.params(**{**dict(num_kv_heads=2, num_q_heads=8, branching=16, top_k=4), **kw})


def T(**kw):
    t = R.Tree(2, 0, 256, 100, FAKE, FAKE, None, None, None, None, None, 0, 0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def refused(code, name, *args):
    got = getattr(lib, name)(*args)
    assert got == code, (name, got, R.last_error())
    assert R.status_string(code) in R.last_error()


def call(op, p=None, t=None, view=None, q=FAKE, n=3, out=FAKE, ws=FAKE, nbytes=1 << 40, k=FAKE, v=FAKE):
    p, t = p or P(), t or T()
    p, t = ctypes.byref(p), ctypes.byref(t)
    view = ctypes.byref(view) if view is not None else None
    return {
        "attend": ("recsa_dense_attend", p, t, view, q, n, out, 1, ws, nbytes, None),
        "prefill": ("recsa_dense_prefill_chunk", p, t, view, k, v, q, n, out, 1, ws, nbytes, None),
        "step": ("recsa_dense_decode_step", p, t, view, k, v, q, out, 1, ws, nbytes, None),
        "weights": ("recsa_accumulate_weights", p, t, view, q, n, out, 0, ws, nbytes, None),
    }[op]


OPS = ["attend", "prefill", "step", "weights"]


def test_every_declared_call_is_exported():
    names = re.findall(r"RECSA_API\s+[^;()]*?\b(recsa_\w+)\s*\(", open(HEADER).read())
    assert set(names) == {"recsa_dense_workspace_size", "recsa_dense_workspace_init", "recsa_dense_attend",
                          "recsa_dense_prefill_chunk", "recsa_dense_decode_step", "recsa_accumulate_weights",
                          "recsa_evict"}
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value


@pytest.mark.parametrize("op", OPS)
def test_bad_caches_and_buffers(op):
    seq = dict(seq_len=FAKE)
    refused(INVALID, *call(op, t=T(k_tok=None, **seq)))
    refused(INVALID, *call(op, t=T(v_tok=FAKE + 8, **seq)))
    refused(INVALID, *call(op, t=T(k_node=FAKE, **seq)))  # a tree is given whole or not at all
    refused(INVALID, *call(op, t=T(length=257, **seq)))
    refused(INVALID, *call(op, t=T(seq_len=FAKE + 4)))
    refused(INVALID, *call(op, t=T(page_table=FAKE, page_size=24, num_pages=9, **seq)))
    refused(INVALID, *call(op, t=T(page_table=FAKE, page_size=16, num_pages=0, **seq)))
    refused(INVALID, *call(op, t=T(**seq), q=None))
    refused(INVALID, *call(op, t=T(**seq), q=FAKE + 2))
    refused(INVALID, *call(op, t=T(**seq), out=None))
    refused(INVALID, *call(op, t=T(**seq), ws=None))
    refused(INVALID, *call(op, t=T(**seq), ws=FAKE + 8))
    refused(WS_SMALL, *call(op, t=T(**seq), nbytes=R.dense_workspace_size(P(), 2, 256) - 1))
    refused(UNSUPPORTED, *call(op, p=P(num_q_heads=6), t=T(**seq)))
    refused(UNSUPPORTED, *call(op, p=P(head_dim=64), t=T(**seq)))
    refused(INVALID, *call(op, p=P(rope_base=0.0), t=T(**seq)))


@pytest.mark.parametrize("op", OPS)
def test_bad_views(op):
    t = T(seq_len=FAKE)
    refused(INVALID, *call(op, t=t, view=R.View(sinks=-1, window=4)))
    refused(INVALID, *call(op, t=t, view=R.View(window=-1)))
    refused(UNSUPPORTED, *call(op, t=t, view=R.View(sinks=1 << 30, window=1)))
    refused(INVALID, *call(op, t=t, view=R.View(kernel=3)))
    refused(INVALID, *call(op, t=t, view=R.View(kernel=-1)))
    if op != "weights":
        refused(UNSUPPORTED, *call(op, t=t, view=R.View(kernel=R.DENSE_CHUNK)))  # (the calls here write fp32)
    v = R.View(window=4)
    v.sink_positions = 2
    refused(INVALID, *call(op, t=t, view=v))


def test_counts_and_room():
    refused(INVALID, *call("attend", n=0))
    refused(INVALID, *call("weights", n=-1))
    refused(INVALID, *call("prefill", n=0))
    refused(CAPACITY, *call("prefill", n=157))
    refused(INVALID, *call("prefill", k=None))
    refused(INVALID, *call("prefill", v=FAKE + 4))
    refused(INVALID, *call("step"))  # no per-sequence lengths
    refused(INVALID, *call("step", t=T(seq_len=FAKE), k=None))
    refused(UNSUPPORTED, *call("weights", view=R.View(window=8)))
    refused(UNSUPPORTED, *call("weights", n=(1 << 31) - 1))
    refused(UNSUPPORTED, *call("attend", n=(1 << 31) - 1))
    assert R.View(sinks=3, window=9, causal=True, own_token=True, token_positions=True).sink_positions == 1


def test_workspace_arguments():
    n = ctypes.c_size_t()
    refused(INVALID, "recsa_dense_workspace_size", ctypes.byref(P()), 0, 64, ctypes.byref(n))
    refused(INVALID, "recsa_dense_workspace_size", ctypes.byref(P()), 1, 0, ctypes.byref(n))
    refused(UNSUPPORTED, "recsa_dense_workspace_size", ctypes.byref(P()), 1, (1 << 30) + 1, ctypes.byref(n))
    refused(INVALID, "recsa_dense_workspace_size", ctypes.byref(P()), 1, 64, None)
    refused(INVALID, "recsa_dense_workspace_init", ctypes.byref(P()), 1, 64, None, 1 << 40, None)
    refused(INVALID, "recsa_dense_workspace_init", ctypes.byref(P()), 1, 64, FAKE + 4, 1 << 40, None)
    refused(WS_SMALL, "recsa_dense_workspace_init", ctypes.byref(P()), 1, 64, FAKE, 1024, None)


def evict(t=None, into=None, keep=32, sinks=0, recent=0, w=FAKE, kept=FAKE, iw=None):
    return ("recsa_evict", ctypes.byref(P()), ctypes.byref(t or T()), w, keep, sinks, recent, kept,
            ctypes.byref(into) if into is not None else None, iw, None)


def test_evict_refusals():
    refused(INVALID, *evict(keep=0))
    refused(INVALID, *evict(sinks=-1))
    refused(INVALID, *evict(recent=-1))
    refused(INVALID, *evict(sinks=20, recent=13))
    refused(INVALID, *evict(w=None))
    refused(INVALID, *evict(w=FAKE + 4))
    refused(INVALID, *evict(kept=None))
    refused(INVALID, *evict(iw=FAKE + 4))
    other = dict(k_tok=FAKE + 4096, v_tok=FAKE + 8192)
    refused(INVALID, *evict(into=T(batch=3, **other)))
    refused(CAPACITY, *evict(into=T(capacity=31, length=0, **other)))
    refused(INVALID, *evict(t=T(seq_len=FAKE), into=T(**other)))
    refused(INVALID, *evict(t=T(seq_len=FAKE), into=T(seq_len=FAKE, **other)))
    refused(INVALID, *evict(into=T(k_tok=FAKE, v_tok=FAKE + 8192)))
    refused(INVALID, *evict(into=T(**other), iw=FAKE))  # weights written while other blocks read them


def test_binding_refuses_wrong_tensors():
    p = P()
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    c = R.TokenCache(p, z(2, 2, 64, 128), z(2, 2, 64, 128), 10)
    assert c.c.k_node is None and c.c.pooler is None
    q = z(2, 3, 8, 128)
    for bad_q, bad_out in ((q.float(), q), (q, q.half()), (z(1, 3, 8, 128), q), (z(2, 3, 4, 128), q),
                           (q.transpose(0, 1), q), (q, z(2, 2, 8, 128)), (z(2, 3, 8, 64), q)):
        with pytest.raises(R.RecsaError):
            R._dense_q(p, c, bad_q, bad_out, None)
    with pytest.raises(R.RecsaError):
        R._dense_new(p, c, z(2, 2, 2, 128), z(2, 3, 2, 128), q)
    with pytest.raises(R.RecsaError):
        R.evict(p, c, z(2, 2, 63, dt=torch.float32), 8, z(2, 2, 8, dt=torch.int32))
    with pytest.raises(R.RecsaError):
        R._weights_of(c, z(2, 2, 64, dt=torch.float64), "weights")
    with pytest.raises(R.RecsaError):
        R.DenseWorkspace(p, 2, 64, "cpu")


def test_own_token_values():
    assert [R.View(own_token=o, at_token=t).own_token for o, t in ((False, False), (True, False), (True, True),
                                                                   (False, True))] == [0, 1, 2, 2]
    for bad in (-1, 3):
        v = R.View()
        v.own_token = bad
        for op in OPS:
            refused(INVALID, *call(op, t=T(seq_len=FAKE), view=v))
