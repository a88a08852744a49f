"""What the binding of the dense calls checks of a cache before it hands out pointers (no GPU: the
current device is taken to be the host's, so that tensors of the meta device are elsewhere)."""

from types import SimpleNamespace

import pytest
import torch

import hierarchical_sparse_attention_build_b200 as R
from test_dense_host import P


def zeros(*s, dt=torch.bfloat16, dev="cpu"):
    return torch.zeros(*s, dtype=dt, device=dev)


@pytest.fixture
def here(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=0))

    class Launched(Exception):
        pass

    def launch(*a):
        raise Launched

    class Library:
        recsa_dense_attend = recsa_dense_prefill_chunk = recsa_dense_decode_step = staticmethod(launch)
        recsa_accumulate_weights = recsa_evict = staticmethod(launch)

        def __getattr__(self, name):
            return getattr(real, name)

    real = R.raw_library()
    monkeypatch.setattr(R, "_lib", Library())
    return Launched


def calls(p, cache, H=2, Hq=8):
    ws = SimpleNamespace(buf=zeros(64, dt=torch.uint8), nbytes=64)
    q, out, new = zeros(2, 1, Hq, 128), zeros(2, 1, Hq, 128), zeros(2, 1, H, 128)
    w, kept = zeros(2, H, 64, dt=torch.float32), zeros(2, H, 8, dt=torch.int32)
    return [lambda: R.dense_attend(p, cache, q, out, ws), lambda: R.dense_prefill_chunk(p, cache, new, new, q, out, ws),
            lambda: R.dense_decode_step(p, cache, new, new, q, out, ws), lambda: R.accumulate_weights(p, cache, q, w, ws),
            lambda: R.evict(p, cache, w, 8, kept)]


def test_a_cache_on_one_device_is_accepted(here):
    cache = R.TokenCache(P(), zeros(2, 2, 64, 128), zeros(2, 2, 64, 128), 10, seq_len=zeros(2, dt=torch.int64))
    for call in calls(P(), cache):
        with pytest.raises(here):
            call()


@pytest.mark.parametrize("what", ["v_tok", "seq_len", "page_table", "pooler", "v_node"])
def test_every_tensor_of_a_cache_is_on_the_current_device(here, what):
    dev = lambda name: "meta" if name == what else "cpu"  # noqa: E731
    paged = what == "page_table"
    rows = [zeros(*((9, 2, 16, 128) if paged else (2, 2, 64, 128)), dev=dev(n)) for n in ("k_tok", "v_tok")]
    kw = dict(seq_len=zeros(2, dt=torch.int64, dev=dev("seq_len")))
    if paged:
        kw["page_table"] = zeros(2, 4, dt=torch.int32, dev=dev("page_table"))
    if what in ("pooler", "v_node"):
        nodes = R.tree_layout(P(), 2, 64)[0]
        cache = R.RecsaTree(P(), *rows, zeros(128, 128, dt=torch.float32, dev=dev("pooler")), 10,
                            k_node=zeros(nodes, 128), v_node=zeros(nodes, 128, dev=dev("v_node")), **kw)
    else:
        cache = R.TokenCache(P(), *rows, 10, **kw)
    for call in calls(P(), cache):
        with pytest.raises(R.RecsaError, match="current device"):
            call()
    other = R.TokenCache(P(), zeros(2, 2, 64, 128), zeros(2, 2, 64, 128), 10)
    with pytest.raises(R.RecsaError, match="current device"):
        R.evict(P(), other, zeros(2, 2, 64, dt=torch.float32), 8, zeros(2, 2, 8, dt=torch.int32), into=cache)


def test_params_and_cache_agree_on_the_heads(here):
    cache = R.TokenCache(P(), zeros(2, 2, 64, 128), zeros(2, 2, 64, 128), 10)
    for call in calls(P(num_kv_heads=4, num_q_heads=8), cache, H=4):
        with pytest.raises(R.RecsaError, match="KV heads|contiguous float32"):
            call()
    four = R.TokenCache(P(num_kv_heads=4), zeros(2, 4, 64, 128), zeros(2, 4, 64, 128), 10)
    with pytest.raises(R.RecsaError, match="KV heads"):
        R.evict(P(), cache, zeros(2, 2, 64, dt=torch.float32), 8, zeros(2, 2, 8, dt=torch.int32), into=four)
