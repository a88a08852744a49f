"""Python binding of librecsa: RecSA tree build and level-wise sparse attend on B200.

Thin ctypes marshalling over the C ABI declared in ``include/recsa.h`` and
``include/recsa_dense.h``; every step of
the computation runs in the library's CUDA kernels.  PyTorch supplies device memory
and the current CUDA stream.  Importing this module fails loudly when the compiled
library is missing: there is no CPU fallback.
"""

from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librecsa.so")

HEAD_DIM = 128
TOPK_ALL = 0x7FFFFFFF
MAX_LEVELS = 40
MAX_CANDIDATES = 4096

STATUS = {
    0: "RECSA_OK",
    1: "RECSA_ERR_INVALID_ARGUMENT",
    2: "RECSA_ERR_UNSUPPORTED",
    3: "RECSA_ERR_WORKSPACE_TOO_SMALL",
    4: "RECSA_ERR_CAPACITY",
    5: "RECSA_ERR_CUDA",
    6: "RECSA_ERR_DEVICE_CHECK",
    7: "RECSA_ERR_TIMEOUT",
}


class RecsaError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{STATUS.get(code, code)}: {message}")
        self.code = code


class Params(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("branching", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("rope_base", ctypes.c_float),
        ("softmax_scale", ctypes.c_float),
    ]


class Tree(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("capacity", ctypes.c_int64),
        ("length", ctypes.c_int64),
        ("k_tok", ctypes.c_void_p),
        ("v_tok", ctypes.c_void_p),
        ("k_node", ctypes.c_void_p),
        ("v_node", ctypes.c_void_p),
        ("pooler", ctypes.c_void_p),
        ("seq_len", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
    ]


class Debug(ctypes.Structure):
    _fields_ = [
        ("sel_idx", ctypes.c_void_p),
        ("entries", ctypes.c_void_p),
        ("sel_levels", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("cluster_size", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


KERNEL_AUTO, KERNEL_CTA, KERNEL_WARP, KERNEL_LEAN = 0, 1, 2, 3


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (nvcc, sm_100a)"
        )
    lib = ctypes.CDLL(LIB_PATH)
    P, T, D = ctypes.POINTER(Params), ctypes.POINTER(Tree), ctypes.POINTER(Debug)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "recsa_tree_layout": [P, i32, i64, ctypes.POINTER(i64), ctypes.POINTER(i32), ctypes.POINTER(i64)],
        "recsa_workspace_size": [P, i64, ctypes.POINTER(sz)],
        "recsa_workspace_init": [P, i64, vp, sz, vp],
        "recsa_build_tree": [P, T, vp],
        "recsa_decode": [P, T, vp, i32, vp, i32, vp, sz, D, vp],
        "recsa_decode_host": [P, T, vp, i32, vp, i32, vp, vp, vp, sz, D, vp],
        "recsa_append": [P, T, vp, vp, i32, vp],
        "recsa_decode_step": [P, T, vp, vp, vp, vp, i32, vp, sz, vp],
        "recsa_prefill_chunk": [P, T, vp, vp, vp, i32, vp, i32, vp, sz, D, vp],
        "recsa_check_device_errors": [vp, vp],
        "recsa_decode_no_alloc": [P, T, vp, i32, vp, i32, vp],
        "recsa_dense_workspace_size": [P, i32, i64, ctypes.POINTER(sz)],
        "recsa_dense_workspace_init": [P, i32, i64, vp, sz, vp],
        "recsa_dense_attend": [P, T, vp, vp, i32, vp, i32, vp, sz, vp],
        "recsa_dense_prefill_chunk": [P, T, vp, vp, vp, vp, i32, vp, i32, vp, sz, vp],
        "recsa_dense_decode_step": [P, T, vp, vp, vp, vp, vp, i32, vp, sz, vp],
        "recsa_accumulate_weights": [P, T, vp, vp, i32, vp, i32, vp, sz, vp],
        "recsa_evict": [P, T, vp, i32, i32, i32, vp, T, vp, vp],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.recsa_status_string.argtypes = [ctypes.c_int]
    lib.recsa_status_string.restype = ctypes.c_char_p
    lib.recsa_last_error.argtypes = []
    lib.recsa_last_error.restype = ctypes.c_char_p
    return lib


_lib = _load()


def _check(code: int) -> None:
    if code != 0:
        raise RecsaError(code, _lib.recsa_last_error().decode())


def _stream(stream=None) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t) -> ctypes.c_void_p | None:
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def params(num_kv_heads: int, num_q_heads: int, branching: int, top_k: int, rope_base: float = 1.0e6,
           softmax_scale: float = 0.0, head_dim: int = HEAD_DIM) -> Params:
    return Params(head_dim, num_kv_heads, num_q_heads, branching, top_k, rope_base, softmax_scale)


def tree_layout(p: Params, batch: int, capacity: int):
    """(node_rows, levels, level_row_offsets[0..levels]) of the node arena."""
    rows = ctypes.c_int64()
    levels = ctypes.c_int32()
    offs = (ctypes.c_int64 * (MAX_LEVELS + 1))()
    _check(_lib.recsa_tree_layout(ctypes.byref(p), batch, capacity, ctypes.byref(rows), ctypes.byref(levels), offs))
    return rows.value, levels.value, list(offs[: levels.value + 1])


def workspace_size(p: Params, capacity: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.recsa_workspace_size(ctypes.byref(p), capacity, ctypes.byref(n)))
    return n.value


class RecsaTree:
    """A layer's token caches plus its node arena (torch tensors) and the C struct over them."""

    def __init__(self, p: Params, k_tok: torch.Tensor, v_tok: torch.Tensor, pooler: torch.Tensor, length: int,
                 k_node: torch.Tensor | None = None, v_node: torch.Tensor | None = None,
                 seq_len: torch.Tensor | None = None, page_table: torch.Tensor | None = None):
        """k_tok, v_tok: contiguous caches [batch][Hkv][capacity][128], or with page_table (int32
        [batch][pages per sequence] device tensor) a page pool [num_pages][Hkv][page_size][128].
        seq_len: optional int64 [batch] device tensor of per-sequence lengths (length is then
        the longest); the library advances it on the device when it appends."""
        assert k_tok.dtype == torch.bfloat16 and v_tok.dtype == torch.bfloat16 and pooler.dtype == torch.float32
        assert k_tok.is_contiguous() and v_tok.is_contiguous() and pooler.is_contiguous()
        assert v_tok.shape == k_tok.shape and k_tok.shape[3] == HEAD_DIM and k_tok.shape[1] == p.num_kv_heads
        if page_table is None:
            batch, _, capacity, _ = k_tok.shape
            num_pages = page_size = 0
        else:
            assert page_table.dtype == torch.int32 and page_table.is_contiguous() and page_table.dim() == 2
            num_pages, _, page_size, _ = k_tok.shape
            batch = page_table.shape[0]
            capacity = page_table.shape[1] * page_size
        self.p = p
        rows, self.levels, self.level_offsets = tree_layout(p, batch, capacity)
        if k_node is None:
            k_node = torch.empty(max(rows, 1), HEAD_DIM, dtype=torch.bfloat16, device=k_tok.device)
            v_node = torch.empty_like(k_node)
        self.k_tok, self.v_tok, self.k_node, self.v_node, self.pooler = k_tok, v_tok, k_node, v_node, pooler
        self.node_rows = rows
        if seq_len is not None:
            assert seq_len.dtype == torch.int64 and seq_len.is_contiguous() and seq_len.numel() == batch
        self.seq_len = seq_len
        self.page_table = page_table
        self.devices = {t.device for t in (k_tok, v_tok, k_node, v_node, pooler, seq_len, page_table) if t is not None}
        self.c = Tree(batch, 0, capacity, length, k_tok.data_ptr(), v_tok.data_ptr(), k_node.data_ptr(),
                      v_node.data_ptr(), pooler.data_ptr(), seq_len.data_ptr() if seq_len is not None else None,
                      page_table.data_ptr() if page_table is not None else None, page_size, num_pages)

    @property
    def length(self) -> int:
        return self.c.length

    @length.setter
    def length(self, v: int) -> None:
        self.c.length = v

    @property
    def batch(self) -> int:
        return self.c.batch

    @property
    def capacity(self) -> int:
        return self.c.capacity

    def level_rows(self, level: int) -> torch.Tensor:
        """Node-arena rows of `level` as [batch][Hkv][slots][128] views (K, V)."""
        slots = -(-self.capacity // self.p.branching ** level)
        o = self.level_offsets[level]
        n = self.batch * self.p.num_kv_heads * slots
        shape = (self.batch, self.p.num_kv_heads, slots, HEAD_DIM)
        return self.k_node[o:o + n].view(shape), self.v_node[o:o + n].view(shape)


class Workspace:
    """Device workspace (RoPE table + error word) initialised for a params/capacity pair."""

    def __init__(self, p: Params, capacity: int, device, stream=None, buffer: torch.Tensor | None = None):
        self.nbytes = workspace_size(p, capacity)
        self.buf = buffer if buffer is not None else torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        workspace_init(p, capacity, self.buf, stream)


def workspace_init(p: Params, capacity: int, buf: torch.Tensor, stream=None) -> None:
    _check(_lib.recsa_workspace_init(ctypes.byref(p), capacity, _ptr(buf), buf.numel() * buf.element_size(),
                                     _stream(stream)))


def build_tree(p: Params, tree: RecsaTree, stream=None) -> None:
    _check(_lib.recsa_build_tree(ctypes.byref(p), ctypes.byref(tree.c), _stream(stream)))


def _debug(sel_idx=None, sel_levels=0, cluster_size=0, entries=None, kernel=0):
    if sel_idx is None and entries is None and cluster_size == 0 and kernel == 0:
        return None
    return Debug(sel_idx.data_ptr() if sel_idx is not None else None,
                 entries.data_ptr() if entries is not None else None, sel_levels, kernel, cluster_size, 0)


def decode(p: Params, tree: RecsaTree, q: torch.Tensor, out: torch.Tensor, ws: Workspace, sel_idx=None,
           sel_levels: int = 0, entries=None, cluster_size: int = 0, kernel: int = 0, stream=None) -> None:
    """recsa_decode: q [B][Q][Hq][128] bf16 -> out [B][Q][Hq][128] (fp32 or bf16)."""
    assert q.dtype == torch.bfloat16 and q.is_contiguous() and out.is_contiguous()
    nq = q.shape[1]
    dbg = _debug(sel_idx, sel_levels, cluster_size, entries, kernel)
    _check(_lib.recsa_decode(ctypes.byref(p), ctypes.byref(tree.c), _ptr(q), nq, _ptr(out),
                             int(out.dtype == torch.float32), _ptr(ws.buf), ws.nbytes,
                             ctypes.byref(dbg) if dbg is not None else None, _stream(stream)))


def decode_host(p: Params, tree: RecsaTree, q_host: torch.Tensor, out_host: torch.Tensor, q_dev: torch.Tensor,
                out_dev: torch.Tensor, ws: Workspace, stream=None) -> None:
    """recsa_decode_host: host q -> device staging -> decode -> host out, queued in one call."""
    for t in (q_host, out_host):
        assert t.device.type == "cpu" and t.is_contiguous()
    assert q_host.dtype == torch.bfloat16 and q_dev.shape == q_host.shape and out_dev.shape == out_host.shape
    assert out_dev.dtype == out_host.dtype and q_dev.is_contiguous() and out_dev.is_contiguous()
    _check(_lib.recsa_decode_host(ctypes.byref(p), ctypes.byref(tree.c), _ptr(q_host), q_host.shape[1],
                                  _ptr(out_host), int(out_host.dtype == torch.float32), _ptr(q_dev), _ptr(out_dev),
                                  _ptr(ws.buf), ws.nbytes, None, _stream(stream)))


def append(p: Params, tree: RecsaTree, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
    """recsa_append: append [B][C][Hkv][128] K/V to every sequence and rebuild the nodes over them."""
    for t in (k_new, v_new):
        assert t.dtype == torch.bfloat16 and t.is_contiguous()
    _check(_lib.recsa_append(ctypes.byref(p), ctypes.byref(tree.c), _ptr(k_new), _ptr(v_new), k_new.shape[1],
                             _stream(stream)))


def decode_step(p: Params, tree: RecsaTree, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                out: torch.Tensor, ws: Workspace, stream=None) -> None:
    """recsa_decode_step: append one token per sequence at its device length, advance the
    lengths, decode the token's query; graph-capturable (needs tree.seq_len)."""
    for t in (k_new, v_new, q):
        assert t.dtype == torch.bfloat16 and t.is_contiguous() and t.shape[1] == 1
    _check(_lib.recsa_decode_step(ctypes.byref(p), ctypes.byref(tree.c), _ptr(k_new), _ptr(v_new), _ptr(q),
                                  _ptr(out), int(out.dtype == torch.float32), _ptr(ws.buf), ws.nbytes,
                                  _stream(stream)))


def prefill_chunk(p: Params, tree: RecsaTree, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                  out: torch.Tensor, ws: Workspace, sel_idx=None, sel_levels: int = 0, entries=None,
                  cluster_size: int = 0, kernel: int = 0, stream=None) -> None:
    """recsa_prefill_chunk: append [B][C][Hkv][128] K/V, extend the tree, attend the C queries causally."""
    for t in (k_new, v_new, q):
        assert t.dtype == torch.bfloat16 and t.is_contiguous()
    chunk = q.shape[1]
    dbg = _debug(sel_idx, sel_levels, cluster_size, entries, kernel)
    _check(_lib.recsa_prefill_chunk(ctypes.byref(p), ctypes.byref(tree.c), _ptr(k_new), _ptr(v_new), _ptr(q), chunk,
                                    _ptr(out), int(out.dtype == torch.float32), _ptr(ws.buf), ws.nbytes,
                                    ctypes.byref(dbg) if dbg is not None else None, _stream(stream)))


def decode_no_alloc(p: Params, tree: RecsaTree, q: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """recsa_decode_no_alloc: recsa_decode with its scratch in the library's fixed device array."""
    assert q.dtype == torch.bfloat16 and q.is_contiguous() and out.is_contiguous()
    _check(_lib.recsa_decode_no_alloc(ctypes.byref(p), ctypes.byref(tree.c), _ptr(q), q.shape[1], _ptr(out),
                                      int(out.dtype == torch.float32), _stream(stream)))


def check_device_errors(ws: Workspace, stream=None) -> None:
    _check(_lib.recsa_check_device_errors(_ptr(ws.buf), _stream(stream)))


# --------------------------------------------------------------------------- dense operators


DENSE_AUTO, DENSE_ROWS, DENSE_CHUNK = 0, 1, 2


class View(ctypes.Structure):
    """recsa_view: which tokens a dense query sees.

    window = 0 sees every token before the query; otherwise the last `window` tokens and the
    first `sinks`.  causal: the queries belong to the cache's last tokens (else all sit at its
    end); own_token: a causal query also sees its own token, from one position past it;
    at_token: it sees it and sits at its position (a query at the cache's end: at the last
    token's), as the layers of a causal RoPE model do.  token_positions: sinks outside the
    window are scored at their token positions instead of their rank among the visible.
    kernel: DENSE_AUTO, DENSE_ROWS or DENSE_CHUNK."""

    _fields_ = [
        ("sinks", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("sink_positions", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("own_token", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
    ]

    def __init__(self, sinks: int = 0, window: int = 0, causal: bool = False, own_token: bool = False,
                 token_positions: bool = False, kernel: int = 0, at_token: bool = False):
        super().__init__(sinks, window, int(token_positions), int(causal), 2 if at_token else int(own_token), kernel)


class TokenCache(RecsaTree):
    """Token caches without a tree, for layers that only run the dense operators (those also
    take a RecsaTree, whose tree they keep up to date)."""

    def __init__(self, p: Params, k_tok: torch.Tensor, v_tok: torch.Tensor, length: int,
                 seq_len: torch.Tensor | None = None, page_table: torch.Tensor | None = None):
        """Arguments as RecsaTree's."""
        none = torch.empty(0, dtype=torch.float32, device=k_tok.device)
        super().__init__(p, k_tok, v_tok, none, length, k_node=none, v_node=none, seq_len=seq_len,
                         page_table=page_table)
        self.k_node = self.v_node = self.pooler = None
        self.c.k_node = self.c.v_node = self.c.pooler = None


def dense_workspace_size(p: Params, batch: int, capacity: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.recsa_dense_workspace_size(ctypes.byref(p), batch, capacity, ctypes.byref(n)))
    return n.value


class DenseWorkspace:
    """Workspace of the dense operators on caches of `batch` sequences of up to `capacity`
    tokens.  Every call writes it: one per stream (or captured graph) that may overlap.  A
    buffer may be larger than dense_workspace_size(); nbytes is what it holds."""

    def __init__(self, p: Params, batch: int, capacity: int, device, stream=None, buffer: torch.Tensor | None = None):
        self.nbytes = dense_workspace_size(p, batch, capacity)
        self.buf = buffer if buffer is not None else torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        if buffer is not None:
            self.nbytes = buffer.numel() * buffer.element_size()
        if not self.buf.is_cuda:
            raise RecsaError(1, "the workspace is not on a CUDA device")
        _on_current_device(self.buf)
        _check(_lib.recsa_dense_workspace_init(ctypes.byref(p), batch, capacity, _ptr(self.buf),
                                               self.buf.numel() * self.buf.element_size(), _stream(stream)))


def _on_current_device(*tensors: torch.Tensor) -> None:
    """The library launches on the current device: every tensor has to be on it."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t.device.index != dev:
            raise RecsaError(1, f"a tensor on {t.device}, the current device is cuda:{dev}")


def _cache_here(p: Params, tree: RecsaTree, name: str = "the cache") -> None:
    """Every tensor of the cache is on the current device, and the cache has p's KV heads."""
    if tree.p.num_kv_heads != p.num_kv_heads:
        raise RecsaError(1, f"{name} has {tree.p.num_kv_heads} KV heads, params {p.num_kv_heads}")
    dev = torch.cuda.current_device()
    if len(tree.devices) != 1 or next(iter(tree.devices)).index != dev:
        raise RecsaError(1, f"{name}'s tensors are on {sorted(map(str, tree.devices))}, the current device is cuda:{dev}")


def _dense_rows(p: Params, tree: RecsaTree, t: torch.Tensor, heads: int, name: str, dtypes=(torch.bfloat16,)) -> None:
    """t is [batch][n][heads][128], contiguous, of one of the types."""
    if t.dtype not in dtypes:
        raise RecsaError(1, f"{name} is {t.dtype}")
    if t.dim() != 4 or t.shape[0] != tree.batch or t.shape[2] != heads or t.shape[3] != HEAD_DIM:
        raise RecsaError(1, f"{name} has shape {tuple(t.shape)}, not [{tree.batch}][n][{heads}][{HEAD_DIM}]")
    if not t.is_contiguous():
        raise RecsaError(1, f"{name} is not contiguous")


_OUT_TYPES = (torch.float32, torch.bfloat16)


def _dense_q(p: Params, tree: RecsaTree, q: torch.Tensor, out: torch.Tensor, ws: DenseWorkspace) -> None:
    _dense_rows(p, tree, q, p.num_q_heads, "q")
    _dense_rows(p, tree, out, p.num_q_heads, "out", _OUT_TYPES)
    if out.shape != q.shape:
        raise RecsaError(1, f"out has shape {tuple(out.shape)}, q {tuple(q.shape)}")
    _cache_here(p, tree)
    _on_current_device(q, out, ws.buf)


def _dense_new(p: Params, tree: RecsaTree, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor) -> None:
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        _dense_rows(p, tree, t, p.num_kv_heads, name)
        if t.shape[1] != q.shape[1]:
            raise RecsaError(1, f"{name} holds {t.shape[1]} tokens, q {q.shape[1]}")
        _on_current_device(t)


def _view(view: View | None):
    return None if view is None else ctypes.byref(view)


def dense_attend(p: Params, tree: RecsaTree, q: torch.Tensor, out: torch.Tensor, ws: DenseWorkspace,
                 view: View | None = None, stream=None) -> None:
    """recsa_dense_attend: q [B][n][Hq][128] bf16 over the cache's tokens -> out of the same
    shape (fp32 or bf16)."""
    _dense_q(p, tree, q, out, ws)
    _check(_lib.recsa_dense_attend(ctypes.byref(p), ctypes.byref(tree.c), _view(view), _ptr(q), q.shape[1], _ptr(out),
                                   int(out.dtype == torch.float32), _ptr(ws.buf), ws.nbytes, _stream(stream)))


def dense_prefill_chunk(p: Params, tree: RecsaTree, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                        out: torch.Tensor, ws: DenseWorkspace, view: View | None = None, stream=None) -> None:
    """recsa_dense_prefill_chunk: append [B][C][Hkv][128] K/V, attend the C queries causally."""
    _dense_q(p, tree, q, out, ws)
    _dense_new(p, tree, k_new, v_new, q)
    _check(_lib.recsa_dense_prefill_chunk(ctypes.byref(p), ctypes.byref(tree.c), _view(view), _ptr(k_new), _ptr(v_new),
                                          _ptr(q), q.shape[1], _ptr(out), int(out.dtype == torch.float32),
                                          _ptr(ws.buf), ws.nbytes, _stream(stream)))


def dense_decode_step(p: Params, tree: RecsaTree, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                      out: torch.Tensor, ws: DenseWorkspace, view: View | None = None, stream=None) -> None:
    """recsa_dense_decode_step: append one token per sequence at its device length, advance the
    lengths, attend the token's query; graph-capturable (needs tree.seq_len)."""
    _dense_q(p, tree, q, out, ws)
    _dense_new(p, tree, k_new, v_new, q)
    if q.shape[1] != 1:
        raise RecsaError(1, f"a decode step takes one token per sequence, not {q.shape[1]}")
    _check(_lib.recsa_dense_decode_step(ctypes.byref(p), ctypes.byref(tree.c), _view(view), _ptr(k_new), _ptr(v_new),
                                        _ptr(q), _ptr(out), int(out.dtype == torch.float32), _ptr(ws.buf), ws.nbytes,
                                        _stream(stream)))


def _weights_of(tree: RecsaTree, w: torch.Tensor, name: str) -> None:
    if w.dtype != torch.float32 or not w.is_contiguous() or tuple(w.shape) != (
            tree.batch, tree.p.num_kv_heads, tree.capacity):
        raise RecsaError(1, f"{name} is {w.dtype} {tuple(w.shape)}, not contiguous float32 "
                            f"[{tree.batch}][{tree.p.num_kv_heads}][{tree.capacity}]")
    _on_current_device(w)


def accumulate_weights(p: Params, tree: RecsaTree, q: torch.Tensor, weights: torch.Tensor, ws: DenseWorkspace,
                       view: View | None = None, accumulate: bool = True, stream=None) -> None:
    """recsa_accumulate_weights: the softmax weight each slot receives from q [B][n][Hq][128],
    summed over queries and group heads, into weights [B][Hkv][capacity] (fp32)."""
    _dense_rows(p, tree, q, p.num_q_heads, "q")
    _weights_of(tree, weights, "weights")
    _cache_here(p, tree)
    _on_current_device(q, ws.buf)
    _check(_lib.recsa_accumulate_weights(ctypes.byref(p), ctypes.byref(tree.c), _view(view), _ptr(q), q.shape[1],
                                         _ptr(weights), int(accumulate), _ptr(ws.buf), ws.nbytes, _stream(stream)))


def evict(p: Params, tree: RecsaTree, weights: torch.Tensor, keep: int, kept: torch.Tensor,
          into: RecsaTree | None = None, into_weights: torch.Tensor | None = None, sinks: int = 0, recent: int = 0,
          stream=None) -> None:
    """recsa_evict: cut every (sequence, KV head) to its `keep` heaviest slots, in place or into
    another cache; kept [B][Hkv][keep] int32 receives the kept slots, into_weights their weights
    (in place, 0 in the slots given up; beside another cache the slots past the kept ones are
    left as they are: clear a buffer that was used before)."""
    _weights_of(tree, weights, "weights")
    if kept.dtype != torch.int32 or not kept.is_contiguous() or tuple(kept.shape) != (tree.batch, p.num_kv_heads, keep):
        raise RecsaError(1, f"kept is {kept.dtype} {tuple(kept.shape)}, not contiguous int32 "
                            f"[{tree.batch}][{p.num_kv_heads}][{keep}]")
    if into_weights is not None:
        _weights_of(tree if into is None else into, into_weights, "into_weights")
    _cache_here(p, tree)
    if into is not None:
        _cache_here(p, into, "into")
    _on_current_device(kept)
    _check(_lib.recsa_evict(ctypes.byref(p), ctypes.byref(tree.c), _ptr(weights), keep, sinks, recent, _ptr(kept),
                            None if into is None else ctypes.byref(into.c), _ptr(into_weights), _stream(stream)))


def status_string(code: int) -> str:
    return _lib.recsa_status_string(code).decode()


def last_error() -> str:
    return _lib.recsa_last_error().decode()


def raw_library() -> ctypes.CDLL:
    """The loaded CDLL (for callers that marshal their own arguments)."""
    return _lib
