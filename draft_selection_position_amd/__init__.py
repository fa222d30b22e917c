"""DFlash 2 draft-path selector for AMD Instinct MI355X (gfx950).

Thin Python binding of ``libdfs.so`` (C ABI declared in ``include/dfs.h``).  It
only checks and marshals arguments: every step of the selector runs in the
library's HIP kernels.  PyTorch supplies device memory and the current stream.
The library is required; there is no other code path.

    import draft_selection_position_amd as dfs
    path, scores = dfs.select(logits, hidden, prev_token, A, B, W_h)

The selector (blog post "DFlash 2: Keep Drafting Parallel", section "A
Lightweight Path Selector"): keep the 16 best candidates per block position,
score every adjacent pair with S_t(a,b) = U_t(b) + <A(a) * sigmoid(h_t W_h), B(b)>,
then walk the scores once from the last verified token.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

__all__ = [
    "DfsError", "K", "E", "MAX_L", "lib", "lib_path", "topk", "gate", "pair_scores", "walk",
    "select", "Selector", "select_workspace_bytes", "topk_workspace_bytes", "PackedWeight", "gate_pack",
    "gate_workspace_bytes", "status_str", "conv2", "conv2_workspace_bytes", "Conv2", "lmhead_topk", "lmhead_logits",
    "lmhead_topk_workspace_bytes", "norm_q8", "linear_q8", "linear_q8_workspace_bytes", "tree_attention",
    "tree_attention_workspace_bytes", "cache_commit", "tree_positions", "rope_frequencies", "rope", "cache_append",
    "tree_attention_shared", "tree_attention_shared_workspace_bytes",
]

K = 16
E = 256
MAX_L = 16
F32, BF16 = 0, 1
GREEDY, GUMBEL, VITERBI = 0, 1, 2
_MODES = {"greedy": GREEDY, "gumbel": GUMBEL, "sampled": GUMBEL, "viterbi": VITERBI}

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None
_lock = threading.Lock()


def lib_path() -> str:
    """libdfs.so next to this file, or the build that DFS_LIBRARY names (another build of the
    same sources, e.g. the host-sanitized one the ABI tests run against)."""
    return os.environ.get("DFS_LIBRARY") or os.path.join(_HERE, "libdfs.so")


class _Shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("L", ctypes.c_int64), ("V", ctypes.c_int64),
                ("d", ctypes.c_int64), ("logits_dtype", ctypes.c_int), ("act_dtype", ctypes.c_int),
                ("table_dtype", ctypes.c_int)]


class _CacheShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "T", "q_heads", "kv_heads", "head_dim", "page_size",
                                              "n_pages", "table_width")] + [("dtype", ctypes.c_int)]


class _RopeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "q_heads", "kv_heads", "head_dim", "rot_dim", "q_stride",
                                              "k_stride", "v_stride")] + [
        ("amplitude", ctypes.c_double), ("layout", ctypes.c_int), ("dtype", ctypes.c_int)]


def lib() -> ctypes.CDLL:
    """Load libdfs.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m draft_selection_position_amd.build`")
        L = ctypes.CDLL(path)
        vp, i64, sz, i32p, f32p = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p
        c_int, c_double, u64 = ctypes.c_int, ctypes.c_double, ctypes.c_uint64
        L.dfs_status_str.argtypes, L.dfs_status_str.restype = [c_int], ctypes.c_char_p
        L.dfs_abi_version.argtypes, L.dfs_abi_version.restype = [], c_int
        L.dfs_topk_workspace_bytes.argtypes, L.dfs_topk_workspace_bytes.restype = [i64, i64, c_int], sz
        L.dfs_topk.argtypes = [vp, c_int, i64, i64, c_int, i32p, f32p, vp, sz, vp]
        L.dfs_topk.restype = c_int
        L.dfs_gate_workspace_bytes.argtypes, L.dfs_gate_workspace_bytes.restype = [i64, i64, c_int], sz
        L.dfs_gate.argtypes = [vp, vp, c_int, i64, i64, i64, f32p, vp, sz, vp]
        L.dfs_gate.restype = c_int
        L.dfs_gate_packed.argtypes = [vp, vp, c_int, i64, i64, i64, f32p, vp, sz, vp]
        L.dfs_gate_packed.restype = c_int
        L.dfs_gate_pack_bytes.argtypes, L.dfs_gate_pack_bytes.restype = [i64, c_int], sz
        L.dfs_gate_pack.argtypes = [vp, c_int, i64, vp, sz, vp]
        L.dfs_gate_pack.restype = c_int
        L.dfs_pair_scores.argtypes = [i32p, f32p, i32p, f32p, vp, vp, c_int, i64, i64, i64, i64, c_int,
                                      f32p, vp]
        L.dfs_pair_scores.restype = c_int
        L.dfs_walk.argtypes = [f32p, i32p, i64, i64, c_int, c_int, c_double, u64, i32p, f32p, vp]
        L.dfs_walk.restype = c_int
        L.dfs_select_workspace_bytes.argtypes = [ctypes.POINTER(_Shape)]
        L.dfs_select_workspace_bytes.restype = sz
        L.dfs_select.argtypes = [vp, vp, i32p, vp, vp, vp, c_int, ctypes.POINTER(_Shape), c_int, c_double,
                                 u64, vp, sz, i32p, f32p, vp]
        L.dfs_select.restype = c_int
        L.dfs_select_packed.argtypes = L.dfs_select.argtypes
        L.dfs_select_packed.restype = c_int
        L.dfs_select_packed_static.argtypes = [vp, vp, i32p, vp, vp, vp, c_int, ctypes.POINTER(_Shape), c_int,
                                               c_double, u64, i32p, f32p, vp]
        L.dfs_select_packed_static.restype = c_int
        L.dfs_select_draft.argtypes = [vp, vp, i32p, vp, vp, vp, c_int, ctypes.POINTER(_Shape), c_int,
                                       c_double, u64, vp, sz, i32p, f32p, f32p, i32p, vp]
        L.dfs_select_draft.restype = c_int
        L.dfs_select_draft_packed.argtypes = L.dfs_select_draft.argtypes
        L.dfs_select_draft_packed.restype = c_int
        L.dfs_verify_workspace_bytes.argtypes, L.dfs_verify_workspace_bytes.restype = [i64, i64, i64, c_int], sz
        L.dfs_verify.argtypes = [vp, c_int, i64, i64, i64, i32p, i32p, f32p, c_int, c_double, u64, vp, sz,
                                 i32p, i32p, vp]
        L.dfs_verify.restype = c_int
        L.dfs_conv2_workspace_bytes.argtypes, L.dfs_conv2_workspace_bytes.restype = [i64, i64, i64, c_int], sz
        L.dfs_conv2.argtypes = [vp, vp, vp, vp, c_int, i64, i64, i64, vp, vp, sz, vp]
        L.dfs_conv2.restype = c_int
        L.dfs_lmhead_topk_workspace_bytes.argtypes = [i64, i64, i64]
        L.dfs_lmhead_topk_workspace_bytes.restype = sz
        L.dfs_lmhead_topk.argtypes = [vp, vp, c_int, i64, i64, i64, c_int, i32p, f32p, vp, sz, vp]
        L.dfs_lmhead_topk.restype = c_int
        L.dfs_lmhead_logits.argtypes = [vp, vp, c_int, i64, i64, i64, f32p, vp]
        L.dfs_lmhead_logits.restype = c_int
        L.dfs_norm_q8.argtypes = [vp, vp, vp, c_int, i64, i64, c_double, vp, f32p, vp, vp, vp]
        L.dfs_norm_q8.restype = c_int
        L.dfs_linear_q8_workspace_bytes.argtypes, L.dfs_linear_q8_workspace_bytes.restype = [i64, i64, i64], sz
        L.dfs_linear_q8.argtypes = [vp, f32p, vp, f32p, i64, i64, i64, c_int, vp, vp, sz, vp]
        L.dfs_linear_q8.restype = c_int
        cache = ctypes.POINTER(_CacheShape)
        L.dfs_tree_attention_workspace_bytes.argtypes = [cache]
        L.dfs_tree_attention_workspace_bytes.restype = sz
        L.dfs_tree_attention.argtypes = [vp, vp, vp, i32p, vp, vp, i32p, i32p, cache, c_double, vp, vp, sz, vp]
        L.dfs_tree_attention.restype = c_int
        L.dfs_cache_commit.argtypes = [vp, vp, i32p, i32p, i64, vp, vp, i32p, i32p, cache, i32p, vp]
        L.dfs_cache_commit.restype = c_int
        L.dfs_tree_positions.argtypes = [i32p, i32p, i32p, i64, i64, i32p, vp]
        L.dfs_tree_positions.restype = c_int
        L.dfs_rope_frequencies.argtypes = [i64, c_double, c_int, c_double, c_double, c_double, c_double, vp, vp]
        L.dfs_rope_frequencies.restype = c_int
        rope = ctypes.POINTER(_RopeShape)
        L.dfs_rope.argtypes = [vp, vp, vp, i32p, f32p, rope, vp, vp, vp, vp]
        L.dfs_rope.restype = c_int
        L.dfs_cache_append.argtypes = [vp, vp, vp, i32p, f32p, rope, i32p, vp, vp, vp, i32p, i32p, cache, i32p, vp]
        L.dfs_cache_append.restype = c_int
        L.dfs_tree_attention_shared_workspace_bytes.argtypes = [cache, i64]
        L.dfs_tree_attention_shared_workspace_bytes.restype = sz
        L.dfs_tree_attention_shared.argtypes = [vp, vp, vp, i32p, vp, vp, i32p, i32p, i64, i32p, i32p, cache, c_double,
                                                vp, vp, sz, vp]
        L.dfs_tree_attention_shared.restype = c_int
        _lib = L
    return _lib


class DfsError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_str(code)}")


def status_str(code: int) -> str:
    return lib().dfs_status_str(int(code)).decode()


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise DfsError(rc, where)


def _dtype_code(t: torch.Tensor, what: str) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"{what} must be float32 or bfloat16, got {t.dtype}")


def _dev(t: torch.Tensor, what: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what} must be on a HIP device, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    return t


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


class _Workspace:
    """Cached scratch buffers, one per (device, stream), grown on demand, never shrunk.

    A call without an explicit workspace uses the buffer of the stream it is enqueued
    on, so calls on different streams never share scratch memory.  Each buffer is
    allocated while its own stream is current, so when a grown buffer replaces it, the
    caching allocator hands the old block out again only to later work on that same
    stream (after everything already enqueued there).
    """

    def __init__(self):
        self._bufs: dict[tuple, torch.Tensor] = {}

    @staticmethod
    def key(device: torch.device) -> tuple:
        return (device, torch.cuda.current_stream(device).cuda_stream)

    def get(self, device: torch.device, nbytes: int) -> torch.Tensor | None:
        if nbytes == 0:
            return None
        key = self.key(device)
        buf = self._bufs.get(key)
        if buf is None or buf.numel() < nbytes:
            with torch.cuda.device(device):
                buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
            self._bufs[key] = buf
        return buf


_WS = _Workspace()


def _ws_arg(ws, device, nbytes):
    if ws is None:
        ws = _WS.get(device, nbytes)
    elif nbytes and (ws.device != device or ws.numel() * ws.element_size() < nbytes):
        raise ValueError(f"workspace must hold {nbytes} bytes on {device}")
    return ws


# ---------------------------------------------------------------- step entry points


def topk_workspace_bytes(rows: int, V: int, dtype: torch.dtype) -> int:
    return int(lib().dfs_topk_workspace_bytes(rows, V, BF16 if dtype == torch.bfloat16 else F32))


def topk(logits: torch.Tensor, k: int = K, workspace: torch.Tensor | None = None):
    """Top-16 of each row of ``logits`` [..., V]: (ids int32 [..., 16], values fp32 [..., 16]).

    Order: value descending, then id ascending.
    """
    _dev(logits, "logits")
    dt = _dtype_code(logits, "logits")
    V = logits.shape[-1]
    rows = logits.numel() // V if V else 0
    lead = tuple(logits.shape[:-1])
    idx = torch.empty(lead + (K,), dtype=torch.int32, device=logits.device)
    val = torch.empty(lead + (K,), dtype=torch.float32, device=logits.device)
    nb = int(lib().dfs_topk_workspace_bytes(rows, V, dt))
    ws = _ws_arg(workspace, logits.device, nb)
    _check(lib().dfs_topk(logits.data_ptr(), dt, rows, V, k, idx.data_ptr(), val.data_ptr(), _ptr(ws), nb,
                          _stream(logits.device)), "dfs_topk")
    return idx, val


def gate_workspace_bytes(rows: int, d: int, dtype: torch.dtype) -> int:
    return int(lib().dfs_gate_workspace_bytes(rows, d, BF16 if dtype == torch.bfloat16 else F32))


class PackedWeight:
    """W_h [d, 256] packed once for the gate's matrix cores (dfs_gate_pack).

    Pass it wherever W_h is taken (``gate``, ``select``, ``Selector``): the results are
    bitwise those of the unpacked weight, without repacking it on every call.  It holds
    its own device bytes; ``d`` and ``dtype`` are those of the weight it came from.
    """

    def __init__(self, data: torch.Tensor, d: int, dtype: torch.dtype):
        self.data, self.d, self.dtype = data, int(d), dtype
        self.device = data.device
        self.shape = (int(d), E)

    def data_ptr(self) -> int:
        return self.data.data_ptr()


def gate_pack(W_h: torch.Tensor) -> PackedWeight:
    """Pack the gate weight W_h [d, 256] (bf16 or fp32) for the matrix cores, once."""
    _dev(W_h, "W_h")
    dt = _dtype_code(W_h, "W_h")
    if W_h.dim() != 2 or W_h.shape[1] != E:
        raise ValueError(f"W_h must be [d, 256], got {tuple(W_h.shape)}")
    d = W_h.shape[0]
    nb = int(lib().dfs_gate_pack_bytes(d, dt))
    if nb == 0:
        raise ValueError(f"unsupported gate width d = {d}")
    out = torch.empty(nb, dtype=torch.uint8, device=W_h.device)
    _check(lib().dfs_gate_pack(W_h.data_ptr(), dt, d, out.data_ptr(), nb, _stream(W_h.device)), "dfs_gate_pack")
    return PackedWeight(out, d, W_h.dtype)


def _weight(W_h, d: int, dtype: torch.dtype, what: str = "W_h"):
    """(pointer, packed?) of a W_h argument: a [d, 256] tensor of `dtype` or a PackedWeight."""
    if isinstance(W_h, PackedWeight):
        if W_h.d != d or W_h.dtype != dtype:
            raise ValueError(f"{what} was packed for d = {W_h.d}, {W_h.dtype}; need d = {d}, {dtype}")
        if W_h.device.type != "cuda":
            raise ValueError(f"{what} must be on a HIP device")
        return W_h.data_ptr(), True
    _dev(W_h, what, dtype)
    if W_h.dim() != 2 or tuple(W_h.shape) != (d, E):
        raise ValueError(f"{what} must be [{d}, 256], got {tuple(W_h.shape)}")
    return W_h.data_ptr(), False


def gate(hidden: torch.Tensor, W_h, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """sigmoid(hidden @ W_h) in fp32: hidden [..., d], W_h [d, 256] (same dtype, or a
    PackedWeight) -> [..., 256]."""
    _dev(hidden, "hidden")
    dt = _dtype_code(hidden, "hidden")
    d = hidden.shape[-1]
    wptr, packed = _weight(W_h, d, hidden.dtype)
    rows = hidden.numel() // d if d else 0
    out = torch.empty(tuple(hidden.shape[:-1]) + (E,), dtype=torch.float32, device=hidden.device)
    nb = int(lib().dfs_gate_workspace_bytes(rows, d, dt))
    ws = _ws_arg(workspace, hidden.device, nb)
    fn = lib().dfs_gate_packed if packed else lib().dfs_gate
    _check(fn(hidden.data_ptr(), wptr, dt, rows, d, E, out.data_ptr(), _ptr(ws), nb, _stream(hidden.device)),
           "dfs_gate_packed" if packed else "dfs_gate")
    return out


def pair_scores(cand_idx: torch.Tensor, cand_val: torch.Tensor, prev_token: torch.Tensor,
                gate_: torch.Tensor, A: torch.Tensor, B: torch.Tensor) -> torch.Tensor:
    """S[b, t, i, j] for all adjacent candidate pairs: fp32 [batch, L, 16, 16]."""
    _dev(cand_idx, "cand_idx", torch.int32)
    _dev(cand_val, "cand_val", torch.float32)
    _dev(prev_token, "prev_token", torch.int32)
    _dev(gate_, "gate", torch.float32)
    _dev(A, "A")
    _dev(B, "B", A.dtype)
    if cand_idx.dim() != 3 or cand_idx.shape[-1] != K or cand_val.shape != cand_idx.shape:
        raise ValueError("cand_idx and cand_val must both be [batch, L, 16]")
    batch, L = cand_idx.shape[0], cand_idx.shape[1]
    if prev_token.shape != (batch,) or gate_.numel() != batch * L * E:
        raise ValueError("prev_token must be [batch] and gate [batch*L, 256]")
    if A.dim() != 2 or A.shape != B.shape:
        raise ValueError("A and B must both be [V, 256]")
    out = torch.empty((batch, L, K, K), dtype=torch.float32, device=cand_idx.device)
    _check(lib().dfs_pair_scores(cand_idx.data_ptr(), cand_val.data_ptr(), prev_token.data_ptr(),
                                 gate_.data_ptr(), A.data_ptr(), B.data_ptr(), _dtype_code(A, "A"), batch, L,
                                 A.shape[0], A.shape[1], K, out.data_ptr(), _stream(A.device)),
           "dfs_pair_scores")
    return out


def walk(pair: torch.Tensor, cand_idx: torch.Tensor, mode: str = "greedy", temperature: float = 1.0,
         seed: int = 0):
    """One walk per sequence over pair [batch, L, 16, 16]: (path int32 [batch, L], scores fp32)."""
    _dev(pair, "pair", torch.float32)
    _dev(cand_idx, "cand_idx", torch.int32)
    if pair.dim() != 4 or pair.shape[2:] != (K, K) or cand_idx.shape != pair.shape[:3]:
        raise ValueError("pair must be [batch, L, 16, 16] and cand_idx [batch, L, 16]")
    batch, L = pair.shape[0], pair.shape[1]
    path = torch.empty((batch, L), dtype=torch.int32, device=pair.device)
    scores = torch.empty((batch, L), dtype=torch.float32, device=pair.device)
    _check(lib().dfs_walk(pair.data_ptr(), cand_idx.data_ptr(), batch, L, K, _MODES[mode], float(temperature),
                          int(seed) & (2**64 - 1), path.data_ptr(), scores.data_ptr(), _stream(pair.device)),
           "dfs_walk")
    return path, scores


# ---------------------------------------------------------------- fused selector


def _shape(batch, L, V, d, logits_dt, act_dt, table_dt) -> _Shape:
    return _Shape(batch, L, V, d, logits_dt, act_dt, table_dt)


def select_workspace_bytes(batch: int, L: int, V: int, d: int, logits_dtype=torch.bfloat16,
                           act_dtype=torch.bfloat16, table_dtype=torch.bfloat16) -> int:
    c = lambda t: BF16 if t == torch.bfloat16 else F32  # noqa: E731
    s = _shape(batch, L, V, d, c(logits_dtype), c(act_dtype), c(table_dtype))
    return int(lib().dfs_select_workspace_bytes(ctypes.byref(s)))


def select(logits: torch.Tensor, hidden: torch.Tensor, prev_token: torch.Tensor, A: torch.Tensor,
           B: torch.Tensor, W_h, k: int = K, mode: str = "greedy", temperature: float = 1.0,
           seed: int = 0, workspace: torch.Tensor | None = None, out=None, draft: bool = False):
    """The whole selector on one draft block per sequence.

    logits [batch, L, V]; hidden [batch, L, d]; prev_token [batch] int32 (last
    verified token); A, B [V, 256]; W_h [d, 256] or a PackedWeight (gate_pack).
    Returns (path int32 [batch, L], scores fp32 [batch, L]).  ``out`` may pass
    preallocated (path, scores).  With ``draft=True`` also the draft distributions q
    fp32 [batch, L, 16] and the candidate ids int32 [batch, L, 16] (dfs_select_draft).
    """
    _dev(logits, "logits")
    _dev(hidden, "hidden")
    _dev(prev_token, "prev_token", torch.int32)
    _dev(A, "A")
    _dev(B, "B", A.dtype)
    if logits.dim() != 3 or hidden.dim() != 3 or hidden.shape[:2] != logits.shape[:2]:
        raise ValueError("logits must be [batch, L, V] and hidden [batch, L, d]")
    batch, L, V = logits.shape
    d = hidden.shape[2]
    wptr, packed = _weight(W_h, d, hidden.dtype)
    if A.shape != (V, E) or B.shape != (V, E) or prev_token.shape != (batch,):
        raise ValueError("A, B must be [V, 256] and prev_token [batch]")
    s = _shape(batch, L, V, d, _dtype_code(logits, "logits"), _dtype_code(hidden, "hidden"),
               _dtype_code(A, "A"))
    nb = int(lib().dfs_select_workspace_bytes(ctypes.byref(s)))
    ws = _ws_arg(workspace, logits.device, nb)
    if out is None:
        path = torch.empty((batch, L), dtype=torch.int32, device=logits.device)
        scores = torch.empty((batch, L), dtype=torch.float32, device=logits.device)
    else:
        path, scores = out
    if not draft:
        fn = lib().dfs_select_packed if packed else lib().dfs_select
        _check(fn(logits.data_ptr(), hidden.data_ptr(), prev_token.data_ptr(), A.data_ptr(), B.data_ptr(), wptr,
                  k, ctypes.byref(s), _MODES[mode], float(temperature), int(seed) & (2**64 - 1), _ptr(ws), nb,
                  path.data_ptr(), scores.data_ptr(), _stream(logits.device)),
               "dfs_select_packed" if packed else "dfs_select")
        return path, scores
    q = torch.empty((batch, L, K), dtype=torch.float32, device=logits.device)
    cand = torch.empty((batch, L, K), dtype=torch.int32, device=logits.device)
    fn = lib().dfs_select_draft_packed if packed else lib().dfs_select_draft
    _check(fn(logits.data_ptr(), hidden.data_ptr(), prev_token.data_ptr(), A.data_ptr(), B.data_ptr(), wptr, k,
              ctypes.byref(s), _MODES[mode], float(temperature), int(seed) & (2**64 - 1), _ptr(ws), nb,
              path.data_ptr(), scores.data_ptr(), q.data_ptr(), cand.data_ptr(), _stream(logits.device)),
           "dfs_select_draft_packed" if packed else "dfs_select_draft")
    return path, scores, q, cand


def verify_workspace_bytes(batch: int, L: int, V: int, dtype: torch.dtype) -> int:
    code = F32 if dtype == torch.float32 else BF16 if dtype == torch.bfloat16 else -1
    return int(lib().dfs_verify_workspace_bytes(batch, L, V, code))


def verify(target_logits: torch.Tensor, path: torch.Tensor, cand: torch.Tensor, q: torch.Tensor,
           temperature: float = 1.0, seed: int = 0, workspace: torch.Tensor | None = None):
    """Speculative-sampling verification of drafted blocks (see dfs_verify).

    target_logits [batch, L + 1, V]; path [batch, L] int32; cand [batch, L, 16] int32 and
    q [batch, L, 16] fp32 (``select(..., draft=True)``).  Returns (accepted int32 [batch],
    token int32 [batch]): the number of draft tokens kept and the token drawn after them.
    """
    _dev(target_logits, "target_logits")
    _dev(path, "path", torch.int32)
    _dev(cand, "cand", torch.int32)
    _dev(q, "q", torch.float32)
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [batch, L + 1, V]")
    batch, L1, V = target_logits.shape
    L = L1 - 1
    if path.shape != (batch, L) or cand.shape != (batch, L, K) or q.shape != (batch, L, K):
        raise ValueError("path must be [batch, L], cand and q [batch, L, 16] with L + 1 target rows")
    dt = _dtype_code(target_logits, "target_logits")
    nb = int(lib().dfs_verify_workspace_bytes(batch, L, V, dt))
    ws = _ws_arg(workspace, target_logits.device, nb)
    accepted = torch.empty(batch, dtype=torch.int32, device=target_logits.device)
    token = torch.empty(batch, dtype=torch.int32, device=target_logits.device)
    _check(lib().dfs_verify(target_logits.data_ptr(), dt, batch, L, V, path.data_ptr(), cand.data_ptr(),
                            q.data_ptr(), K, float(temperature), int(seed) & (2**64 - 1), _ptr(ws), nb,
                            accepted.data_ptr(), token.data_ptr(), _stream(target_logits.device)), "dfs_verify")
    return accepted, token


def conv2_workspace_bytes(batch: int, L: int, D: int, dtype: torch.dtype) -> int:
    code = F32 if dtype == torch.float32 else BF16 if dtype == torch.bfloat16 else -1
    return int(lib().dfs_conv2_workspace_bytes(batch, L, D, code))


def conv2(x: torch.Tensor, x_prev: torch.Tensor, base: torch.Tensor, W_c: torch.Tensor,
          out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Two-tap dynamic depthwise convolution across block positions (see dfs_conv2).

    x [batch, L, D], x_prev [batch, D], base [2, D], W_c [D/16, 2, D], all of one dtype
    (bf16 or fp32).  Returns y [batch, L, D] (written into ``out`` when given)."""
    _dev(x, "x")
    dt = _dtype_code(x, "x")
    _dev(x_prev, "x_prev", x.dtype)
    _dev(base, "base", x.dtype)
    _dev(W_c, "W_c", x.dtype)
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, D]")
    batch, L, D = x.shape
    if x_prev.shape != (batch, D) or base.shape != (2, D) or W_c.shape != (D // 16, 2, D):
        raise ValueError(f"x_prev must be [{batch}, {D}], base [2, {D}] and W_c [{D // 16}, 2, {D}]")
    if out is None:
        out = torch.empty_like(x)
    else:
        _dev(out, "out", x.dtype)
        if out.shape != x.shape:
            raise ValueError("out must have the shape of x")
    nb = int(lib().dfs_conv2_workspace_bytes(batch, L, D, dt))
    ws = _ws_arg(workspace, x.device, nb)
    _check(lib().dfs_conv2(x.data_ptr(), x_prev.data_ptr(), base.data_ptr(), W_c.data_ptr(), dt, batch, L, D,
                           out.data_ptr(), _ptr(ws), nb, _stream(x.device)), "dfs_conv2")
    return out


def _lmhead_args(hidden, W_lm):
    _dev(hidden, "hidden", torch.bfloat16)
    _dev(W_lm, "W_lm", torch.bfloat16)
    d = hidden.shape[-1]
    if W_lm.dim() != 2 or W_lm.shape[1] != d:
        raise ValueError(f"W_lm must be [V, {d}], got {tuple(W_lm.shape)}")
    return hidden.numel() // d, W_lm.shape[0], d


def lmhead_topk_workspace_bytes(rows: int, V: int, d: int) -> int:
    return int(lib().dfs_lmhead_topk_workspace_bytes(rows, V, d))


def lmhead_topk(hidden: torch.Tensor, W_lm: torch.Tensor, workspace: torch.Tensor | None = None):
    """Top-16 of U = hidden @ W_lm.T per row without writing U (see dfs_lmhead_topk).

    hidden [..., d] and W_lm [V, d], bf16.  Returns (ids int32 [..., 16], values fp32 [..., 16])."""
    rows, V, d = _lmhead_args(hidden, W_lm)
    lead = tuple(hidden.shape[:-1])
    idx = torch.empty(lead + (K,), dtype=torch.int32, device=hidden.device)
    val = torch.empty(lead + (K,), dtype=torch.float32, device=hidden.device)
    nb = lmhead_topk_workspace_bytes(rows, V, d)
    ws = _ws_arg(workspace, hidden.device, nb)
    _check(lib().dfs_lmhead_topk(hidden.data_ptr(), W_lm.data_ptr(), BF16, rows, V, d, K, idx.data_ptr(),
                                 val.data_ptr(), _ptr(ws), nb, _stream(hidden.device)), "dfs_lmhead_topk")
    return idx, val


def lmhead_logits(hidden: torch.Tensor, W_lm: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """U = hidden @ W_lm.T in fp32 by the same product as lmhead_topk: [..., V]."""
    rows, V, d = _lmhead_args(hidden, W_lm)
    if out is None:
        out = torch.empty(tuple(hidden.shape[:-1]) + (V,), dtype=torch.float32, device=hidden.device)
    _dev(out, "out", torch.float32)
    _check(lib().dfs_lmhead_logits(hidden.data_ptr(), W_lm.data_ptr(), BF16, rows, V, d, out.data_ptr(),
                                   _stream(hidden.device)), "dfs_lmhead_logits")
    return out


# ---------------------------------------------------------------- verification pass
#
# These calls are short where few rows are decoded (a few microseconds on the GPU), so what is
# checked on every call is one attribute each; the words for a refusal are found afterwards.

_CODES = {torch.float32: F32, torch.bfloat16: BF16}


def _fits(t, dtype, index: int) -> bool:
    """Whether t is a contiguous tensor of dtype on HIP device `index`."""
    return (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.get_device() == index
            and t.is_contiguous())


def _refuse(first: str, tensors: dict, dtypes: dict) -> None:
    """Raises for the first of the named tensors that does not fit: a HIP device, contiguous, its dtype, and
    the first one's device.  None of them is optional."""
    device = None
    for what, t in tensors.items():
        _dev(t, what, dtypes.get(what))
        if what == first:
            device = t.device
    for what, t in tensors.items():
        if t.device != device:
            raise ValueError(f"{what} must be on {device}, got {t.device}")


def _call(index: int, where: str, fn, *args) -> None:
    """fn(*args, stream) on HIP device `index` and its current stream."""
    stream = torch._C._cuda_getCurrentRawStream(index)  # looked up here: a CPU build of torch has no such name
    if index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != 0:
        raise DfsError(rc, where)


def _scratch(workspace, like: torch.Tensor, nbytes: int):
    """The workspace of a call: the caller's, or a new block of the current stream's (a graph's own under capture)."""
    if nbytes == 0:
        return None
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    _dev(workspace, "workspace")
    return _ws_arg(workspace, like.device, nbytes)


def norm_q8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
            normed: bool = False, total_out: torch.Tensor | None = None):
    """Root-mean-square norm of x + residual with an e4m3 output (see dfs_norm_q8).

    x, residual [..., d] and weight [d], all bf16 or all fp32.  Returns (q e4m3 [..., d], scale fp32
    [ceil(d / 128), rows]), then with a residual the sum in x's dtype (written into ``total_out`` when
    given, which may be ``x`` or ``residual`` itself), then with ``normed=True`` the norm in x's dtype."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _CODES:
        _dev(x, "x")
        _dtype_code(x, "x")
    dtype, index = x.dtype, x.get_device()
    if not (_fits(x, dtype, index) and _fits(weight, dtype, index)
            and (residual is None or _fits(residual, dtype, index))
            and (total_out is None or _fits(total_out, dtype, index))):
        given = {"x": x, "weight": weight, "residual": residual, "total_out": total_out}
        given = {k: t for k, t in given.items() if k in ("x", "weight") or t is not None}
        _refuse("x", given, dict.fromkeys(given, dtype))
    shape = x.shape
    if not shape or weight.shape != shape[-1:]:
        raise ValueError("x must be [..., d] and weight [d]")
    if residual is not None:
        if residual.shape != shape:
            raise ValueError("residual must have the shape of x")
        if total_out is None:
            total_out = torch.empty_like(x)
        elif total_out.shape != shape:
            raise ValueError("total_out must have the shape of x")
    elif total_out is not None:
        raise ValueError("total_out needs a residual")
    d = shape[-1]
    rows = x.numel() // d if d else 0
    q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    scale = x.new_empty((-(-d // 128), rows), dtype=torch.float32)
    y = torch.empty_like(x) if normed else None
    _call(index, "dfs_norm_q8", lib().dfs_norm_q8, x.data_ptr(), _ptr(residual), weight.data_ptr(), _CODES[dtype], rows,
          d, eps, q.data_ptr(), scale.data_ptr(), _ptr(total_out), _ptr(y))
    if residual is None:
        return (q, scale, y) if normed else (q, scale)
    return (q, scale, total_out, y) if normed else (q, scale, total_out)


def linear_q8_workspace_bytes(rows: int, N: int, K: int) -> int:
    return int(lib().dfs_linear_q8_workspace_bytes(rows, N, K))


def linear_q8(q: torch.Tensor, scale: torch.Tensor, W: torch.Tensor, W_scale: torch.Tensor,
              out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The product of e4m3 operands with a scale for each block of 128 (see dfs_linear_q8): [..., N].

    q [..., K] e4m3 with scale [ceil(K / 128), rows] fp32 (``norm_q8``'s); W [N, K] e4m3 with W_scale
    [ceil(N / 128), ceil(K / 128)] fp32.  ``out_dtype`` bf16 or fp32.  With bf16 and more than 16 rows sums may be
    off by 2^-10 of their products' magnitudes, which shows where large ones cancel; never with fp32.
    ``workspace`` is not used: no size needs any."""
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    index = q.get_device() if isinstance(q, torch.Tensor) else -1
    if not (_fits(q, e4m3, index) and _fits(scale, f32, index) and _fits(W, e4m3, index)
            and _fits(W_scale, f32, index) and (out is None or _fits(out, out_dtype, index))):
        given = {"q": q, "scale": scale, "W": W, "W_scale": W_scale} | ({} if out is None else {"out": out})
        _refuse("q", given, {"q": e4m3, "scale": f32, "W": e4m3, "W_scale": f32, "out": out_dtype})
    if out_dtype not in _CODES:
        raise ValueError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    shape = q.shape
    if not shape or W.dim() != 2 or W.shape[1] != shape[-1]:
        raise ValueError("q must be [..., K] and W [N, K]")
    N, K = W.shape
    rows = q.numel() // K if K else 0
    G = -(-K // 128)
    if scale.shape != (G, rows) or W_scale.shape != (-(-N // 128), G):
        raise ValueError(f"scale must be [{G}, {rows}] and W_scale [{-(-N // 128)}, {G}]")
    if out is None:
        out = scale.new_empty(shape[:-1] + (N,), dtype=out_dtype)
    elif out.shape != shape[:-1] + (N,):
        raise ValueError("out must be [..., N]")
    _call(index, "dfs_linear_q8", lib().dfs_linear_q8, q.data_ptr(), scale.data_ptr(), W.data_ptr(), W_scale.data_ptr(),
          rows, N, K, _CODES[out_dtype], out.data_ptr(), None, 0)
    return out


@functools.lru_cache(maxsize=1024)
def _cache_shape(batch, T, q_heads, kv_heads, head_dim, page_size, n_pages, table_width, dt):
    """A call's sizes as the library takes them (a reference that is read during calls only), and the bytes
    of scratch that attention over them needs."""
    s = _CacheShape(batch, T, q_heads, kv_heads, head_dim, page_size, n_pages, table_width, dt)
    return ctypes.byref(s), int(lib().dfs_tree_attention_workspace_bytes(ctypes.byref(s)))


def _cache_sizes(k_new, v_new, k_pages, v_pages, block_table, lens, index):
    """(batch, T, kv_heads, head_dim, page_size, n_pages, table_width, dtype code) of a call on a paged cache."""
    dtype, i32 = k_new.dtype, torch.int32
    if not (dtype in _CODES and _fits(k_new, dtype, index) and _fits(v_new, dtype, index)
            and _fits(k_pages, dtype, index) and _fits(v_pages, dtype, index) and _fits(block_table, i32, index)
            and _fits(lens, i32, index)):
        _dev(k_new, "k_new")
        _dtype_code(k_new, "k_new")
        given = {"k_new": k_new, "v_new": v_new, "k_pages": k_pages, "v_pages": v_pages, "block_table": block_table,
                 "lens": lens}
        _refuse("k_new", given, dict.fromkeys(given, dtype) | {"block_table": i32, "lens": i32})
    new, pages, table = k_new.shape, k_pages.shape, block_table.shape
    if len(new) != 4 or v_new.shape != new:
        raise ValueError("k_new and v_new must both be [batch, T, kv_heads, head_dim]")
    if len(pages) != 4 or v_pages.shape != pages or pages[1] != new[2] or pages[3] != new[3]:
        raise ValueError(f"k_pages and v_pages must both be [n_pages, {new[2]}, page_size, {new[3]}]")
    if len(table) != 2 or table[0] != new[0] or lens.shape != new[:1]:
        raise ValueError(f"block_table must be [{new[0]}, width] and lens [{new[0]}]")
    return new[0], new[1], new[2], new[3], pages[2], pages[0], table[1], _CODES[dtype]


def tree_attention_workspace_bytes(batch: int, T: int, q_heads: int, kv_heads: int, head_dim: int, page_size: int,
                                   n_pages: int, table_width: int) -> int:
    return _cache_shape(batch, T, q_heads, kv_heads, head_dim, page_size, n_pages, table_width, BF16)[1]


def tree_attention(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, parents: torch.Tensor,
                   k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                   scale: float | None = None, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of a tree of drafted tokens over a paged cache (see dfs_tree_attention), bf16.

    q [batch, T, q_heads, D]; k_new, v_new [batch, T, kv_heads, D] (the nodes' own keys and values);
    parents [batch, T] int32 (-1: child of the cache's last token; -2: unused node); k_pages, v_pages
    [n_pages, kv_heads, page_size, D]; block_table [batch, width] int32; lens [batch] int32.  ``scale``
    defaults to D ** -0.5.  Returns [batch, T, q_heads, D]."""
    bf16 = torch.bfloat16
    index = q.get_device() if isinstance(q, torch.Tensor) else -1
    if not (_fits(q, bf16, index) and _fits(parents, torch.int32, index) and isinstance(k_new, torch.Tensor)
            and (out is None or _fits(out, bf16, index))):
        given = {"q": q, "k_new": k_new, "parents": parents} | ({} if out is None else {"out": out})
        _refuse("q", given, {"q": bf16, "k_new": bf16, "parents": torch.int32, "out": bf16})
    batch, T, Hkv, D, page, n_pages, width, dt = _cache_sizes(k_new, v_new, k_pages, v_pages, block_table, lens, index)
    shape = q.shape
    if len(shape) != 4 or dt != BF16 or shape[0] != batch or shape[1] != T or shape[3] != D:
        raise ValueError("q must be [batch, T, q_heads, head_dim], with k_new's dtype, batch, T and head_dim")
    if parents.shape != shape[:2]:
        raise ValueError("parents must be [batch, T]")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != shape:
        raise ValueError("out must have the shape of q")
    s, nb = _cache_shape(batch, T, shape[2], Hkv, D, page, n_pages, width, dt)
    ws = _scratch(workspace, q, nb)
    _call(index, "dfs_tree_attention", lib().dfs_tree_attention, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
          parents.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), lens.data_ptr(), s,
          D ** -0.5 if scale is None else scale, out.data_ptr(), _ptr(ws), nb)
    return out


def cache_commit(k_new: torch.Tensor, v_new: torch.Tensor, nodes: torch.Tensor | None, counts: torch.Tensor,
                 k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                 out_lens: torch.Tensor | None = None) -> torch.Tensor:
    """Puts accepted nodes' keys and values into a paged cache (see dfs_cache_commit), in place.

    k_new, v_new [batch, T, kv_heads, D]; nodes [batch, path_len] int32 (None: node i of a path is i);
    counts [batch] int32: nodes of the path to take.  Returns the new lengths (``lens`` stays as it is)."""
    i32 = torch.int32
    index = counts.get_device() if isinstance(counts, torch.Tensor) else -1
    if not (_fits(counts, i32, index) and isinstance(k_new, torch.Tensor) and (nodes is None or _fits(nodes, i32, index))
            and (out_lens is None or _fits(out_lens, i32, index))):
        given = {"counts": counts, "k_new": k_new, "nodes": nodes, "out_lens": out_lens}
        given = {k: t for k, t in given.items() if k in ("counts", "k_new") or t is not None}
        _refuse("counts", given, {"counts": i32, "nodes": i32, "out_lens": i32})
    batch, T, Hkv, D, page, n_pages, width, dt = _cache_sizes(k_new, v_new, k_pages, v_pages, block_table, lens, index)
    if counts.shape != lens.shape:
        raise ValueError("counts must be [batch]")
    path = T
    if nodes is not None:
        if nodes.dim() != 2 or nodes.shape[0] != batch:
            raise ValueError("nodes must be [batch, path_len]")
        path = nodes.shape[1]
    if out_lens is None:
        out_lens = torch.empty_like(lens)
    elif out_lens.shape != lens.shape:
        raise ValueError("out_lens must be [batch]")
    s, _ = _cache_shape(batch, T, Hkv, Hkv, D, page, n_pages, width, dt)
    _call(index, "dfs_cache_commit", lib().dfs_cache_commit, k_new.data_ptr(), v_new.data_ptr(), _ptr(nodes),
          counts.data_ptr(), path, k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), lens.data_ptr(), s,
          out_lens.data_ptr())
    return out_lens


def tree_positions(parents: torch.Tensor, lens: torch.Tensor, prefix_len: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """Positions of a drafted tree's nodes, for ``rope`` (see dfs_tree_positions): int32 [batch, T].

    parents [batch, T] int32 (as for ``tree_attention``), lens [batch] int32, prefix_len [1] int32: tokens that a
    shared prefix puts in front of every sequence's own."""
    i32 = torch.int32
    index = parents.get_device() if isinstance(parents, torch.Tensor) else -1
    if not (_fits(parents, i32, index) and _fits(lens, i32, index)
            and (prefix_len is None or _fits(prefix_len, i32, index)) and (out is None or _fits(out, i32, index))):
        given = {"parents": parents, "lens": lens, "prefix_len": prefix_len, "out": out}
        given = {k: t for k, t in given.items() if k in ("parents", "lens") or t is not None}
        _refuse("parents", given, dict.fromkeys(given, i32))
    shape = parents.shape
    if len(shape) != 2 or lens.shape != shape[:1]:
        raise ValueError("parents must be [batch, T] and lens [batch]")
    if prefix_len is not None and prefix_len.numel() != 1:
        raise ValueError("prefix_len must be [1]")
    if out is None:
        out = torch.empty_like(parents)
    elif out.shape != shape:
        raise ValueError("out must have the shape of parents")
    _call(index, "dfs_tree_positions", lib().dfs_tree_positions, parents.data_ptr(), lens.data_ptr(), _ptr(prefix_len),
          shape[0], shape[1], out.data_ptr())
    return out


_LAYOUTS = {"half": 0, "interleaved": 1}
_DENSE = torch.contiguous_format
_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """(freqs fp32 [rot_dim / 2], amplitude) of a model's rotary positions (see dfs_rope_frequencies), for ``rope``.

    ``scaling`` None, "linear", "ntk", "yarn" or "bands"; ``original``: the positions that the model was trained
    on, for the last two ("bands": beta_fast and beta_slow are its high and low frequency factors).  ``device``:
    where freqs goes; without one it stays on the host."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {list(_SCALINGS)}, got {scaling!r}")
    if not 0 <= rot_dim <= 1024:
        rot_dim = 0  # refused as any other that no head has, but held by the library's 64 bits
    freqs = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float32, device="cpu")  # whatever the default device is
    amplitude = ctypes.c_double()
    _check(lib().dfs_rope_frequencies(rot_dim, base, _SCALINGS[scaling], factor, original, beta_fast, beta_slow,
                                      freqs.data_ptr(), ctypes.byref(amplitude)), "dfs_rope_frequencies")
    return freqs if device is None else freqs.to(device), amplitude.value


def _rows_of(shape, step, what: str):
    """(rows, heads, head_dim, values from a row to the next) of [..., heads, head_dim], whose rows may lie apart (a slice
    of a joint projection's heads), but evenly, and each in one piece."""
    if len(shape) < 3:
        raise ValueError(f"{what} must be [..., heads, head_dim]")
    H, D = shape[-2:]
    if not ((step[-1] == 1 or D == 1) and (step[-2] == D or H == 1)):
        raise ValueError(f"{what}: a token's heads must lie in one piece")
    rows, apart = 1, H * D
    for n, by in zip(shape[-3::-1], step[-3::-1]):
        if n != 1:
            if rows == 1:
                apart = by
            elif by != apart * rows:
                raise ValueError(f"{what}: rows must lie evenly apart")
            rows *= n
    return rows, H, D, apart


@functools.lru_cache(maxsize=1024)
def _rope_shape(q, k, v, rot, layout, amplitude, dt):
    """A call's sizes as the library takes them (a reference that is read during calls only), and its rows, kv heads and
    head_dim.  q, k, v: (shape, strides), or None."""
    rows = D = None
    sizes = []
    for t, what in ((q, "q"), (k, "k"), (v, "v")):
        if t is None:
            sizes.append((0, 0))
            continue
        n, H, d, apart = _rows_of(*t, what)
        if rows is None:
            rows, D = n, d
        elif (n, d) != (rows, D):
            raise ValueError(f"{what} must have {rows} tokens and heads of {D}")
        sizes.append((H, apart))
    if k is not None and v is not None and k[0] != v[0]:
        raise ValueError("v must have the shape of k")
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {list(_LAYOUTS)}, got {layout!r}")
    (Hq, sq), (Hk, sk), (Hv, sv) = sizes
    s = _RopeShape(rows, Hq, Hk or Hv, D, rot, sq, sk, sv, amplitude, _LAYOUTS[layout], dt)
    return ctypes.byref(s), rows, Hk or Hv, D


def _on(t, dtype, index: int) -> bool:
    """Whether t is a tensor of dtype on HIP device `index`."""
    return isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.get_device() == index


def _rope_lead(t, what: str):
    """(dtype, its code, device index) of the tensor that the others of a call go by."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _CODES:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what} must be a torch.Tensor")
        _dtype_code(t, what)
    return t.dtype, _CODES[t.dtype], t.get_device()


def _refuse_rope(lead, strided: dict, dense: dict, dtypes: dict) -> None:
    """Raises for the first of the named tensors that is not on a HIP device, of its dtype and on lead's device, and for
    those of `dense` not contiguous.  None of them is optional."""
    for what, t in (strided | dense).items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what} must be a torch.Tensor")
    for what, t in (strided | dense).items():
        if not t.is_cuda:
            raise ValueError(f"{what} must be on a HIP device, got {t.device}")
        if t.dtype != dtypes[what]:
            raise ValueError(f"{what} must be {dtypes[what]}, got {t.dtype}")
        if t.device != lead.device:
            raise ValueError(f"{what} must be on {lead.device}, got {t.device}")
        if what in dense and not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")


def rope(q: torch.Tensor | None, k: torch.Tensor | None, v: torch.Tensor | None, positions: torch.Tensor,
         freqs: torch.Tensor, layout: str = "half", amplitude: float = 1.0, out=None):
    """Rotary positions (see dfs_rope): (q, k, v) with q and k turned and v as it is, dense; None stays None.

    q [..., q_heads, D], k and v [..., kv_heads, D], bf16 or fp32, may be slices of a joint projection's heads, as
    in ``qkv.view(B, T, -1, D)[:, :, :q_heads]``; positions int32, one for each token (``tree_positions`` for drafted
    nodes); freqs and amplitude as ``rope_frequencies`` gives them.  ``layout`` "half" or "interleaved".  ``out`` may
    pass preallocated (q, k, v), which for dense q and k may be these themselves."""
    lead = k if q is None else q
    if lead is None:
        raise ValueError("q or k must be given")
    dtype, dt, index = _rope_lead(lead, "k" if q is None else "q")
    if not (_fits(positions, torch.int32, index) and _fits(freqs, torch.float32, index) and _on(lead, dtype, index)
            and (k is None or _on(k, dtype, index)) and (v is None or _on(v, dtype, index))):
        given = {n: t for n, t in (("q", q), ("k", k), ("v", v)) if t is not None}
        _refuse_rope(lead, given, {"positions": positions, "freqs": freqs},
                     dict.fromkeys("qkv", dtype) | {"positions": torch.int32, "freqs": torch.float32})
    if freqs.dim() != 1:
        raise ValueError("freqs must be [rot_dim / 2]")
    s, rows, _, _ = _rope_shape(None if q is None else (q.shape, q.stride()), None if k is None else (k.shape, k.stride()),
                                None if v is None else (v.shape, v.stride()), 2 * freqs.shape[0], layout, float(amplitude), dt)
    if positions.numel() != rows:
        raise ValueError(f"positions must be one for each of {rows} tokens")
    if out is None:
        oq = None if q is None else torch.empty_like(q, memory_format=_DENSE)
        ok = None if k is None else torch.empty_like(k, memory_format=_DENSE)
        ov = None if v is None else torch.empty_like(v, memory_format=_DENSE)
    else:
        if len(out) != 3:
            raise ValueError("out must be (q, k, v)")
        for t, o, what in zip((q, k, v), out, "qkv"):
            if (t is None) != (o is None):
                raise ValueError(f"out must hold {what} if and only if {what} is given")
            if o is not None and not (_fits(o, dtype, index) and o.shape == t.shape):
                raise ValueError(f"out's {what} must be a contiguous {dtype} tensor of {what}'s shape on cuda:{index}")
        oq, ok, ov = out
    _call(index, "dfs_rope", lib().dfs_rope, _ptr(q), _ptr(k), _ptr(v), positions.data_ptr(), freqs.data_ptr(), s, _ptr(oq),
          _ptr(ok), _ptr(ov))
    return oq, ok, ov


def cache_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor,
                 freqs: torch.Tensor | None, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                 lens: torch.Tensor, layout: str = "half", amplitude: float = 1.0,
                 prefix_len: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                 out_lens: torch.Tensor | None = None):
    """Puts tokens of several sequences into a paged cache, their keys (and q) turned on the way (see dfs_cache_append).

    k, v [rows, kv_heads, D] and q [rows, q_heads, D] (None: no queries), which may be slices of a joint projection's
    heads; starts [batch + 1] int32: rows starts[b] .. starts[b + 1] - 1 go behind sequence b's lens[b] tokens.
    freqs None: nothing is turned.  Writes the pools in place.  Returns (turned q or None, new lengths); rows of
    q that belong to no sequence are left as ``q_out`` holds them."""
    i32 = torch.int32
    dtype, dt, index = _rope_lead(k, "k")
    if not (_on(k, dtype, index) and _on(v, dtype, index) and (q is None or _on(q, dtype, index))
            and _fits(k_pages, dtype, index) and _fits(v_pages, dtype, index) and _fits(starts, i32, index)
            and _fits(block_table, i32, index) and _fits(lens, i32, index)
            and (freqs is None or _fits(freqs, torch.float32, index))
            and (prefix_len is None or _fits(prefix_len, i32, index)) and (q_out is None or _fits(q_out, dtype, index))
            and (out_lens is None or _fits(out_lens, i32, index))):
        dense = {"starts": starts, "k_pages": k_pages, "v_pages": v_pages, "block_table": block_table, "lens": lens}
        more = {"freqs": freqs, "prefix_len": prefix_len, "q_out": q_out, "out_lens": out_lens}
        _refuse_rope(k, {"k": k, "v": v} | ({} if q is None else {"q": q}),
                     dense | {n: t for n, t in more.items() if t is not None},
                     dict.fromkeys((*dense, *more), i32) | dict.fromkeys(("q", "k", "v", "k_pages", "v_pages", "q_out"), dtype)
                     | {"freqs": torch.float32})
    if freqs is not None and freqs.dim() != 1:
        raise ValueError("freqs must be [rot_dim / 2]")
    s, _, Hkv, D = _rope_shape(None if q is None else (q.shape, q.stride()), (k.shape, k.stride()), (v.shape, v.stride()),
                               0 if freqs is None else 2 * freqs.shape[0], layout, float(amplitude), dt)
    pages, table, batch = k_pages.shape, block_table.shape, lens.shape
    if len(pages) != 4 or v_pages.shape != pages or pages[1] != Hkv or pages[3] != D:
        raise ValueError(f"k_pages and v_pages must both be [n_pages, {Hkv}, page_size, {D}]")
    if len(batch) != 1 or len(table) != 2 or table[0] != batch[0] or starts.shape != (batch[0] + 1,):
        raise ValueError("lens must be [batch], block_table [batch, width] and starts [batch + 1]")
    if prefix_len is not None and prefix_len.numel() != 1:
        raise ValueError("prefix_len must be [1]")
    if q is None:
        if q_out is not None:
            raise ValueError("q_out needs a q")
    elif q_out is None:
        q_out = torch.empty_like(q, memory_format=_DENSE)
    elif q_out.shape != q.shape:
        raise ValueError("q_out must have the shape of q")
    if out_lens is None:
        out_lens = torch.empty_like(lens)
    elif out_lens.shape != batch:
        raise ValueError("out_lens must be [batch]")
    c, _ = _cache_shape(batch[0], 1, Hkv, Hkv, D, pages[2], pages[0], table[1], dt)
    _call(index, "dfs_cache_append", lib().dfs_cache_append, _ptr(q), k.data_ptr(), v.data_ptr(), starts.data_ptr(),
          _ptr(freqs), s, _ptr(prefix_len), _ptr(q_out), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
          lens.data_ptr(), c, out_lens.data_ptr())
    return q_out, out_lens


@functools.lru_cache(maxsize=1024)
def _shared_scratch(batch, T, q_heads, kv_heads, head_dim, page_size, n_pages, table_width, dt, prefix_width):
    s, _ = _cache_shape(batch, T, q_heads, kv_heads, head_dim, page_size, n_pages, table_width, dt)
    return s, int(lib().dfs_tree_attention_shared_workspace_bytes(s, prefix_width))


def tree_attention_shared_workspace_bytes(batch: int, T: int, q_heads: int, kv_heads: int, head_dim: int,
                                          page_size: int, n_pages: int, table_width: int, prefix_width: int) -> int:
    return _shared_scratch(batch, T, q_heads, kv_heads, head_dim, page_size, n_pages, table_width, BF16, prefix_width)[1]


def tree_attention_shared(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, parents: torch.Tensor,
                          k_pages: torch.Tensor, v_pages: torch.Tensor, prefix_table: torch.Tensor,
                          prefix_len: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                          scale: float | None = None, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None) -> torch.Tensor:
    """``tree_attention`` for a batch whose sequences begin with one shared prefix (see dfs_tree_attention_shared).

    prefix_table [width] int32: the prefix's pages in the pools; prefix_len [1] int32.  The other arguments are
    ``tree_attention``'s, with block_table and lens of what follows the prefix."""
    bf16, i32 = torch.bfloat16, torch.int32
    index = q.get_device() if isinstance(q, torch.Tensor) else -1
    if not (_fits(q, bf16, index) and _fits(parents, i32, index) and isinstance(k_new, torch.Tensor)
            and _fits(prefix_table, i32, index) and _fits(prefix_len, i32, index)
            and (out is None or _fits(out, bf16, index))):
        given = {"q": q, "k_new": k_new, "parents": parents, "prefix_table": prefix_table, "prefix_len": prefix_len}
        given |= {} if out is None else {"out": out}
        _refuse("q", given, dict.fromkeys(given, i32) | {"q": bf16, "k_new": bf16, "out": bf16})
    batch, T, Hkv, D, page, n_pages, width, dt = _cache_sizes(k_new, v_new, k_pages, v_pages, block_table, lens, index)
    shape = q.shape
    if len(shape) != 4 or dt != BF16 or shape[0] != batch or shape[1] != T or shape[3] != D:
        raise ValueError("q must be [batch, T, q_heads, head_dim], with k_new's dtype, batch, T and head_dim")
    if parents.shape != shape[:2]:
        raise ValueError("parents must be [batch, T]")
    if prefix_table.dim() != 1 or prefix_len.numel() != 1:
        raise ValueError("prefix_table must be [width] and prefix_len [1]")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != shape:
        raise ValueError("out must have the shape of q")
    prefix_width = prefix_table.shape[0]
    s, nb = _shared_scratch(batch, T, shape[2], Hkv, D, page, n_pages, width, dt, prefix_width)
    ws = _scratch(workspace, q, nb)
    _call(index, "dfs_tree_attention_shared", lib().dfs_tree_attention_shared, q.data_ptr(), k_new.data_ptr(),
          v_new.data_ptr(), parents.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), prefix_table.data_ptr(),
          prefix_len.data_ptr(), prefix_width, block_table.data_ptr(), lens.data_ptr(), s,
          D ** -0.5 if scale is None else scale, out.data_ptr(), _ptr(ws), nb)
    return out


class Selector:
    """Fixed-shape selector with its own workspace and output buffers (no per-call allocation).

    Tensor shapes, dtypes and devices are checked against the construction-time
    shape on every call, but with one tuple comparison each; the call then goes
    straight to dfs_select.  The path and scores buffers are reused by every call.
    """

    def __init__(self, batch: int, L: int, V: int, d: int, device="cuda", logits_dtype=torch.bfloat16,
                 act_dtype=torch.bfloat16, table_dtype=torch.bfloat16, mode: str = "greedy",
                 temperature: float = 1.0, seed: int = 0):
        self.device = torch.device(device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.mode, self.temperature, self.seed = _MODES[mode], float(temperature), int(seed) & (2**64 - 1)
        c = lambda t: BF16 if t == torch.bfloat16 else F32  # noqa: E731
        self._shape = _Shape(batch, L, V, d, c(logits_dtype), c(act_dtype), c(table_dtype))
        nb = int(lib().dfs_select_workspace_bytes(ctypes.byref(self._shape)))
        if nb == 0:
            raise ValueError("unsupported selector shape")
        self._ws_bytes = nb
        self.workspace = torch.empty(nb, dtype=torch.uint8, device=self.device)
        self.path = torch.empty((batch, L), dtype=torch.int32, device=self.device)
        self.scores = torch.empty((batch, L), dtype=torch.float32, device=self.device)
        self._expect = (
            ((batch, L, V), logits_dtype), ((batch, L, d), act_dtype), ((batch,), torch.int32),
            ((V, E), table_dtype), ((V, E), table_dtype), ((d, E), act_dtype),
        )
        self._fn = lib().dfs_select
        self._fn_packed = lib().dfs_select_packed

    def __call__(self, logits, hidden, prev_token, A, B, W_h):
        """W_h: the [d, 256] weight, or a PackedWeight of it (then dfs_select_packed)."""
        packed = isinstance(W_h, PackedWeight)
        args = (logits, hidden, prev_token, A, B) if packed else (logits, hidden, prev_token, A, B, W_h)
        for t, (shape, dtype) in zip(args, self._expect):
            if t.shape != shape or t.dtype != dtype or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"selector input must be a contiguous {dtype} tensor of shape {shape} "
                                 f"on {self.device}")
        if packed and (W_h.d, W_h.dtype, W_h.device) != (self._expect[5][0][0], self._expect[5][1], self.device):
            raise ValueError("packed W_h does not match the selector's d, dtype or device")
        fn = self._fn_packed if packed else self._fn
        rc = fn(logits.data_ptr(), hidden.data_ptr(), prev_token.data_ptr(), A.data_ptr(), B.data_ptr(),
                W_h.data_ptr(), K, ctypes.byref(self._shape), self.mode, self.temperature, self.seed,
                self.workspace.data_ptr(), self._ws_bytes, self.path.data_ptr(), self.scores.data_ptr(),
                torch.cuda.current_stream(self.device).cuda_stream)
        _check(rc, "dfs_select_packed" if packed else "dfs_select")
        return self.path, self.scores


class Conv2:
    """Fixed-shape two-tap convolution (dfs_conv2) with its own workspace and output.

    Inputs are checked against the construction-time shape with one tuple
    comparison each; the call then goes straight to dfs_conv2 and writes ``self.y``.
    """

    def __init__(self, batch: int, L: int, D: int, device="cuda", dtype=torch.bfloat16):
        self.device = torch.device(device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._dt = BF16 if dtype == torch.bfloat16 else F32
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("dtype must be bfloat16 or float32")
        self._dims = (batch, L, D)
        self._ws_bytes = int(lib().dfs_conv2_workspace_bytes(batch, L, D, self._dt))
        if D % 256 or D < 256 or batch < 1 or L < 1:
            raise ValueError("unsupported convolution shape")
        self.workspace = torch.empty(max(1, self._ws_bytes), dtype=torch.uint8, device=self.device)
        self.y = torch.empty((batch, L, D), dtype=dtype, device=self.device)
        self._expect = (((batch, L, D), dtype), ((batch, D), dtype), ((2, D), dtype), ((D // 16, 2, D), dtype))
        self._fn = lib().dfs_conv2

    def __call__(self, x, x_prev, base, W_c):
        args = (x, x_prev, base, W_c)
        for t, (shape, dtype) in zip(args, self._expect):
            if t.shape != shape or t.dtype != dtype or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"convolution input must be a contiguous {dtype} tensor of shape {shape} "
                                 f"on {self.device}")
        rc = self._fn(x.data_ptr(), x_prev.data_ptr(), base.data_ptr(), W_c.data_ptr(), self._dt, *self._dims,
                      self.y.data_ptr(), self.workspace.data_ptr(), self._ws_bytes,
                      torch.cuda.current_stream(self.device).cuda_stream)
        _check(rc, "dfs_conv2")
        return self.y
