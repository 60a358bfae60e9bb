"""Python binding of libmsa_b200.so, the B200 (sm_100a) MiniMax Sparse Attention forward path.

Argument marshalling only: every step of the path runs in the library's CUDA kernels. Tensors are
torch CUDA tensors (bf16 data may be passed as torch.bfloat16 or as 16-bit integer bit patterns);
the current torch CUDA stream is used unless one is given. Functions keep the C names.

If the compiled library is missing the import fails loudly: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa_b200.so")

MSA_OK = 0
STATUS_NAMES = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARG", 2: "MSA_ERR_UNSUPPORTED", 3: "MSA_ERR_WORKSPACE",
                4: "MSA_ERR_CUDA", 5: "MSA_ERR_TIMEOUT", 6: "MSA_ERR_DEVICE_CHECK"}


class MsaError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}" + (f" [{detail}]" if detail else ""))
        self.status = status


class msa_kv2q_layout(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("H_kv", ctypes.c_int32), ("B_k", ctypes.c_int32), ("k", ctypes.c_int32),
                ("nb", ctypes.c_int32), ("window", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("n_windows", ctypes.c_int32), ("max_items", ctypes.c_int64), ("offsets", ctypes.c_size_t),
                ("entries", ctypes.c_size_t), ("items", ctypes.c_size_t), ("window_items", ctypes.c_size_t),
                ("counts", ctypes.c_size_t), ("bases", ctypes.c_size_t), ("total_bytes", ctypes.c_size_t)]


class msa_kv4_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("B", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("d_h", ctypes.c_int32),
                ("L_max", ctypes.c_int64), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


_vp, _i64, _int, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_LP = ctypes.POINTER(msa_kv2q_layout)
_CP = ctypes.POINTER(msa_kv4_cache)

# (name, restype, argtypes) for every symbol declared in include/msa.h
SIGNATURES = [
    ("msa_status_string", ctypes.c_char_p, [_int]),
    ("msa_get_device_error", _int, [_vp, _vp]),
    ("msa_index_topk_workspace_size", _sz, [_i64, _int, _int, _int, _int]),
    ("msa_index_topk", _int, [_vp, _vp, _i64, _int, _int, _int, _int, _vp, _vp, _sz, _vp]),
    ("msa_kv2q_layout_get", _int, [_i64, _int, _int, _int, _int, _int, _LP]),
    ("msa_build_kv2q_workspace_size", _sz, [_LP]),
    ("msa_build_kv2q", _int, [_vp, _LP, _vp, _vp, _sz, _vp]),
    ("msa_build_kv2q_static", _int, [_vp, _LP, _vp, _vp]),
    ("msa_sparse_prefill_workspace_size", _sz, [_i64, _int, _int, _int, _int, _int, _i64, _int]),
    ("msa_sparse_prefill", _int, [_vp, _vp, _vp, _i64, _int, _int, _int, _int, _int, _vp, _LP, _vp, _vp, _vp, _vp,
                                  _sz, _vp]),
    ("msa_sparse_decode_workspace_size", _sz, [_int, _i64, _int, _int, _int, _int, _int, _int]),
    ("msa_sparse_decode", _int, [_vp, _vp, _vp, _vp, _vp, _vp, _int, _i64, _int, _int, _int, _int, _int, _int, _vp,
                                 _vp, _vp, _vp, _sz, _vp]),
    ("msa_sparse_prefill_varlen_workspace_size", _sz, [_vp, _vp, _int, _int, _int, _int, _int, _int, _i64]),
    ("msa_sparse_prefill_varlen", _int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _int, _int,
                                         _vp, _vp, _vp, _vp, _sz, _vp]),
    ("msa_sparse_backward_workspace_size", _sz, [_i64, _int, _int, _int, _int, _int, _int, _int]),
    ("msa_sparse_backward", _int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _int, _int, _vp, _LP, _vp,
                                   _vp, _vp, _vp, _vp, _vp, _int, ctypes.c_float, _vp, _vp, _vp, _vp, _sz, _vp]),
    ("msa_quantize_e4m3", _int, [_vp, _i64, _int, _int, _vp, _vp, _vp, _vp, _vp]),
    ("msa_sparse_prefill_fp8", _int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _int, _int,
                                      _vp, _LP, _vp, _vp, _vp, _vp, _sz, _vp]),
    ("msa_kv4_rows_workspace_size", _sz, []),
    ("msa_kv4_append", _int, [_CP, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    ("msa_kv4_read", _int, [_CP, _vp, _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
    ("msa_kv4_decode_workspace_size", _sz, [_int, _int]),
    ("msa_kv4_decode", _int, [_CP, _vp, _vp, _int, _vp, _int, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _sz, _vp]),
    ("msa_sparse_decode_kv4_workspace_size", _sz, [_int, _i64, _int, _int, _int, _int]),
    ("msa_sparse_decode_kv4", _int, [_CP, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _vp, _vp, ctypes.c_float, _vp,
                                     _vp, _vp, _vp, _sz, _vp]),
    ("msa_kv4_evict_workspace_size", _sz, [_int, _int, _int]),
    ("msa_kv4_evict", _int, [_CP, _CP, _vp, _vp, _int, _int, _int, _vp, _vp, _int, _vp, _vp, _vp, _vp, _sz, _vp]),
    ("msa_selftest_workspace_size", _sz, []),
    ("msa_selftest_wait_timeout", _int, [_vp, _sz, _i64, _vp]),
    ("msa_trace_set", None, [_vp]),
    ("msa_last_error_string", ctypes.c_char_p, []),
    ("msa_launch_count", ctypes.c_uint64, []),
]

KERNEL_NAMES = {1: "index_topk", 2: "kv2q", 3: "attn", 4: "combine", 5: "dec_pool", 6: "dec_topk", 7: "dec_attn",
                8: "dec_combine", 9: "bwd_prep", 10: "bwd_attn", 11: "bwd_convert", 12: "quant",
                13: "kv4_append", 14: "kv4_read", 15: "kv4_attn", 16: "kv4_weights", 17: "kv4_evict"}


class msa_trace(ctypes.Structure):
    _fields_ = [("events", ctypes.POINTER(ctypes.c_void_p)), ("capacity", ctypes.c_int), ("count", ctypes.c_int),
                ("kernel_ids", ctypes.POINTER(ctypes.c_int))]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m block_sparse_long_idx_b200.build` "
                          "(there is no CPU or PyTorch fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, res, args in SIGNATURES:
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def _check(fn: str, status: int):
    if status != MSA_OK:
        detail = lib.msa_last_error_string().decode() if status == 4 else ""
        raise MsaError(fn, status, detail)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bf16(t, name):
    if not t.is_cuda or not t.is_contiguous() or t.element_size() != 2:
        raise ValueError(f"{name}: expected a contiguous 16-bit CUDA tensor")
    return t


def _workspace(nbytes: int, device, ws):
    if ws is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    if ws.numel() * ws.element_size() < nbytes:
        raise ValueError("workspace too small")
    return ws


def _side(stream):
    """The stream given to a call as torch's, or None where it is the current one."""
    handle = _stream(stream)
    if handle == torch.cuda.current_stream().cuda_stream:
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(0 if handle == 1 else handle)  # 1: the legacy default stream, torch's 0


def _own_tensors(result):
    if isinstance(result, torch.Tensor):
        return [result]
    if isinstance(result, (tuple, list)):
        return [t for r in result for t in _own_tensors(r)]
    return [t for t in getattr(result, "__dict__", {}).values() if isinstance(t, torch.Tensor)]


def _under(side, call, at, args, kw):
    """The call with `side` as the current stream: what it allocates belongs to that stream, whose kernels use it. (Memory
    from the pool of the stream that was current may still be in use by work queued there, which `side` does not wait
    for.) Results are kept from reuse until both streams, as they stand when they are let go of, are done with them."""
    here = torch.cuda.current_stream(side.device)
    if len(args) > at:
        args = args[:at] + (None,) + args[at + 1:]
    else:
        kw = {**kw, "stream": None}
    with torch.cuda.stream(side):
        result = call(*args, **kw)
    for t in _own_tensors(result):
        t.record_stream(side)
        t.record_stream(here)
    return result


def _on_stream(call):
    """Runs a call whose `stream` is given and is not the current one under that stream."""
    at = list(inspect.signature(call).parameters).index("stream")

    @functools.wraps(call)
    def run(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        side = None if stream is None else _side(stream)
        return call(*args, **kw) if side is None else _under(side, call, at, args, kw)

    return run


def msa_launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(lib.msa_launch_count())


class KernelTrace:
    """Per-kernel CUDA-event timing of library calls made while active (``with KernelTrace(n) as t``).

    After the traced work has finished, ``t.durations()`` maps kernel name -> list of durations (ms)."""

    def __init__(self, max_kernels: int = 4096):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * max_kernels)]
        for e in self.events:  # torch creates the CUDA event lazily, at its first record
            e.record()
        torch.cuda.synchronize()
        self._handles = (ctypes.c_void_p * len(self.events))(*[e.cuda_event for e in self.events])
        self._ids = (ctypes.c_int * max_kernels)()
        self.rec = msa_trace(self._handles, len(self.events), 0, self._ids)

    def __enter__(self):
        self.rec.count = 0
        lib.msa_trace_set(ctypes.byref(self.rec))
        return self

    def __exit__(self, *exc):
        lib.msa_trace_set(None)
        return False

    def durations(self):
        torch.cuda.synchronize()
        out = {}
        for j in range(self.rec.count // 2):
            name = KERNEL_NAMES.get(self._ids[j], str(self._ids[j]))
            out.setdefault(name, []).append(self.events[2 * j].elapsed_time(self.events[2 * j + 1]))
        return out


def status_string(status: int) -> str:
    return lib.msa_status_string(status).decode()


def msa_get_device_error(workspace: torch.Tensor, stream=None) -> int:
    """Device error word of a workspace used by a previous call (synchronises the stream)."""
    return lib.msa_get_device_error(workspace.data_ptr(), _stream(stream))


@_on_stream
def msa_sparse_prefill_varlen(q, k_, v, q_idx, k_idx, cu_seqlens, B_k: int = 128, k: int = 16, block_idx=None,
                              out=None, lse=None, want_lse: bool = True, workspace=None, max_rows_per_pass: int = 0,
                              stream=None, cu_seqlens_k=None):
    """Packed batch of independent sequences (cu_seqlens [B+1], host ints, over the query rows;
    cu_seqlens_k over the key rows when keys hold cached prefixes): index branch, inversion,
    attention and combine in one call. Returns (out [T, H_q, d_h], lse [T, H_q], block_idx [H_kv, T, k])."""
    for t, n in ((q, "q"), (k_, "k"), (v, "v"), (q_idx, "q_idx"), (k_idx, "k_idx")):
        _bf16(t, n)
    T, H_q, d_h = q.shape
    H_kv, d_idx = k_idx.shape[1], k_idx.shape[2]
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    B = len(cu) - 1
    cu_p = cu.ctypes.data_as(ctypes.c_void_p)
    cuk = None if cu_seqlens_k is None else np.ascontiguousarray(np.asarray(cu_seqlens_k, dtype=np.int32))
    cuk_p = None if cuk is None else cuk.ctypes.data_as(ctypes.c_void_p)
    if block_idx is None:
        block_idx = torch.empty((H_kv, T, k), dtype=torch.int32, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((T, H_q), dtype=torch.float32, device=q.device)
    need = lib.msa_sparse_prefill_varlen_workspace_size(cu_p, cuk_p, B, H_q, H_kv, d_h, B_k, k, max_rows_per_pass)
    if need == 0:
        raise MsaError("msa_sparse_prefill_varlen_workspace_size", 1, "arguments rejected")
    ws = _workspace(need, q.device, workspace)
    _check("msa_sparse_prefill_varlen", lib.msa_sparse_prefill_varlen(
        q.data_ptr(), k_.data_ptr(), v.data_ptr(), q_idx.data_ptr(), k_idx.data_ptr(), cu_p, cuk_p, B, H_q, H_kv, d_h,
        d_idx,
        B_k, k, block_idx.data_ptr(), out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _stream(stream)))
    return out, lse, block_idx


@_on_stream
def msa_selftest_wait_timeout(limit_cycles: int = 1_000_000, workspace=None, device=None, stream=None) -> int:
    """Runs the bounded-wait failure path on the device (a wait that can never complete) and
    returns the device status it left: MSA_ERR_TIMEOUT when the path works."""
    dev = workspace.device if workspace is not None else (device or torch.device("cuda"))
    ws = _workspace(lib.msa_selftest_workspace_size(), dev, workspace)
    _check("msa_selftest_wait_timeout", lib.msa_selftest_wait_timeout(ws.data_ptr(), ws.numel(), int(limit_cycles),
                                                                       _stream(stream)))
    return msa_get_device_error(ws, stream)


@_on_stream
def msa_index_topk(q_idx, k_idx, B_k: int = 128, k: int = 16, block_idx=None, workspace=None, stream=None):
    """Index Branch: scores, block max-pool, Top-k with forced local block. Returns block_idx [H_kv, N, k] int32."""
    _bf16(q_idx, "q_idx")
    _bf16(k_idx, "k_idx")
    N, H_kv, d_idx = k_idx.shape
    if block_idx is None:
        block_idx = torch.empty((H_kv, N, k), dtype=torch.int32, device=k_idx.device)
    ws = _workspace(lib.msa_index_topk_workspace_size(N, H_kv, d_idx, B_k, k), k_idx.device, workspace)
    _check("msa_index_topk", lib.msa_index_topk(q_idx.data_ptr(), k_idx.data_ptr(), N, H_kv, d_idx, B_k, k,
                                                 block_idx.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
    return block_idx


def msa_kv2q_layout_get(N: int, H_kv: int, B_k: int = 128, k: int = 16, window: int = 0, chunk: int = 0):
    L = msa_kv2q_layout()
    _check("msa_kv2q_layout_get", lib.msa_kv2q_layout_get(N, H_kv, B_k, k, window, chunk, ctypes.byref(L)))
    return L


class KV2Q:
    """A built KV->Q inversion: the host layout plus the device buffer it describes."""

    def __init__(self, layout: msa_kv2q_layout, buf: torch.Tensor):
        self.layout = layout
        self.buf = buf

    def _i32(self, off: int, n: int) -> torch.Tensor:
        return self.buf[off: off + 4 * n].view(torch.int32)

    def offsets(self) -> torch.Tensor:
        L = self.layout
        return self._i32(L.offsets, L.H_kv * (L.nb + 1)).view(L.H_kv, L.nb + 1)

    def entries(self) -> torch.Tensor:
        L = self.layout
        return self._i32(L.entries, L.H_kv * L.N * L.k).view(L.H_kv, L.N * L.k)

    def window_items(self) -> torch.Tensor:
        L = self.layout
        return self._i32(L.window_items, L.n_windows + 1)

    def items(self, n: int) -> torch.Tensor:
        """First n work items as int32 [n, 4] = (r, b, start, len)."""
        return self._i32(self.layout.items, 4 * n).view(n, 4)


@_on_stream
def msa_build_kv2q(block_idx, B_k: int = 128, window: int = 0, chunk: int = 0, workspace=None, stream=None) -> KV2Q:
    """KV->Q inversion of block_idx [H_kv, N, k] into per-block query lists and a work list."""
    H_kv, N, k = block_idx.shape
    L = msa_kv2q_layout_get(N, H_kv, B_k, k, window, chunk)
    buf = torch.empty(L.total_bytes, dtype=torch.uint8, device=block_idx.device)
    ws = _workspace(lib.msa_build_kv2q_workspace_size(ctypes.byref(L)), block_idx.device, workspace)
    _check("msa_build_kv2q", lib.msa_build_kv2q(block_idx.data_ptr(), ctypes.byref(L), buf.data_ptr(),
                                                 ws.data_ptr(), ws.numel(), _stream(stream)))
    return KV2Q(L, buf)


def msa_sparse_prefill_workspace_size(N, H_q, H_kv, d_h, B_k=128, k=16, max_rows_per_pass=0, internal_kv2q=False):
    return lib.msa_sparse_prefill_workspace_size(N, H_q, H_kv, d_h, B_k, k, max_rows_per_pass, int(internal_kv2q))


@_on_stream
def msa_sparse_prefill(q, k_, v, block_idx, kv2q: KV2Q | None = None, B_k: int = 128, out=None, lse=None,
                       want_lse: bool = True, workspace=None, max_rows_per_pass: int = 0, stream=None):
    """Main Branch: exact block-sparse attention on the selected blocks. Returns (out, lse)."""
    for t, n in ((q, "q"), (k_, "k"), (v, "v")):
        _bf16(t, n)
    N, H_q, d_h = q.shape
    H_kv = k_.shape[1]
    kk = block_idx.shape[2]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((N, H_q), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(msa_sparse_prefill_workspace_size(N, H_q, H_kv, d_h, B_k, kk, max_rows_per_pass,
                                                                  kv2q is None), dtype=torch.uint8, device=q.device)
    lp = ctypes.byref(kv2q.layout) if kv2q is not None else None
    _check("msa_sparse_prefill", lib.msa_sparse_prefill(
        q.data_ptr(), k_.data_ptr(), v.data_ptr(), N, H_q, H_kv, d_h, B_k, kk, block_idx.data_ptr(), lp,
        _ptr(kv2q.buf) if kv2q is not None else None, out.data_ptr(), _ptr(lse), workspace.data_ptr(),
        workspace.numel(), _stream(stream)))
    return out, lse


@_on_stream
def msa_sparse_backward(q, k_, v, out, lse, dout, block_idx=None, kv2q: KV2Q | None = None, B_k: int = 128,
                        k: int | None = None, dq=None, dk=None, dv=None, q_idx=None, k_idx=None,
                        kl_weight: float = 1.0, want_kl: bool = True, workspace=None, stream=None):
    """Main-branch backward with the selections held fixed: gradients of sum(dout * out) in q, k, v.

    out, lse: the forward's results for the same q, k, v and selections. Returns (dq, dk, dv) bf16.
    With q_idx, k_idx (the index branch's inputs; needs block_idx) the same pass also returns the
    KL alignment's gradients and per-(row, group) KL: (dq, dk, dv, dq_idx, dk_idx, kl)."""
    for t, n in ((q, "q"), (k_, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _bf16(t, n)
    if not lse.is_cuda or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse: expected a contiguous float32 CUDA tensor")
    N, H_q, d_h = q.shape
    H_kv = k_.shape[1]
    if k is None:
        if block_idx is None:
            raise ValueError("msa_sparse_backward: k is needed when block_idx is not given")
        k = block_idx.shape[2]
    if kv2q is None and block_idx is None:
        raise ValueError("msa_sparse_backward: give block_idx or a built kv2q")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k_) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    with_kl = q_idx is not None
    d_idx = 0
    dq_idx = dk_idx = kl = None
    if with_kl:
        _bf16(q_idx, "q_idx")
        _bf16(k_idx, "k_idx")
        if block_idx is None:
            raise ValueError("msa_sparse_backward: the KL part needs block_idx")
        d_idx = q_idx.shape[2]
        dq_idx, dk_idx = torch.empty_like(q_idx), torch.empty_like(k_idx)
        kl = torch.empty((N, H_kv), dtype=torch.float32, device=q.device) if want_kl else None
    ws = _workspace(lib.msa_sparse_backward_workspace_size(N, H_q, H_kv, d_h, B_k, k, d_idx, kv2q is None),
                    q.device, workspace)
    lp = ctypes.byref(kv2q.layout) if kv2q is not None else None
    _check("msa_sparse_backward", lib.msa_sparse_backward(
        q.data_ptr(), k_.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(), N, H_q, H_kv, d_h,
        B_k, k, _ptr(block_idx), lp, _ptr(kv2q.buf) if kv2q is not None else None, dq.data_ptr(), dk.data_ptr(),
        dv.data_ptr(), _ptr(q_idx), _ptr(k_idx), d_idx, float(kl_weight), _ptr(dq_idx), _ptr(dk_idx), _ptr(kl),
        ws.data_ptr(), ws.numel(), _stream(stream)))
    if with_kl:
        return dq, dk, dv, dq_idx, dk_idx, kl
    return dq, dk, dv


@_on_stream
def msa_sparse_decode(q, q_idx, k_cache, v_cache, k_idx_cache, lens, B_k: int = 128, k: int = 16, out=None, lse=None,
                      want_lse: bool = True, block_idx_out=None, workspace=None, stream=None):
    """Decode: one query per sequence at position lens-1. Returns (out, lse, block_idx)."""
    for t, n in ((q, "q"), (q_idx, "q_idx"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (k_idx_cache, "k_idx_cache")):
        _bf16(t, n)
    B, H_q, d_h = q.shape
    L_max, H_kv = k_cache.shape[1], k_cache.shape[2]
    d_idx = q_idx.shape[2]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H_q), dtype=torch.float32, device=q.device)
    if block_idx_out is None:
        block_idx_out = torch.empty((B, H_kv, k), dtype=torch.int32, device=q.device)
    ws = _workspace(lib.msa_sparse_decode_workspace_size(B, L_max, H_q, H_kv, d_h, d_idx, B_k, k), q.device,
                    workspace)
    _check("msa_sparse_decode", lib.msa_sparse_decode(
        q.data_ptr(), q_idx.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_idx_cache.data_ptr(),
        lens.data_ptr(), B, L_max, H_q, H_kv, d_h, d_idx, B_k, k, out.data_ptr(), _ptr(lse),
        block_idx_out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
    return out, lse, block_idx_out


class E4M3Rows:
    """Per-row E4M3 quantisation of a [N, H, d] tensor: codes [N, H, d] uint8, scales and rscales
    [H, S] float32 (S = N rounded up to whole 128-token blocks), blkmax [H, S / 128] float32."""

    def __init__(self, codes, scales, rscales, blkmax):
        self.codes, self.scales, self.rscales, self.blkmax = codes, scales, rscales, blkmax


@_on_stream
def msa_quantize_e4m3(x, with_rscales: bool = True, with_blkmax: bool = True, stream=None) -> E4M3Rows:
    """E4M3 codes and per-row scales (amax / 448) of x [N, H, d] bf16."""
    _bf16(x, "x")
    N, H, d = x.shape
    S = (N + 127) // 128 * 128
    codes = torch.empty((N, H, d), dtype=torch.uint8, device=x.device)
    scales = torch.empty((H, S), dtype=torch.float32, device=x.device)
    rscales = torch.empty((H, S), dtype=torch.float32, device=x.device) if with_rscales else None
    blkmax = torch.empty((H, S // 128), dtype=torch.float32, device=x.device) if with_blkmax else None
    _check("msa_quantize_e4m3", lib.msa_quantize_e4m3(x.data_ptr(), N, H, d, codes.data_ptr(), scales.data_ptr(),
                                                       _ptr(rscales), _ptr(blkmax), _stream(stream)))
    return E4M3Rows(codes, scales, rscales, blkmax)


@_on_stream
def msa_sparse_prefill_fp8(q8: E4M3Rows, k8: E4M3Rows, v8: E4M3Rows, block_idx, kv2q: KV2Q | None = None,
                           B_k: int = 128, out=None, lse=None, want_lse: bool = True, workspace=None,
                           max_rows_per_pass: int = 0, stream=None):
    """FP8 main branch on E4M3 codes and scales from msa_quantize_e4m3. Returns (out bf16, lse)."""
    N, H_q, d_h = q8.codes.shape
    H_kv = k8.codes.shape[1]
    kk = block_idx.shape[2]
    if out is None:
        out = torch.empty((N, H_q, d_h), dtype=torch.bfloat16, device=q8.codes.device)
    if lse is None and want_lse:
        lse = torch.empty((N, H_q), dtype=torch.float32, device=q8.codes.device)
    if workspace is None:
        workspace = torch.empty(msa_sparse_prefill_workspace_size(N, H_q, H_kv, d_h, B_k, kk, max_rows_per_pass,
                                                                  kv2q is None), dtype=torch.uint8,
                                device=q8.codes.device)
    lp = ctypes.byref(kv2q.layout) if kv2q is not None else None
    _check("msa_sparse_prefill_fp8", lib.msa_sparse_prefill_fp8(
        q8.codes.data_ptr(), q8.scales.data_ptr(), k8.codes.data_ptr(), k8.scales.data_ptr(), v8.codes.data_ptr(),
        v8.scales.data_ptr(), v8.rscales.data_ptr(), v8.blkmax.data_ptr(), N, H_q, H_kv, d_h, B_k, kk,
        block_idx.data_ptr(), lp, _ptr(kv2q.buf) if kv2q is not None else None, out.data_ptr(), _ptr(lse),
        workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out, lse


# --------------------------------------------------------------------------- 4-bit key/value cache
def _is(t, name, dtypes, shape, device):
    """A contiguous CUDA tensor of one of `dtypes` and of `shape` on `device`, else ValueError."""
    if t.shape != shape or t.dtype not in dtypes or t.device != device or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {'/'.join(str(d) for d in dtypes)} tensor of shape {tuple(shape)} "
                         f"on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


class KV4Cache:
    """A K/V cache held in 4 bits: E2M1 codes [B, H_kv, L_max, d_h / 2] uint8 (the even element in the low
    nibble), one E4M3 scale per 16 elements [B, H_kv, L_max, d_h / 16] uint8, one fp32 scale per tensor.

    L_max is a multiple of 128, d_h 64 or 128. The scales place the format's range: 16-element maxima
    between 0.1 and 2688 times the scale keep full precision. The kernels read the addresses and scales given here, so the
    handle's fields are fixed (the tensors' contents are not); other scales on the same tensors are another KV4Cache."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_scale: float = 1.0, v_scale: float = 1.0):
        if k_codes.dim() != 4:
            raise ValueError("k_codes: expected [B, H_kv, L_max, d_h / 2]")
        B, H_kv, L_max, half = k_codes.shape
        dev = k_codes.device
        for t, n, last in ((k_codes, "k_codes", half), (k_scales, "k_scales", half // 8), (v_codes, "v_codes", half),
                           (v_scales, "v_scales", half // 8)):
            _is(t, n, (torch.uint8,), (B, H_kv, L_max, last), dev)
        k_scale, v_scale = float(k_scale), float(v_scale)
        c = msa_kv4_cache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), B, H_kv, 2 * half, L_max,
                          k_scale, v_scale)
        fields = dict(k_codes=k_codes, k_scales=k_scales, v_codes=v_codes, v_scales=v_scales, k_scale=k_scale, v_scale=v_scale, B=B,
                      H_kv=H_kv, L_max=L_max, d_h=2 * half, device=dev, _c=c, _ref=ctypes.byref(c))
        for name in self._FIXED:
            super().__setattr__(name, fields[name])

    _FIXED = ("k_codes", "k_scales", "v_codes", "v_scales", "k_scale", "v_scale", "B", "H_kv", "L_max", "d_h", "device", "_c", "_ref")

    def __setattr__(self, name, value):
        if name in self._FIXED:
            raise AttributeError(f"KV4Cache.{name} is fixed: make another KV4Cache (it may hold the same tensors)")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        self.__setattr__(name, None)
        super().__delattr__(name)

    @classmethod
    def empty(cls, B: int, L_max: int, H_kv: int, d_h: int, k_scale: float = 1.0, v_scale: float = 1.0, device="cuda"):
        """A cache of uninitialised rows (rows are written by msa_kv4_append before lens covers them)."""
        def rows(n):
            return torch.empty((B, H_kv, L_max, n), dtype=torch.uint8, device=device)

        return cls(rows(d_h // 2), rows(d_h // 16), rows(d_h // 2), rows(d_h // 16), k_scale, v_scale)


def _on_device(call):
    """Runs a call of this section, whose tensors live on the device of its KV4Cache argument, with that device
    current (the library launches on the current device), and under the given stream (_under)."""
    names = list(inspect.signature(call).parameters)
    at, at_stream = names.index("cache"), names.index("stream")

    @functools.wraps(call)
    def run(*args, **kw):
        device = (args[at] if len(args) > at else kw["cache"]).device
        if device.index != torch.cuda.current_device():
            with torch.cuda.device(device):
                return run(*args, **kw)
        stream = args[at_stream] if len(args) > at_stream else kw.get("stream")
        side = None if stream is None else _side(stream)
        return call(*args, **kw) if side is None else _under(side, call, at_stream, args, kw)

    return run


def _raw_stream(device, stream):
    """The device's current stream, or the given one, as the library takes it."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else _stream(stream)


def _tables(cache, T, starts, cu_seqlens):
    _is(starts, "starts", _I32, (cache.B,), cache.device)
    if cu_seqlens is not None:
        _is(cu_seqlens, "cu_seqlens", _I32, (cache.B + 1,), cache.device)
    elif T != cache.B:
        raise ValueError("without cu_seqlens there is one row per sequence")


def _token_stride(t, name, cache):
    """Elements between the rows of t [T, H_kv, d_h], whose rows are contiguous."""
    T, H, d = t.shape if t.dim() == 3 else (0, 0, 0)
    strides = t.stride()
    if (H != cache.H_kv or d != cache.d_h or strides[2] != 1 or (H > 1 and strides[1] != d) or t.dtype not in _BF16 or
            t.device != cache.device or not t.is_cuda):
        raise ValueError(f"{name}: expected a 16-bit tensor [T, {cache.H_kv}, {cache.d_h}] on {cache.device} whose rows are "
                         f"contiguous, got {t.dtype} {tuple(t.shape)} strides {t.stride()}")
    return strides[0] if T > 1 else H * d


@_on_device
def msa_kv4_append(cache: KV4Cache, k, v, starts, cu_seqlens=None, workspace=None, stream=None):
    """Quantises new rows k, v [T, H_kv, d_h] (bf16; the token stride is free) into the cache: the rows
    cu_seqlens[b] .. cu_seqlens[b + 1] - 1 go to the positions starts[b], starts[b] + 1, ... of sequence b;
    without cu_seqlens T = B, one row per sequence. starts, cu_seqlens: int32 device tensors. Rows outside the
    cache are left out; a workspace (optional, msa_kv4_rows_workspace_size bytes) tells msa_get_device_error."""
    T = k.shape[0]
    ks, vs = _token_stride(k, "k", cache), _token_stride(v, "v", cache)
    if v.shape[0] != T:
        raise ValueError("k and v: different numbers of rows")
    _tables(cache, T, starts, cu_seqlens)
    ws = None if workspace is None else _workspace(lib.msa_kv4_rows_workspace_size(), cache.device, workspace)
    _check("msa_kv4_append", lib.msa_kv4_append(
        cache._ref, k.data_ptr(), v.data_ptr(), ks, vs, T, starts.data_ptr(), _ptr(cu_seqlens), _ptr(ws), 0 if ws is None else ws.numel(),
        _raw_stream(cache.device, stream)))


@_on_device
def msa_kv4_read(cache: KV4Cache, starts, cu_seqlens=None, T: int | None = None, k=None, v=None, workspace=None,
                 stream=None):
    """The rows that msa_kv4_append with the same starts, cu_seqlens and T writes, as bf16 values.
    Returns (k, v) [T, H_kv, d_h]."""
    if T is None:
        if cu_seqlens is not None:
            raise ValueError("msa_kv4_read: T (the number of rows) is needed with cu_seqlens")
        T = cache.B
    _tables(cache, T, starts, cu_seqlens)
    shape = (T, cache.H_kv, cache.d_h)
    if k is None:
        k = torch.empty_strided(shape, (cache.H_kv * cache.d_h, cache.d_h, 1), dtype=torch.bfloat16, device=cache.device)
    else:
        _is(k, "k", _BF16, shape, cache.device)
    if v is None:
        v = torch.empty_like(k)
    else:
        _is(v, "v", _BF16, shape, cache.device)
    ws = None if workspace is None else _workspace(lib.msa_kv4_rows_workspace_size(), cache.device, workspace)
    _check("msa_kv4_read", lib.msa_kv4_read(
        cache._ref, k.data_ptr(), v.data_ptr(), T, starts.data_ptr(), _ptr(cu_seqlens), _ptr(ws), 0 if ws is None else ws.numel(),
        _raw_stream(cache.device, stream)))
    return k, v


def _decode_tensors(q, cache, lens, out, lse, weights, weights_out):
    if q.dim() != 3:
        raise ValueError("q: expected [B, H_q, d_h]")
    H_q = q.shape[1]
    _is(q, "q", _BF16, (cache.B, H_q, cache.d_h), cache.device)
    _is(lens, "lens", _I32, (cache.B,), cache.device)
    if out is not None:
        _is(out, "out", _BF16, q.shape, cache.device)
    if lse is not None:
        _is(lse, "lse", _F32, (cache.B, H_q), cache.device)
    for t, n in ((weights, "weights"), (weights_out, "weights_out")):
        if t is not None:
            _is(t, n, _F32, (cache.B, cache.H_kv, cache.L_max), cache.device)
    if weights is not None and weights_out is None:
        raise ValueError("weights: give weights_out too (it may be the same tensor)")
    return H_q


@functools.lru_cache
def _kv4_decode_bytes(B, H_q):
    return lib.msa_kv4_decode_workspace_size(B, H_q)


@functools.lru_cache
def _sparse_decode_kv4_bytes(B, L_max, H_q, H_kv, B_k, k):
    return lib.msa_sparse_decode_kv4_workspace_size(B, L_max, H_q, H_kv, B_k, k)


@_on_device
def msa_kv4_decode(q, cache: KV4Cache, lens, block_idx=None, weights=None, weights_out=None, decay: float = 1.0, out=None,
                   lse=None, want_lse: bool = True, workspace=None, stream=None):
    """Attention of one query token per sequence (q [B, H_q, d_h]) over the first lens[b] rows of the 4-bit
    cache, or over those of them in the blocks block_idx [B, H_kv, k] (ascending, -1 padded, 128 rows each).
    With weights_out [B, H_kv, L_max] fp32 also weights_out = decay * weights + the group's attention
    weights, at the visible positions. Returns (out, lse)."""
    H_q = _decode_tensors(q, cache, lens, out, lse, weights, weights_out)
    k = 0
    if block_idx is not None:
        if block_idx.dim() != 3:
            raise ValueError("block_idx: expected [B, H_kv, k]")
        k = block_idx.shape[2]
        _is(block_idx, "block_idx", _I32, (cache.B, cache.H_kv, k), cache.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty_strided((cache.B, H_q), (H_q, 1), dtype=torch.float32, device=cache.device)
    ws = _workspace(_kv4_decode_bytes(cache.B, H_q), cache.device, workspace)
    _check("msa_kv4_decode", lib.msa_kv4_decode(
        cache._ref, q.data_ptr(), lens.data_ptr(), H_q, _ptr(block_idx), k, _ptr(weights), _ptr(weights_out), decay,
        out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _raw_stream(cache.device, stream)))
    return out, lse


@_on_device
def msa_sparse_decode_kv4(q, q_idx, cache: KV4Cache, k_idx_cache, lens, B_k: int = 128, k: int = 16, weights=None,
                          weights_out=None, decay: float = 1.0, out=None, lse=None, want_lse: bool = True,
                          block_idx_out=None, workspace=None, stream=None):
    """msa_sparse_decode with K and V in a 4-bit cache (the index keys k_idx_cache [B, L_max, H_kv, d_idx]
    stay bf16); weights, weights_out and decay as for msa_kv4_decode. Returns (out, lse, block_idx)."""
    H_q = _decode_tensors(q, cache, lens, out, lse, weights, weights_out)
    if q_idx.dim() != 3:
        raise ValueError("q_idx: expected [B, H_kv, d_idx]")
    d_idx = q_idx.shape[2]
    _is(q_idx, "q_idx", _BF16, (cache.B, cache.H_kv, d_idx), cache.device)
    _is(k_idx_cache, "k_idx_cache", _BF16, (cache.B, cache.L_max, cache.H_kv, d_idx), cache.device)
    if block_idx_out is not None:
        _is(block_idx_out, "block_idx_out", _I32, (cache.B, cache.H_kv, k), cache.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty_strided((cache.B, H_q), (H_q, 1), dtype=torch.float32, device=cache.device)
    if block_idx_out is None:
        block_idx_out = torch.empty((cache.B, cache.H_kv, max(k, 0)), dtype=torch.int32, device=cache.device)
    ws = _workspace(_sparse_decode_kv4_bytes(cache.B, cache.L_max, H_q, cache.H_kv, B_k, k), cache.device, workspace)
    _check("msa_sparse_decode_kv4", lib.msa_sparse_decode_kv4(
        cache._ref, q.data_ptr(), q_idx.data_ptr(), k_idx_cache.data_ptr(), lens.data_ptr(), H_q, d_idx, B_k, k,
        _ptr(weights), _ptr(weights_out), decay, out.data_ptr(), _ptr(lse), block_idx_out.data_ptr(), ws.data_ptr(),
        ws.numel(), _raw_stream(cache.device, stream)))
    return out, lse, block_idx_out


@_on_device
def msa_kv4_evict(cache: KV4Cache, to: KV4Cache, weights, lens, keep: int, recent: int = 0, first: int = 0,
                  weights_dst=None, k_idx_cache=None, k_idx_dst=None, lens_out=None, kept=None, workspace=None,
                  stream=None):
    """Copies the kept tokens of every (sequence, KV head) of `cache` to the front of `to`: the first `first`,
    the last `recent` and, of the others, those with the largest weights [B, H_kv, L_max] (equal ones: the
    lower position), `keep` in all, in their order; all of a sequence of at most `keep` tokens. weights_dst
    [B, H_kv, to.L_max] and k_idx_dst [B, to.L_max, H_kv, d_idx] get the kept tokens' weights and index
    keys. Returns (lens_out [B], kept [B, H_kv, keep] positions, -1 padded)."""
    dev = cache.device
    _is(weights, "weights", _F32, (cache.B, cache.H_kv, cache.L_max), dev)
    _is(lens, "lens", _I32, (cache.B,), dev)
    if to.device != dev:
        raise ValueError("to: a cache on another device")
    if weights_dst is not None:
        _is(weights_dst, "weights_dst", _F32, (to.B, to.H_kv, to.L_max), dev)
    if (k_idx_cache is None) != (k_idx_dst is None):
        raise ValueError("give k_idx_cache and k_idx_dst together")
    d_idx = 0
    if k_idx_cache is not None:
        d_idx = k_idx_cache.shape[-1]
        _is(k_idx_cache, "k_idx_cache", _BF16, (cache.B, cache.L_max, cache.H_kv, d_idx), dev)
        _is(k_idx_dst, "k_idx_dst", _BF16, (to.B, to.L_max, to.H_kv, d_idx), dev)
    if lens_out is not None:
        _is(lens_out, "lens_out", _I32, (cache.B,), dev)
    if kept is not None:
        _is(kept, "kept", _I32, (cache.B, cache.H_kv, keep), dev)
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    if kept is None:
        keep_ = max(keep, 0)
        kept = torch.empty_strided((cache.B, cache.H_kv, keep_), (cache.H_kv * keep_, keep_, 1), dtype=torch.int32, device=dev)
    ws = None if workspace is None else _workspace(lib.msa_kv4_evict_workspace_size(cache.B, cache.H_kv, keep), dev, workspace)
    _check("msa_kv4_evict", lib.msa_kv4_evict(
        cache._ref, to._ref, weights.data_ptr(), lens.data_ptr(), keep, recent, first, _ptr(k_idx_cache), _ptr(k_idx_dst),
        d_idx, _ptr(weights_dst), lens_out.data_ptr(), kept.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(),
        _raw_stream(dev, stream)))
    return lens_out, kept
