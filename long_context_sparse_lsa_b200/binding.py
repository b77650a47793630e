"""Python binding of liblsa.so (include/lsa.h): argument marshalling only.

Every function takes torch tensors, passes their device pointers and sizes to
the C ABI on the current CUDA stream, and raises LsaError on a non-zero
status. Every step of the hot path runs in the library's CUDA kernels; there
is no fallback. If the library is missing, loading it raises immediately.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblsa.so")

LSA_DEV_BAD_LENGTH = 0x1
LSA_DEV_BAD_SEQ = 0x2
LSA_DEV_BAD_INDEX = 0x4
LSA_DEV_BAD_WEIGHT = 0x8
LSA_DEV_TIMEOUT = 0x10
LSA_DEV_BAD_QUERY = 0x20
LSA_DEV_BAD_VALUE = 0x40

STATUS = {0: "LSA_OK", 1: "LSA_ERR_INVALID_ARG", 2: "LSA_ERR_UNSUPPORTED", 3: "LSA_ERR_CUDA",
          4: "LSA_ERR_WORKSPACE"}

EXPORTS = ["lsa_version", "lsa_last_cuda_error", "lsa_status_string", "lsa_hi_block_sums", "lsa_append",
           "lsa_index_workspace_size", "lsa_index", "lsa_attend_workspace_size", "lsa_attend", "lsa_attend_fp8",
           "lsa_merge_pairs", "lsa_score_tokens", "lsa_score_blocks", "lsa_attend_lse", "lsa_shard_sets",
           "lsa_combine", "lsa_attend_grouped_workspace_size", "lsa_attend_grouped_launches", "lsa_attend_grouped",
           "lsa_attend_si_workspace_size", "lsa_attend_si_launches", "lsa_attend_si",
           "lsa_attend_noalloc", "lsa_append_index", "lsa_append_index_launches", "lsa_store_fp4",
           "lsa_attend_fp4_workspace_size", "lsa_attend_fp4_launches", "lsa_attend_fp4",
           "lsa_attend_prompt_workspace_size", "lsa_attend_prompt_launches", "lsa_attend_prompt"]

MERGE_ID_BITS = 24  # LSA_MERGE_ID_BITS


class LsaError(RuntimeError):
    def __init__(self, func: str, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        msg = f"{func} failed: {STATUS.get(status, status)}"
        if status == 3:
            msg += f" (cudaError {cuda_error})"
        super().__init__(msg)


class _Budget(ctypes.Structure):
    _fields_ = [("sink", ctypes.c_int32), ("window", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("hi_block", ctypes.c_int32), ("hi_topblocks", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("n_q", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("kv_offset", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("blk_offset", ctypes.c_void_p),
                ("q_seq", ctypes.c_void_p), ("q_len", ctypes.c_void_p)]


class _Prompts(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("row_offset", ctypes.c_void_p), ("kv_offset", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p)]


# the same two structures for struct.pack (native alignment)
_BATCH, _PROMPTS = struct.Struct("@4iq5P"), struct.Struct("@4iq3P")
assert _BATCH.size == ctypes.sizeof(_Batch) and _PROMPTS.size == ctypes.sizeof(_Prompts)


@dataclass
class Budget:
    sink: int
    window: int
    topk: int
    hi_block: int = 0
    hi_topblocks: int = 0

    @property
    def length(self) -> int:
        return self.sink + self.window + self.topk

    def c(self) -> _Budget:
        return _Budget(self.sink, self.window, self.topk, self.hi_block, self.hi_topblocks)


@dataclass
class Batch:
    """Packed-sequence batch; tensors live on the device that runs the call."""
    kv_offset: torch.Tensor   # int64 [n_seq]
    seq_lens: torch.Tensor    # int32 [n_seq]
    q_seq: torch.Tensor       # int32 [n_q]
    q_len: torch.Tensor       # int32 [n_q]
    max_len: int
    total_tokens: int
    blk_offset: torch.Tensor | None = None  # int64 [n_seq]

    def packed(self) -> bytes:
        """lsa_batch_t as bytes (cheaper to build and to pass than a ctypes structure)."""
        ko, sl, qs, ql, bo = self.kv_offset, self.seq_lens, self.q_seq, self.q_len, self.blk_offset
        i32, i64 = torch.int32, torch.int64
        if not (ko.dtype is i64 and sl.dtype is i32 and qs.dtype is i32 and ql.dtype is i32 and ko.is_contiguous()
                and sl.is_contiguous() and qs.is_contiguous() and ql.is_contiguous()):
            for name, t, dt in (("kv_offset", ko, i64), ("seq_lens", sl, i32), ("q_seq", qs, i32), ("q_len", ql, i32)):
                if t.dtype != dt or not t.is_contiguous():
                    raise TypeError(f"{name} must be a contiguous {dt} tensor")
        if bo is not None and (bo.dtype is not i64 or not bo.is_contiguous()):
            raise TypeError("blk_offset must be a contiguous int64 tensor")
        return _BATCH.pack(sl.numel(), qs.numel(), int(self.max_len), 0, int(self.total_tokens), ko.data_ptr(),
                           sl.data_ptr(), 0 if bo is None else bo.data_ptr(), qs.data_ptr(), ql.data_ptr())

    def c(self) -> _Batch:
        return _Batch.from_buffer_copy(self.packed())


@dataclass
class Prompts:
    """The newest rows of packed sequences of different lengths (include/lsa.h, lsa_prompts_t); tensors live on
    the device that runs the call. row_offset is ascending: sequence b's rows are row_offset[b] ..
    row_offset[b + 1] - 1, its newest tokens."""
    row_offset: torch.Tensor  # int32 [n_seq + 1]
    kv_offset: torch.Tensor   # int64 [n_seq]
    seq_lens: torch.Tensor    # int32 [n_seq]
    n_rows: int
    max_len: int
    total_tokens: int

    def packed(self) -> bytes:
        """lsa_prompts_t as bytes."""
        ro, ko, sl = self.row_offset, self.kv_offset, self.seq_lens
        if (ro.dtype is not torch.int32 or ko.dtype is not torch.int64 or sl.dtype is not torch.int32
                or not (ro.is_contiguous() and ko.is_contiguous() and sl.is_contiguous())):
            raise TypeError("row_offset and seq_lens must be contiguous int32, kv_offset contiguous int64 tensors")
        n_seq = sl.numel()
        if ro.numel() != n_seq + 1 or ko.numel() != n_seq:
            raise ValueError("row_offset must hold n_seq + 1 values, kv_offset and seq_lens n_seq")
        return _PROMPTS.pack(n_seq, self.n_rows, self.max_len, 0, self.total_tokens, ro.data_ptr(), ko.data_ptr(),
                             sl.data_ptr())

    def tensors(self) -> tuple:
        return self.row_offset, self.kv_offset, self.seq_lens

    def c(self) -> _Prompts:
        return _Prompts.from_buffer_copy(self.packed())


_lib = None


def library_path() -> str:
    return LIB_PATH


def load_library():
    """Load liblsa.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m long_context_sparse_lsa_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.lsa_version.restype = i32
    lib.lsa_version.argtypes = []
    lib.lsa_last_cuda_error.restype = i32
    lib.lsa_last_cuda_error.argtypes = []
    lib.lsa_status_string.restype = ctypes.c_char_p
    lib.lsa_status_string.argtypes = [i32]
    lib.lsa_hi_block_sums.restype = i32
    lib.lsa_hi_block_sums.argtypes = [vp, i32, i32, ctypes.POINTER(_Batch), i32, vp, i64, vp, vp]
    lib.lsa_append.restype = i32
    lib.lsa_append.argtypes = [vp, vp, i32, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp),
                               ctypes.POINTER(vp), i32, i32, i32, vp, i64, ctypes.POINTER(_Batch), i32, vp, vp]
    lib.lsa_append_index.restype = i32
    lib.lsa_append_index.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                     i32, i32, i32, vp, vp, vp, i32, i32, i32, ctypes.POINTER(_Batch), _Budget, vp, i64,
                                     vp, vp, sz, vp, vp]
    lib.lsa_append_index_launches.restype = i32
    lib.lsa_append_index_launches.argtypes = [ctypes.POINTER(_Batch), i32, i32, _Budget, i32]
    lib.lsa_index_workspace_size.restype = sz
    lib.lsa_index_workspace_size.argtypes = [ctypes.POINTER(_Batch), i32, i32, _Budget]
    lib.lsa_index_launches.restype = i32
    lib.lsa_index_launches.argtypes = [ctypes.POINTER(_Batch), i32, i32, _Budget]
    lib.lsa_attend_launches.restype = i32
    lib.lsa_attend_launches.argtypes = [ctypes.POINTER(_Batch), i32, i32, i32, i32, i32]
    lib.lsa_index_uses_tensor_cores.restype = i32
    lib.lsa_index_uses_tensor_cores.argtypes = [ctypes.POINTER(_Batch), i32, i32, _Budget]
    lib.lsa_index.restype = i32
    lib.lsa_index.argtypes = [vp, vp, vp, i32, i32, i32, ctypes.POINTER(_Batch), _Budget, vp, i64, vp, vp, sz, vp, vp]
    lib.lsa_attend_workspace_size.restype = sz
    lib.lsa_attend_workspace_size.argtypes = [ctypes.POINTER(_Batch), i32, i32, i32, i32, i32]
    lib.lsa_attend.restype = i32
    lib.lsa_attend.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), i32, i32, i32, vp, i32,
                               ctypes.POINTER(_Batch), i32, ctypes.POINTER(vp), vp, sz, vp, vp]
    lib.lsa_attend_fp8.restype = i32
    lib.lsa_attend_fp8.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                   ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_float), i32, i32, i32, vp,
                                   i32, ctypes.POINTER(_Batch), i32, ctypes.POINTER(vp), vp, sz, vp, vp]
    lib.lsa_store_fp4.restype = i32
    lib.lsa_store_fp4.argtypes = [vp, i64, vp, i64, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp,
                                  vp, vp, vp]
    lib.lsa_attend_fp4_workspace_size.restype = sz
    lib.lsa_attend_fp4_workspace_size.argtypes = [ctypes.POINTER(_Batch), i32, i32, i32, i32, i32]
    lib.lsa_attend_fp4_launches.restype = i32
    lib.lsa_attend_fp4_launches.argtypes = [ctypes.POINTER(_Batch), i32, i32, i32, i32, i32]
    lib.lsa_attend_fp4.restype = i32
    lib.lsa_attend_fp4.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp, i32, vp, vp, sz, vp, vp]
    lib.lsa_attend_prompt_workspace_size.restype = sz
    lib.lsa_attend_prompt_workspace_size.argtypes = [ctypes.POINTER(_Prompts), i32, i32, i32]
    lib.lsa_attend_prompt_launches.restype = i32
    lib.lsa_attend_prompt_launches.argtypes = [ctypes.POINTER(_Prompts), i32, i32, i32]
    lib.lsa_attend_prompt.restype = i32
    lib.lsa_attend_prompt.argtypes = [vp, i64, vp, i64, vp, i64, i32, i32, i32, vp, vp, vp, vp, sz, vp, vp]
    lib.lsa_score_tokens.restype = i32
    lib.lsa_score_tokens.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, i64, vp, i32, vp, vp, vp]
    lib.lsa_score_blocks.restype = i32
    lib.lsa_score_blocks.argtypes = [vp, vp, i32, i32, i32, i32, vp, i64, vp, vp, i32, vp, vp, vp]
    lib.lsa_merge_pairs.restype = i32
    lib.lsa_merge_pairs.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp]
    lib.lsa_attend_lse.restype = i32
    lib.lsa_attend_lse.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), i32, i32, i32, vp, i32,
                                   ctypes.POINTER(_Batch), i32, ctypes.POINTER(vp), ctypes.POINTER(vp), vp, sz, vp, vp]
    lib.lsa_shard_sets.restype = i32
    lib.lsa_shard_sets.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
    lib.lsa_combine.restype = i32
    lib.lsa_combine.argtypes = [vp, vp, i32, i64, i32, vp, vp, vp]
    lib.lsa_attend_grouped_workspace_size.restype = sz
    lib.lsa_attend_grouped_workspace_size.argtypes = [ctypes.POINTER(_Batch), i32, i32, i32, i32, i32, i32]
    lib.lsa_attend_grouped_launches.restype = i32
    lib.lsa_attend_grouped_launches.argtypes = [ctypes.POINTER(_Batch), i32, i32, i32, i32, i32, i32]
    lib.lsa_attend_grouped.restype = i32
    lib.lsa_attend_grouped.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), i32, i32, i32, vp,
                                       i32, ctypes.POINTER(_Batch), i32, i32, ctypes.POINTER(vp), vp, sz, vp, vp]
    lib.lsa_attend_si_workspace_size.restype = sz
    lib.lsa_attend_si_workspace_size.argtypes = [ctypes.POINTER(_Batch), i32, i32, i32, _Budget, i32]
    lib.lsa_attend_si_launches.restype = i32
    lib.lsa_attend_si_launches.argtypes = [ctypes.POINTER(_Batch), i32, i32, i32, _Budget, i32]
    lib.lsa_attend_si.restype = i32
    lib.lsa_attend_si.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), i32, i32, i32, vp,
                                  _Budget, ctypes.POINTER(_Batch), i32, ctypes.POINTER(vp), vp, sz, vp, vp]
    lib.lsa_attend_noalloc.restype = i32
    lib.lsa_attend_noalloc.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), i32, i32, i32, vp,
                                       i32, ctypes.POINTER(_Batch), i32, ctypes.POINTER(vp), vp, vp]
    _lib = lib
    return lib


def _check(func: str, status: int):
    if status != 0:
        raise LsaError(func, status, load_library().lsa_last_cuda_error() if status == 3 else 0)


def _stream(stream) -> int:
    if stream is None:  # torch.cuda.current_stream().cuda_stream, without the 3 us of the stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def lsa_version() -> int:
    return load_library().lsa_version()


def lsa_hi_block_sums(k_idx: torch.Tensor, hi_block: int, batch: Batch, block_sums: torch.Tensor,
                      n_new: int = 0, dev_status: torch.Tensor | None = None, stream=None) -> None:
    """HI block sums into ``block_sums`` (int8 [rows, 2*d_I]); n_new > 0 only
    refreshes the blocks holding each sequence's last n_new tokens."""
    lib = load_library()
    d_I = k_idx.shape[-1]
    cb = batch.c()
    st = lib.lsa_hi_block_sums(_ptr(k_idx), d_I, hi_block, ctypes.byref(cb), n_new, _ptr(block_sums),
                               block_sums.shape[0], _ptr(dev_status), _stream(stream))
    _check("lsa_hi_block_sums", st)


def lsa_index_workspace_size(batch: Batch, H_I: int, d_I: int, budget: Budget) -> int:
    cb = batch.c()
    return int(load_library().lsa_index_workspace_size(ctypes.byref(cb), H_I, d_I, budget.c()))


def lsa_index_launches(batch: Batch, H_I: int, d_I: int, budget: Budget) -> int:
    """Kernel launches lsa_index issues for this shape."""
    cb = batch.c()
    return int(load_library().lsa_index_launches(ctypes.byref(cb), H_I, d_I, budget.c()))


def lsa_attend_launches(batch: Batch, H_q: int, H_kv: int, d: int, budget: int, layers: int) -> int:
    """Kernel launches lsa_attend issues for this shape."""
    cb = batch.c()
    return int(load_library().lsa_attend_launches(ctypes.byref(cb), H_q, H_kv, d, budget, layers))


def lsa_index_uses_tensor_cores(batch: Batch, H_I: int, d_I: int, budget: Budget) -> bool:
    """True when lsa_index scores this batch as one dense tcgen05 contraction."""
    cb = batch.c()
    return bool(load_library().lsa_index_uses_tensor_cores(ctypes.byref(cb), H_I, d_I, budget.c()))


def lsa_index(q_idx: torch.Tensor, k_idx: torch.Tensor, w: torch.Tensor, w_max: int, batch: Batch,
              budget: Budget, index_sets: torch.Tensor, block_sums: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Index sets [n_q, sink+window+topk] (int32) into ``index_sets``."""
    lib = load_library()
    n_q, H_I, d_I = q_idx.shape
    cb = batch.c()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.lsa_index(_ptr(q_idx), _ptr(k_idx), _ptr(w), w_max, H_I, d_I, ctypes.byref(cb), budget.c(),
                       _ptr(block_sums), 0 if block_sums is None else block_sums.shape[0], _ptr(index_sets),
                       _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))
    _check("lsa_index", st)


def lsa_attend_workspace_size(batch: Batch, H_q: int, H_kv: int, d: int, budget: int, layers: int) -> int:
    cb = batch.c()
    return int(load_library().lsa_attend_workspace_size(ctypes.byref(cb), H_q, H_kv, d, budget, layers))


def lsa_append(k_idx_new: torch.Tensor, k_idx: torch.Tensor, k_new: list, v_new: list, k: list, v: list,
               hi_block: int, block_sums: torch.Tensor | None, batch: Batch, n_new: int,
               dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Write the n_new newest tokens of every sequence (keys k_idx_new [n_seq, n_new, d_I], per-layer K/V
    rows k_new/v_new [n_seq, n_new, H_kv, d], bf16 or FP8 codes like the caches k/v) into the caches and
    refresh their blocks' sums (HI on)."""
    lib = load_library()
    G = len(k_new)
    d_I = k_idx.shape[-1]
    row_bytes = k[0].shape[1] * k[0].shape[2] * k[0].element_size() if G else 0
    arr = ctypes.c_void_p * max(G, 1)
    kn, vn, kc, vc = (arr(*[t.data_ptr() for t in x]) for x in (k_new, v_new, k, v))
    cb = batch.c()
    rows = block_sums.shape[0] if block_sums is not None else 0
    st = lib.lsa_append(_ptr(k_idx_new), _ptr(k_idx), d_I, kn, vn, kc, vc, row_bytes, G, hi_block, _ptr(block_sums),
                        rows, ctypes.byref(cb), n_new, _ptr(dev_status), _stream(stream))
    _check("lsa_append", st)


def lsa_append_index(k_idx_new: torch.Tensor, k_new: list, v_new: list, k: list, v: list, n_new: int,
                     q_idx: torch.Tensor, k_idx: torch.Tensor, w: torch.Tensor, w_max: int, batch: Batch,
                     budget: Budget, index_sets: torch.Tensor, block_sums: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                     stream=None) -> None:
    """lsa_append (the n_new newest tokens' keys and K/V rows, their blocks' sums) followed by lsa_index, in one
    call; with HI on and the new tokens inside every window the append runs inside the block selection."""
    lib = load_library()
    G = len(k_new)
    n_q, H_I, d_I = q_idx.shape
    row_bytes = k[0].shape[1] * k[0].shape[2] * k[0].element_size() if G else 0
    arr = ctypes.c_void_p * max(G, 1)
    kn, vn, kc, vc = (arr(*[t.data_ptr() for t in x]) for x in (k_new, v_new, k, v))
    cb = batch.c()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rows = block_sums.shape[0] if block_sums is not None else 0
    st = lib.lsa_append_index(_ptr(k_idx_new), kn, vn, kc, vc, row_bytes, G, n_new, _ptr(q_idx), _ptr(k_idx), _ptr(w),
                              w_max, H_I, d_I, ctypes.byref(cb), budget.c(), _ptr(block_sums), rows,
                              _ptr(index_sets), _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))
    _check("lsa_append_index", st)


def lsa_append_index_launches(batch: Batch, H_I: int, d_I: int, budget: Budget, n_new: int) -> int:
    """Kernel launches lsa_append_index issues for this shape."""
    cb = batch.c()
    return int(load_library().lsa_append_index_launches(ctypes.byref(cb), H_I, d_I, budget.c(), n_new))


def lsa_attend(q: list, k: list, v: list, index_sets: torch.Tensor, batch: Batch, out: list,
               workspace: torch.Tensor, dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Sparse attention of G layers (lists of G tensors) over one index set per row."""
    lib = load_library()
    G = len(q)
    n_q, H_q, d = q[0].shape
    H_kv = k[0].shape[1]
    arr = ctypes.c_void_p * G
    qa, ka, va, oa = (arr(*[t.data_ptr() for t in x]) for x in (q, k, v, out))
    cb = batch.c()
    st = lib.lsa_attend(qa, ka, va, H_q, H_kv, d, _ptr(index_sets), index_sets.shape[1], ctypes.byref(cb), G, oa,
                        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_status),
                        _stream(stream))
    _check("lsa_attend", st)


def lsa_attend_grouped_workspace_size(batch: Batch, H_q: int, H_kv: int, d: int, budget: int, layers: int,
                                      group_rows: int) -> int:
    return load_library().lsa_attend_grouped_workspace_size(ctypes.byref(batch.c()), H_q, H_kv, d, budget, layers,
                                                            group_rows)


def lsa_attend_grouped_launches(batch: Batch, H_q: int, H_kv: int, d: int, budget: int, layers: int,
                                group_rows: int) -> int:
    return load_library().lsa_attend_grouped_launches(ctypes.byref(batch.c()), H_q, H_kv, d, budget, layers,
                                                      group_rows)


def lsa_attend_grouped(q: list, k: list, v: list, index_sets: torch.Tensor, batch: Batch, group_rows: int,
                       out: list, workspace: torch.Tensor, dev_status: torch.Tensor | None = None,
                       stream=None) -> None:
    """lsa_attend for rows in groups of group_rows draft rows of one sequence:
    each group's sets are gathered once as their union."""
    lib = load_library()
    G = len(q)
    n_q, H_q, d = q[0].shape
    H_kv = k[0].shape[1]
    arr = ctypes.c_void_p * G
    qa, ka, va, oa = (arr(*[t.data_ptr() for t in x]) for x in (q, k, v, out))
    cb = batch.c()
    st = lib.lsa_attend_grouped(qa, ka, va, H_q, H_kv, d, _ptr(index_sets), index_sets.shape[1], ctypes.byref(cb),
                                G, group_rows, oa, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _ptr(dev_status), _stream(stream))
    _check("lsa_attend_grouped", st)


def lsa_attend_si_workspace_size(batch: Batch, H_q: int, H_kv: int, d: int, budget: Budget, layers: int) -> int:
    return load_library().lsa_attend_si_workspace_size(ctypes.byref(batch.c()), H_q, H_kv, d, budget.c(), layers)


def lsa_attend_si_launches(batch: Batch, H_q: int, H_kv: int, d: int, budget: Budget, layers: int) -> int:
    return load_library().lsa_attend_si_launches(ctypes.byref(batch.c()), H_q, H_kv, d, budget.c(), layers)


def lsa_attend_si(q: list, k: list, v: list, index_sets: torch.Tensor, budget: Budget, batch: Batch, out: list,
                  workspace: torch.Tensor, dev_status: torch.Tensor | None = None, stream=None) -> None:
    """lsa_attend over SI-structured sets (as lsa_index writes them): the sink
    and window runs as dense tiles, the selected entries gathered per row."""
    lib = load_library()
    G = len(q)
    n_q, H_q, d = q[0].shape
    H_kv = k[0].shape[1]
    if index_sets.shape[1] != budget.length:
        raise ValueError("index_sets must be [n_q, sink + window + topk]")
    arr = ctypes.c_void_p * G
    qa, ka, va, oa = (arr(*[t.data_ptr() for t in x]) for x in (q, k, v, out))
    cb = batch.c()
    st = lib.lsa_attend_si(qa, ka, va, H_q, H_kv, d, _ptr(index_sets), budget.c(), ctypes.byref(cb), G, oa,
                           _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_status),
                           _stream(stream))
    _check("lsa_attend_si", st)


def lsa_attend_lse(q: list, k: list, v: list, index_sets: torch.Tensor, batch: Batch, out: list, lse: list,
                   workspace: torch.Tensor, dev_status: torch.Tensor | None = None, stream=None) -> None:
    """lsa_attend that also writes lse[g] (fp32 [n_q, H_q]): the log of each
    row and head's softmax denominator (-inf for an empty set)."""
    lib = load_library()
    G = len(q)
    n_q, H_q, d = q[0].shape
    H_kv = k[0].shape[1]
    for t in lse:
        if t.dtype != torch.float32 or t.shape != (n_q, H_q) or not t.is_contiguous():
            raise TypeError("lse must hold contiguous float32 [n_q, H_q] tensors")
    arr = ctypes.c_void_p * G
    qa, ka, va, oa, la = (arr(*[t.data_ptr() for t in x]) for x in (q, k, v, out, lse))
    cb = batch.c()
    st = lib.lsa_attend_lse(qa, ka, va, H_q, H_kv, d, _ptr(index_sets), index_sets.shape[1], ctypes.byref(cb), G, oa,
                            la, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_status),
                            _stream(stream))
    _check("lsa_attend_lse", st)


def lsa_shard_sets(index_sets: torch.Tensor, lo: int, hi: int, local_sets: torch.Tensor,
                   dev_status: torch.Tensor | None = None, stream=None) -> None:
    """The entries of each row's set inside [lo, hi), as e - lo in set order,
    -1 after (int32 [n_q, budget] in and out)."""
    lib = load_library()
    if index_sets.dtype != torch.int32 or local_sets.dtype != torch.int32:
        raise TypeError("index sets must be int32")
    if local_sets.shape != index_sets.shape or not (index_sets.is_contiguous() and local_sets.is_contiguous()):
        raise TypeError("local_sets must be a contiguous tensor shaped like index_sets")
    n_q, budget = index_sets.shape
    st = lib.lsa_shard_sets(_ptr(index_sets), n_q, budget, int(lo), int(hi), _ptr(local_sets), _ptr(dev_status),
                            _stream(stream))
    _check("lsa_shard_sets", st)


def lsa_combine(o_parts: torch.Tensor, lse_parts: torch.Tensor, out: torch.Tensor,
                lse_out: torch.Tensor | None = None, stream=None) -> None:
    """Exact log-sum-exp combination of attention partials: o_parts fp32
    [n_parts, rows..., d], lse_parts fp32 [n_parts, rows...], out fp32
    [rows..., d], lse_out fp32 [rows...] or None."""
    lib = load_library()
    for t in (o_parts, lse_parts, out) + ((lse_out,) if lse_out is not None else ()):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise TypeError("lsa_combine takes contiguous float32 tensors")
    n_parts, d = o_parts.shape[0], o_parts.shape[-1]
    rows = o_parts[0].numel() // max(d, 1)
    if lse_parts.numel() != n_parts * rows or out.numel() != rows * d:
        raise ValueError("lse_parts must hold n_parts x rows values and out rows x d")
    if lse_out is not None and lse_out.numel() != rows:
        raise ValueError("lse_out must hold one value per row")
    st = lib.lsa_combine(_ptr(o_parts), _ptr(lse_parts), n_parts, rows, d, _ptr(out), _ptr(lse_out), _stream(stream))
    _check("lsa_combine", st)


def lsa_attend_fp8(q: list, k8: list, v8: list, k_scale: list, v_scale: list, index_sets: torch.Tensor,
                   batch: Batch, out: list, workspace: torch.Tensor, dev_status: torch.Tensor | None = None,
                   stream=None) -> None:
    """lsa_attend over FP8 E4M3 K/V caches (uint8 tensors [T, H_kv, d]) with per-layer scales."""
    lib = load_library()
    G = len(q)
    n_q, H_q, d = q[0].shape
    H_kv = k8[0].shape[1]
    arr = ctypes.c_void_p * G
    qa, ka, va, oa = (arr(*[t.data_ptr() for t in x]) for x in (q, k8, v8, out))
    fa = ctypes.c_float * G
    ks, vs = fa(*[float(x) for x in k_scale]), fa(*[float(x) for x in v_scale])
    cb = batch.c()
    st = lib.lsa_attend_fp8(qa, ka, va, ks, vs, H_q, H_kv, d, _ptr(index_sets), index_sets.shape[1],
                            ctypes.byref(cb), G, oa, _ptr(workspace), workspace.numel() * workspace.element_size(),
                            _ptr(dev_status), _stream(stream))
    _check("lsa_attend_fp8", st)


def lsa_attend_noalloc(q: list, k: list, v: list, index_sets: torch.Tensor, batch: Batch, out: list,
                       dev_status: torch.Tensor | None = None, stream=None) -> None:
    """lsa_attend without a workspace: for callers that cannot allocate device
    memory on this path; the library's fixed static scratch is used instead
    (see include/lsa.h for the size limit and the sharing rules)."""
    lib = load_library()
    G = len(q)
    n_q, H_q, d = q[0].shape
    H_kv = k[0].shape[1]
    arr = ctypes.c_void_p * G
    qa, ka, va, oa = (arr(*[t.data_ptr() for t in x]) for x in (q, k, v, out))
    cb = batch.c()
    st = lib.lsa_attend_noalloc(qa, ka, va, H_q, H_kv, d, _ptr(index_sets), index_sets.shape[1], ctypes.byref(cb),
                                G, oa, _ptr(dev_status), _stream(stream))
    _check("lsa_attend_noalloc", st)


def _here(*tensors) -> None:
    """Refuse tensors that are not on the device the call would run on."""
    dev = tensors[0].get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("tensors must be on the current CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors must be on the current CUDA device")


def _status(t):
    if t is not None and (t.dtype is not torch.int32 or t.numel() < 1):
        raise TypeError("dev_status must be an int32 tensor")
    return _ptr(t)


_POINTERS = [struct.Struct(f"@{n}P") for n in range(9)]  # a host array of up to LSA_MAX_LAYERS device pointers
_FLOATS = [struct.Struct(f"@{n}f") for n in range(9)]


def _layers(name: str, ts: list, n: int, dtype: torch.dtype, shape: tuple) -> bytes:
    """The device pointers of a per-layer list of contiguous tensors, as a host array."""
    if len(ts) != n:
        raise ValueError(f"{name} must hold one tensor per layer")
    ptrs = []
    for t in ts:
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            raise TypeError(f"{name} must hold contiguous {dtype} tensors of shape {shape}")
        ptrs.append(t.data_ptr())
    return _POINTERS[n].pack(*ptrs)


def _layer_count(ts: list) -> int:
    if not 1 <= len(ts) <= 8:
        raise ValueError("1 to 8 layers")
    return len(ts)


def _scales(k_scale: list, v_scale: list, n: int) -> tuple[bytes, bytes]:
    if len(k_scale) != n or len(v_scale) != n:
        raise ValueError("k_scale and v_scale must hold one scale per layer")
    return _FLOATS[n].pack(*k_scale), _FLOATS[n].pack(*v_scale)


def _rows(name: str, ts: list, n: int, shape: tuple) -> tuple[bytes, int]:
    """Device pointers and row stride of a per-layer list of bf16 [rows, H, d] views, all with the same stride."""
    if len(ts) != n:
        raise ValueError(f"{name} must hold one tensor per layer")
    ptrs, stride = [], None
    for t in ts:
        if t.dtype is not torch.bfloat16 or t.shape != shape:
            raise TypeError(f"{name} must hold bfloat16 tensors of shape {shape}")
        s = _row_stride(name, t, shape[1], shape[2])
        if stride is not None and s != stride:
            raise ValueError(f"{name}: every layer must have the same row stride")
        stride = s
        ptrs.append(t.data_ptr())
    return _POINTERS[n].pack(*ptrs), stride


def _row_stride(name: str, t: torch.Tensor, H: int, d: int) -> int:
    """Elements from one token to the next of a [tokens, H, d] view whose heads are contiguous."""
    s = t.stride()
    if s[2] != 1 or (H > 1 and s[1] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return s[0] if t.shape[0] > 1 else H * d


def lsa_store_fp4(k_new: list, v_new: list, k: list, k_group: list, v: list, v_group: list, k_scale: list, v_scale: list,
                  prompts: Prompts, k_round: list | None = None, v_round: list | None = None,
                  dev_status: torch.Tensor | None = None, stream=None) -> None:
    """New K/V rows (lists of G bf16 tensors [n_rows, H_kv, 128]; views whose rows are apart, as of a fused
    projection, are taken as they are) into 4-bit caches (codes uint8 [T, H_kv, 64], group scales uint8 E4M3
    [T, H_kv, 8]) with per-layer power-of-two scales. k_round, v_round: the values the caches now hold (bf16
    [n_rows, H_kv, 128])."""
    lib = load_library()
    G = _layer_count(k_new)
    rows = tuple(k_new[0].shape)
    n_rows, H_kv, d = rows
    T = k[0].shape[0]
    if n_rows != prompts.n_rows or T < prompts.total_tokens:
        raise ValueError("k_new must hold prompts.n_rows rows and the caches prompts.total_tokens")
    kn, k_stride = _rows("k_new", k_new, G, rows)
    vn, v_stride = _rows("v_new", v_new, G, rows)
    u8, code, group = torch.uint8, (T, H_kv, d // 2), (T, H_kv, d // 16)
    if (k_round is None) != (v_round is None):
        raise ValueError("k_round and v_round come together")
    kr = vr = None
    if k_round is not None:
        kr = _layers("k_round", k_round, G, torch.bfloat16, rows)
        vr = _layers("v_round", v_round, G, torch.bfloat16, rows)
    args = (kn, k_stride, vn, v_stride, H_kv, d, prompts.packed(), G, *_scales(k_scale, v_scale, G),
            _layers("k", k, G, u8, code), _layers("k_group", k_group, G, u8, group), _layers("v", v, G, u8, code),
            _layers("v_group", v_group, G, u8, group), kr, vr, _status(dev_status))
    _here(*k_new, *v_new, *k, *k_group, *v, *v_group, *(k_round or ()), *(v_round or ()), *prompts.tensors(), dev_status)
    st = lib.lsa_store_fp4(*args, _stream(stream))
    if st:
        _check("lsa_store_fp4", st)


def lsa_attend_fp4_workspace_size(batch: Batch, H_q: int, H_kv: int, d: int, budget: int, layers: int) -> int:
    return load_library().lsa_attend_fp4_workspace_size(batch.c(), H_q, H_kv, d, budget, layers)


def lsa_attend_fp4_launches(batch: Batch, H_q: int, H_kv: int, d: int, budget: int, layers: int) -> int:
    """Kernel launches lsa_attend_fp4 issues for this shape."""
    return load_library().lsa_attend_fp4_launches(batch.c(), H_q, H_kv, d, budget, layers)


def lsa_attend_fp4(q: list, k: list, k_group: list, v: list, v_group: list, k_scale: list, v_scale: list,
                   index_sets: torch.Tensor, batch: Batch, out: list, workspace: torch.Tensor | None,
                   dev_status: torch.Tensor | None = None, stream=None) -> None:
    """lsa_attend over 4-bit K/V caches: codes uint8 [T, H_kv, 64], group scales uint8 E4M3 [T, H_kv, 8], per-layer
    scales (lists of G tensors and floats)."""
    lib = load_library()
    G = _layer_count(q)
    rows = tuple(q[0].shape)
    n_q, H_q, d = rows
    T, H_kv, _ = k[0].shape
    if index_sets.dtype is not torch.int32 or not index_sets.is_contiguous() or index_sets.shape[0] != n_q:
        raise TypeError("index_sets must be a contiguous int32 [n_q, budget] tensor")
    if T < batch.total_tokens or batch.q_seq.numel() != n_q:
        raise ValueError("the caches must hold batch.total_tokens rows, q the batch's rows")
    u8, code, group = torch.uint8, (T, H_kv, d // 2), (T, H_kv, d // 16)
    args = (_layers("q", q, G, torch.bfloat16, rows), _layers("k", k, G, u8, code),
            _layers("k_group", k_group, G, u8, group), _layers("v", v, G, u8, code),
            _layers("v_group", v_group, G, u8, group), *_scales(k_scale, v_scale, G), H_q, H_kv, d,
            index_sets.data_ptr(), index_sets.shape[1], batch.packed(), G, _layers("out", out, G, torch.float32, rows),
            _ptr(workspace), 0 if workspace is None else workspace.nbytes, _status(dev_status))
    _here(*q, *k, *k_group, *v, *v_group, index_sets, batch.kv_offset, batch.seq_lens, batch.q_seq, batch.q_len, *out,
          workspace, dev_status)
    st = lib.lsa_attend_fp4(*args, _stream(stream))
    if st:
        _check("lsa_attend_fp4", st)


def lsa_attend_prompt_workspace_size(prompts: Prompts, H_q: int, H_kv: int, d: int) -> int:
    return load_library().lsa_attend_prompt_workspace_size(prompts.c(), H_q, H_kv, d)


def lsa_attend_prompt_launches(prompts: Prompts, H_q: int, H_kv: int, d: int) -> int:
    """Kernel launches lsa_attend_prompt issues for this shape."""
    return load_library().lsa_attend_prompt_launches(prompts.c(), H_q, H_kv, d)


def lsa_attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, prompts: Prompts, out: torch.Tensor,
                      workspace: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Causal attention of the prompts' rows over every token each sees: q bf16 [n_rows, H_q, 128], k and v bf16
    [T, H_kv, 128] (views whose rows are apart, as of a fused projection, are taken as they are), out bf16 [n_rows,
    H_q, 128], lse fp32 [n_rows, H_q] or None."""
    lib = load_library()
    n_rows, H_q, d = q.shape
    T, H_kv = k.shape[:2]
    bf16 = torch.bfloat16
    if q.dtype is not bf16 or k.dtype is not bf16 or v.dtype is not bf16 or out.dtype is not bf16:
        raise TypeError("q, k, v and out must be bfloat16 tensors")
    if k.shape != (T, H_kv, d) or v.shape != k.shape or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("k and v must be [T, H_kv, d], out contiguous [n_rows, H_q, d]")
    if n_rows != prompts.n_rows or T < prompts.total_tokens:
        raise ValueError("q must hold prompts.n_rows rows, k and v prompts.total_tokens")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (n_rows, H_q) or not lse.is_contiguous()):
        raise TypeError("lse must be a contiguous float32 [n_rows, H_q] tensor")
    args = (q.data_ptr(), _row_stride("q", q, H_q, d), k.data_ptr(), _row_stride("k", k, H_kv, d), v.data_ptr(),
            _row_stride("v", v, H_kv, d), H_q, H_kv, d, prompts.packed(), out.data_ptr(), _ptr(lse), _ptr(workspace),
            0 if workspace is None else workspace.nbytes, _status(dev_status))
    _here(q, k, v, out, *prompts.tensors(), lse, workspace, dev_status)
    st = lib.lsa_attend_prompt(*args, _stream(stream))
    if st:
        _check("lsa_attend_prompt", st)


def lsa_merge_pairs(pairs: torch.Tensor, counts: torch.Tensor, k: int, out: torch.Tensor,
                    out_values: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                    stream=None) -> None:
    """Exact top-k of each row's packed (key, id) values (include/lsa.h):
    pairs int64 [n_rows, cap] holding the uint64 bit patterns (0 = empty),
    counts int32 [n_rows], out int32 [n_rows, k] (ids ascending, -1 padded),
    out_values int64 [n_rows, k] or None (the kept entries, 0 padded)."""
    lib = load_library()
    if pairs.dtype != torch.int64 or counts.dtype != torch.int32 or out.dtype != torch.int32:
        raise TypeError("pairs must be int64, counts and out int32")
    if not (pairs.is_contiguous() and counts.is_contiguous() and out.is_contiguous()):
        raise TypeError("pairs, counts and out must be contiguous")
    n_rows, cap = pairs.shape
    if counts.shape != (n_rows,) or out.shape != (n_rows, k):
        raise ValueError("counts must be [n_rows] and out [n_rows, k]")
    if out_values is not None and (out_values.dtype != torch.int64 or out_values.shape != (n_rows, k)
                                   or not out_values.is_contiguous()):
        raise TypeError("out_values must be a contiguous int64 [n_rows, k] tensor")
    st = lib.lsa_merge_pairs(_ptr(pairs), _ptr(counts), n_rows, cap, k, _ptr(out), _ptr(out_values),
                             _ptr(dev_status), _stream(stream))
    _check("lsa_merge_pairs", st)


def lsa_score_tokens(q_idx: torch.Tensor, k_idx: torch.Tensor, w: torch.Tensor, w_max: int,
                     row_offset: torch.Tensor, positions: torch.Tensor, keys: torch.Tensor,
                     dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Fine indexer keys (score + 1) of given positions: q_idx int8 [n_q, H_I,
    d_I], k_idx int8 [T, d_I], w int32 [n_q, H_I], row_offset int64 [n_q],
    positions int32 [n_q, n] (-1 empty), keys int32 [n_q, n] (uint32 bits)."""
    lib = load_library()
    n_q, H_I, d_I = q_idx.shape
    n = positions.shape[1]
    if keys.shape != (n_q, n) or keys.dtype != torch.int32 or positions.dtype != torch.int32:
        raise TypeError("positions and keys must be int32 [n_q, n]")
    st = lib.lsa_score_tokens(_ptr(q_idx), _ptr(k_idx), _ptr(w), w_max, H_I, d_I, n_q, _ptr(row_offset),
                              k_idx.shape[0], _ptr(positions), n, _ptr(keys), _ptr(dev_status), _stream(stream))
    _check("lsa_score_tokens", st)


def lsa_score_blocks(q_idx: torch.Tensor, w: torch.Tensor, w_max: int, block_sums: torch.Tensor,
                     blk_row_offset: torch.Tensor, blocks: torch.Tensor, keys: torch.Tensor,
                     dev_status: torch.Tensor | None = None, stream=None) -> None:
    """HI coarse keys (score + 1) of given blocks: block_sums int8 [rows,
    2*d_I] (byte planes), blk_row_offset int64 [n_q], blocks int32 [n_q, n]
    (-1 empty), keys int64 [n_q, n] (uint64 bits)."""
    lib = load_library()
    n_q, H_I, d_I = q_idx.shape
    n = blocks.shape[1]
    if keys.shape != (n_q, n) or keys.dtype != torch.int64 or blocks.dtype != torch.int32:
        raise TypeError("blocks must be int32 and keys int64 [n_q, n]")
    st = lib.lsa_score_blocks(_ptr(q_idx), _ptr(w), w_max, H_I, d_I, n_q, _ptr(block_sums), block_sums.shape[0],
                              _ptr(blk_row_offset), _ptr(blocks), n, _ptr(keys), _ptr(dev_status), _stream(stream))
    _check("lsa_score_blocks", st)
