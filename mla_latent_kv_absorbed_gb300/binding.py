"""Thin ctypes binding of libmla_decode.so (include/mla_decode.h).

Argument marshalling only: every step of the decode path runs in the
library's kernels.  torch is used for device memory and streams.  Importing
this module loads the library and raises if it has not been built (there is
no fallback path).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmla_decode.so")

MLA_OK = 0
STATUS_NAMES = {
    0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE",
    4: "MLA_ERR_CUDA", 5: "MLA_ERR_TIMEOUT", 6: "MLA_ERR_INDEX_OOB", 7: "MLA_ERR_PLAN_MISMATCH",
    8: "MLA_ERR_TREE",
}
EXPORTS = ("mla_status_string", "mla_abi_version", "mla_decode_plan", "mla_decode_run",
           "mla_decode_attend", "mla_decode_merge", "mla_merge_states", "mla_check_errors",
           "mla_decode_run_noalloc", "mla_absorb_query", "mla_project_output",
           "mla_append_kv", "mla_step_staging_bytes", "mla_decode_step_host", "mla_decode_run_multi_query",
           "mla_merge_two_states", "mla_decode_fp8_workspace_bytes", "mla_decode_run_fp8", "mla_append_kv_fp8",
           "mla_decode_graph_sizes", "mla_decode_run_graph", "mla_noalloc_check_errors", "mla_decode_run_tree",
           "mla_probe_wait_limit", "mla_rope_frequencies", "mla_rope_query", "mla_rope_append_kv",
           "mla_rope_append_kv_fp8", "mla_expand_kv", "mla_expand_kv_fp8", "mla_prefill_plan", "mla_prefill_run",
           "mla_decode_run_fp8_rows", "mla_rope_append_kv_fp8_rows", "mla_expand_kv_fp8_rows", "mla_verify_drafts",
           "mla_slots_workspace_bytes", "mla_repack_requests", "mla_copy_rows", "mla_compact_cache")
NOALLOC_SCRATCH_BYTES = 32 << 20

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with mla_latent_kv_absorbed_gb300.build.build()")

_lib = ctypes.CDLL(LIB_PATH)
_c_i32p = ctypes.POINTER(ctypes.c_int32)
_c_szp = ctypes.POINTER(ctypes.c_size_t)
_vp = ctypes.c_void_p

_lib.mla_status_string.restype = ctypes.c_char_p
_lib.mla_status_string.argtypes = [ctypes.c_int]
_lib.mla_abi_version.restype = ctypes.c_int
_lib.mla_decode_plan.restype = ctypes.c_int
_lib.mla_decode_plan.argtypes = [_vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp,
                                 ctypes.c_size_t, _c_szp, _c_szp]
_lib.mla_decode_run.restype = ctypes.c_int
_lib.mla_decode_run.argtypes = [_vp, _vp, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp, ctypes.c_float,
                                _vp, ctypes.c_int32, _vp, _vp, ctypes.c_size_t, _vp]
_lib.mla_decode_attend.restype = ctypes.c_int
_lib.mla_decode_attend.argtypes = _lib.mla_decode_run.argtypes
_lib.mla_decode_merge.restype = ctypes.c_int
_lib.mla_decode_merge.argtypes = [_vp, _vp, _vp, ctypes.c_int32, _vp, _vp, ctypes.c_size_t, _vp]
_lib.mla_merge_states.restype = ctypes.c_int
_lib.mla_merge_states.argtypes = [_vp, _vp, _vp, ctypes.c_int32, ctypes.c_int32, _vp, ctypes.c_int32,
                                  _vp, _vp]
_lib.mla_decode_run_noalloc.restype = ctypes.c_int
_lib.mla_decode_run_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp, ctypes.c_float, _vp,
                                        ctypes.c_int32, _vp, _vp]
_lib.mla_check_errors.restype = ctypes.c_int
_lib.mla_check_errors.argtypes = [_vp, _vp]
_lib.mla_noalloc_check_errors.restype = ctypes.c_int
_lib.mla_noalloc_check_errors.argtypes = [_vp]
_lib.mla_probe_wait_limit.restype = ctypes.c_int
_lib.mla_probe_wait_limit.argtypes = [_vp, _vp]
_lib.mla_absorb_query.restype = ctypes.c_int
_lib.mla_absorb_query.argtypes = [_vp, _vp, _vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp, _vp]
_lib.mla_decode_run_multi_query.restype = ctypes.c_int
_lib.mla_decode_run_multi_query.argtypes = [_vp, _vp, ctypes.c_int32, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp,
                                            ctypes.c_float, _vp, ctypes.c_int32, _vp, _vp, ctypes.c_size_t, _vp]
_lib.mla_decode_run_tree.restype = ctypes.c_int
_lib.mla_decode_run_tree.argtypes = [_vp, _vp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp,
                                     ctypes.c_float, _vp, ctypes.c_int32, _vp, _vp, ctypes.c_size_t, _vp]
_lib.mla_merge_two_states.restype = ctypes.c_int
_lib.mla_merge_two_states.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int64, _vp, ctypes.c_int32, _vp, _vp]
_lib.mla_step_staging_bytes.restype = ctypes.c_size_t
_lib.mla_step_staging_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int32]
_lib.mla_decode_step_host.restype = ctypes.c_int
_lib.mla_decode_step_host.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int32, ctypes.c_int32, _vp, ctypes.c_int64,
                                      ctypes.c_float, _vp, ctypes.c_int32, _vp, _vp, ctypes.c_size_t, _vp,
                                      ctypes.c_size_t, _vp, ctypes.c_size_t, _vp, _vp, _vp]
_lib.mla_append_kv.restype = ctypes.c_int
_lib.mla_append_kv.argtypes = [_vp, ctypes.c_int64, _vp, _vp, ctypes.c_int32, _vp, _vp]
_lib.mla_decode_fp8_workspace_bytes.restype = ctypes.c_int
_lib.mla_decode_fp8_workspace_bytes.argtypes = [_vp, _c_szp]
_lib.mla_decode_run_fp8.restype = ctypes.c_int
_lib.mla_decode_run_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, ctypes.c_int64, ctypes.c_float, _vp, _vp,
                                    ctypes.c_float, _vp, ctypes.c_int32, _vp, _vp, ctypes.c_size_t, _vp]
_lib.mla_append_kv_fp8.restype = ctypes.c_int
_lib.mla_append_kv_fp8.argtypes = [_vp, ctypes.c_int64, _vp, _vp, ctypes.c_int32, ctypes.c_float, _vp, _vp]
_lib.mla_decode_graph_sizes.restype = ctypes.c_int
_lib.mla_decode_graph_sizes.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _c_szp, _c_szp]
_lib.mla_decode_run_graph.restype = ctypes.c_int
_lib.mla_decode_run_graph.argtypes = [_vp, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp, _vp,
                                      _vp, ctypes.c_int64, _vp, _vp, ctypes.c_float, _vp, ctypes.c_int32, _vp, _vp,
                                      ctypes.c_size_t, _vp]
_lib.mla_project_output.restype = ctypes.c_int
_lib.mla_project_output.argtypes = [_vp, _vp, _vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                    _vp, _vp]
_i32, _i64, _f32, _f64, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_size_t
_lib.mla_rope_frequencies.restype = ctypes.c_int
_lib.mla_rope_frequencies.argtypes = [_f64, _i32, _f64, _i32, _f64, _f64, _vp]
_lib.mla_rope_query.restype = ctypes.c_int
_lib.mla_rope_query.argtypes = [_vp, _i64, _i64, _vp, _i32, _i32, _i32, _vp, _f32, _i32, _vp, _i64, _i64, _vp, _vp]
_lib.mla_rope_append_kv.restype = ctypes.c_int
_lib.mla_rope_append_kv.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _i32, _vp, _f32, _vp, _f32, _i32, _vp, _vp]
_lib.mla_rope_append_kv_fp8.restype = ctypes.c_int
_lib.mla_rope_append_kv_fp8.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _i32, _vp, _f32, _vp, _f32, _i32, _f32, _vp,
                                        _vp]
_lib.mla_expand_kv.restype = ctypes.c_int
_lib.mla_expand_kv.argtypes = [_vp, _i64, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]
_lib.mla_expand_kv_fp8.restype = ctypes.c_int
_lib.mla_expand_kv_fp8.argtypes = [_vp, _i64, _f32, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]
_lib.mla_prefill_plan.restype = ctypes.c_int
_lib.mla_prefill_plan.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _sz, _c_szp, _c_szp]
_lib.mla_prefill_run.restype = ctypes.c_int
_lib.mla_prefill_run.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _f32, _vp,
                                 _vp, _vp, _sz, _vp]
_lib.mla_decode_run_fp8_rows.restype = ctypes.c_int
_lib.mla_decode_run_fp8_rows.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _f32, _vp, _i32, _vp, _vp, _sz,
                                         _vp]
_lib.mla_rope_append_kv_fp8_rows.restype = ctypes.c_int
_lib.mla_rope_append_kv_fp8_rows.argtypes = [_vp, _vp, _i64, _vp, _vp, _i64, _vp, _i32, _vp, _f32, _vp, _f32, _i32, _vp,
                                             _vp]
_lib.mla_expand_kv_fp8_rows.restype = ctypes.c_int
_lib.mla_expand_kv_fp8_rows.argtypes = [_vp, _vp, _i64, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]
_lib.mla_verify_drafts.restype = ctypes.c_int
_lib.mla_verify_drafts.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                   _vp]
_lib.mla_slots_workspace_bytes.restype = _sz
_lib.mla_slots_workspace_bytes.argtypes = [_i64]
_lib.mla_repack_requests.restype = ctypes.c_int
_lib.mla_repack_requests.argtypes = [_vp, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _i64, _i64, _vp, _i64,
                                     _vp, _vp, _sz, _vp]
_lib.mla_copy_rows.restype = ctypes.c_int
_lib.mla_copy_rows.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _i32, _i32, _i32, _vp, _vp]
_lib.mla_compact_cache.restype = ctypes.c_int
_lib.mla_compact_cache.argtypes = [_vp, _vp, _i64, _i64, _i32, _i32, _vp, _i32, _vp, _i64, _vp, _vp, _vp, _sz, _vp]


class MLAError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


def status_string(status: int) -> str:
    return _lib.mla_status_string(int(status)).decode()


def abi_version() -> int:
    return int(_lib.mla_abi_version())


def library():
    return _lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return int(t.data_ptr())


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    h = getattr(stream, "cuda_stream", stream)
    return int(h) if h else None


def decode_plan(kv_indptr_host, num_heads: int, num_sms: int = 0):
    """Host plan for a batch.  Returns (plan words as int32 numpy array, workspace bytes)."""
    indptr = np.ascontiguousarray(np.asarray(kv_indptr_host), dtype=np.int32)
    B = indptr.shape[0] - 1
    need = ctypes.c_size_t(0)
    ws = ctypes.c_size_t(0)
    st = _lib.mla_decode_plan(indptr.ctypes.data, B, int(num_heads), int(num_sms), None, 0,
                              ctypes.byref(need), ctypes.byref(ws))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_plan")
    plan = np.zeros(need.value, dtype=np.int32)
    st = _lib.mla_decode_plan(indptr.ctypes.data, B, int(num_heads), int(num_sms), plan.ctypes.data,
                              plan.shape[0], ctypes.byref(need), ctypes.byref(ws))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_plan")
    return plan, int(ws.value)


_H_BATCH, _H_HEADS, _H_WORKERS, _H_ITEMS = 2, 3, 6, 8      # plan header words (include/mla_decode.h)


def plan_nnz(plan_host) -> int:
    """Token count a plan covers: the largest kv_end of its work items (the
    items tile [0, kv_indptr[batch]) exactly), 0 when it has none."""
    h = np.asarray(plan_host)
    n = int(h[_H_ITEMS])
    if n <= 0:
        return 0
    off = 16 + int(h[_H_WORKERS]) + 1
    return int(h[off + 2: off + 4 * n: 4].max())


def _check_csr(plan_host, kv_indptr, kv_indices, where) -> None:
    """The kernels trust kv_indptr to hold batch + 1 entries and kv_indices
    the slots kv_indptr names (the ABI passes no lengths); with the host plan
    both sizes are checked here, before any launch."""
    h = np.asarray(plan_host)
    batch = int(h[_H_BATCH])
    if kv_indptr is None or kv_indptr.numel() != batch + 1:
        n = 0 if kv_indptr is None else kv_indptr.numel()
        raise ValueError(f"{where}: kv_indptr has {n} entries, the plan was built for {batch + 1}")
    nnz = plan_nnz(h)
    if nnz > 0 and (kv_indices is None or kv_indices.numel() < nnz):
        n = 0 if kv_indices is None else kv_indices.numel()
        raise ValueError(f"{where}: kv_indices has {n} entries, the plan's items reach {nnz}")


def _out_dtype(out, where):
    import torch
    code = {torch.float32: 0, torch.bfloat16: 1}.get(out.dtype)
    if code is None:
        raise MLAError(2, where + ": out dtype")
    return code


def decode_run(plan_host: np.ndarray, plan_dev, q_nope, q_rope, kv_cache, kv_indptr, kv_indices,
               sm_scale: float, out, lse, workspace, stream=None, _entry="mla_decode_run") -> None:
    """Launch the decode (and merge) kernels.  Tensors are torch CUDA tensors:
    q_nope bf16 [B,H,512], q_rope bf16 [B,H,64], kv_cache bf16 [slots,576],
    kv_indptr/kv_indices int32, out fp32 or bf16 [B,H,512], lse fp32 [B,H] or
    None, workspace uint8 (zero-filled before first use)."""
    out_dtype = _out_dtype(out, _entry)
    plan_host = np.ascontiguousarray(plan_host, dtype=np.int32)
    _check_csr(plan_host, kv_indptr, kv_indices, _entry)
    st = getattr(_lib, _entry)(plan_host.ctypes.data, _ptr(plan_dev), _ptr(q_nope), _ptr(q_rope),
                             _ptr(kv_cache), int(kv_cache.shape[0]), _ptr(kv_indptr), _ptr(kv_indices),
                             float(sm_scale), _ptr(out), out_dtype, _ptr(lse), _ptr(workspace),
                             int(workspace.numel() * workspace.element_size()), _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, _entry)


def decode_attend(plan_host, plan_dev, q_nope, q_rope, kv_cache, kv_indptr, kv_indices, sm_scale, out, lse,
                  workspace, stream=None) -> None:
    """The decode kernel alone (whole requests to out/lse, cut ones to partials)."""
    decode_run(plan_host, plan_dev, q_nope, q_rope, kv_cache, kv_indptr, kv_indices, sm_scale, out, lse,
               workspace, stream, _entry="mla_decode_attend")


def decode_merge(plan_host, plan_dev, out, lse, workspace, stream=None) -> None:
    """The plan's LSE merge of partial states (no launch if nothing was cut)."""
    out_dtype = _out_dtype(out, "mla_decode_merge")
    plan_host = np.ascontiguousarray(plan_host, dtype=np.int32)
    st = _lib.mla_decode_merge(plan_host.ctypes.data, _ptr(plan_dev), _ptr(out), out_dtype, _ptr(lse),
                               _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                               _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_merge")


def decode_run_noalloc(plan_host, plan_dev, q_nope, q_rope, kv_cache, kv_indptr, kv_indices, sm_scale, out, lse,
                       stream=None) -> None:
    """mla_decode_run without a workspace: for callers that cannot allocate
    device memory.  Partial states live in the library's static 32 MiB
    device buffer, shared by every call -- calls must not overlap on the GPU."""
    out_dtype = _out_dtype(out, "mla_decode_run_noalloc")
    plan_host = np.ascontiguousarray(plan_host, dtype=np.int32)
    _check_csr(plan_host, kv_indptr, kv_indices, "mla_decode_run_noalloc")
    st = _lib.mla_decode_run_noalloc(plan_host.ctypes.data, _ptr(plan_dev), _ptr(q_nope), _ptr(q_rope),
                                     _ptr(kv_cache), int(kv_cache.shape[0]), _ptr(kv_indptr), _ptr(kv_indices),
                                     float(sm_scale), _ptr(out), out_dtype, _ptr(lse), _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_run_noalloc")


def noalloc_check_errors(stream=None) -> int:
    """Synchronise, read and clear the status word of the static buffer that
    mla_decode_run_noalloc uses on the current device."""
    return int(_lib.mla_noalloc_check_errors(_stream_handle(stream)))


def merge_states(v_partial, s_partial, merge_indptr, out, lse, stream=None) -> None:
    out_dtype = _out_dtype(out, "mla_merge_states")
    B = int(merge_indptr.shape[0]) - 1
    H = int(v_partial.shape[1])
    st = _lib.mla_merge_states(_ptr(v_partial), _ptr(s_partial), _ptr(merge_indptr), B, H, _ptr(out),
                               out_dtype, _ptr(lse), _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_merge_states")


def absorb_query(q_pre, w_kc, q_nope, workspace=None, stream=None) -> None:
    """q_nope[b,h,:] = q_pre[b,h,:] . w_kc[h]: bf16 [B,H,128] x [H,128,512] -> bf16 [B,H,512]."""
    B, H, n = (int(x) for x in q_pre.shape)
    st = _lib.mla_absorb_query(_ptr(q_pre), _ptr(w_kc), _ptr(q_nope), B, H, n, _ptr(workspace),
                               _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_absorb_query")


def project_output(o_lat, w_vc, out, workspace=None, stream=None) -> None:
    """out[b,h,:] = o_lat[b,h,:] . w_vc[h]: bf16 [B,H,512] x [H,512,128] -> fp32 or bf16 [B,H,128]."""
    out_dtype = _out_dtype(out, "mla_project_output")
    B, H = int(o_lat.shape[0]), int(o_lat.shape[1])
    st = _lib.mla_project_output(_ptr(o_lat), _ptr(w_vc), _ptr(out), out_dtype, B, H, int(w_vc.shape[2]),
                                 _ptr(workspace), _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_project_output")


def append_kv(kv_cache, slots, rows, workspace=None, stream=None) -> None:
    """kv_cache[slots[b]] = rows[b]: bf16 [num_slots, 576] <- bf16 [B, 576] at int32 slots [B]."""
    st = _lib.mla_append_kv(_ptr(kv_cache), int(kv_cache.shape[0]), _ptr(slots), _ptr(rows), int(rows.shape[0]),
                            _ptr(workspace), _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_append_kv")


def decode_graph_sizes(max_batch: int, num_heads: int, num_sms: int):
    """(plan_words, workspace_bytes) capacities of mla_decode_run_graph."""
    w, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = _lib.mla_decode_graph_sizes(int(max_batch), int(num_heads), int(num_sms), ctypes.byref(w), ctypes.byref(b))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_graph_sizes")
    return int(w.value), int(b.value)


def decode_run_graph(plan_dev, max_batch, num_heads, num_sms, q_nope, q_rope, kv_cache, kv_indptr, kv_indices,
                     sm_scale, out, lse, workspace, stream=None) -> None:
    """Decode reading its plan only from the device buffer plan_dev (int32, capacity words), so a captured
    graph can be replayed after a new plan (and new CSR arrays) are copied into the same buffers."""
    out_dtype = _out_dtype(out, "mla_decode_run_graph")
    if kv_indptr is None or kv_indptr.numel() != int(max_batch) + 1:
        raise ValueError(f"mla_decode_run_graph: kv_indptr must hold max_batch + 1 = {int(max_batch) + 1} entries")
    st = _lib.mla_decode_run_graph(_ptr(plan_dev), int(plan_dev.numel()), int(max_batch), int(num_heads),
                                   int(num_sms), _ptr(q_nope), _ptr(q_rope), _ptr(kv_cache), int(kv_cache.shape[0]),
                                   _ptr(kv_indptr), _ptr(kv_indices), float(sm_scale), _ptr(out), out_dtype,
                                   _ptr(lse), _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                                   _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_run_graph")


def decode_fp8_workspace_bytes(plan_host) -> int:
    """Workspace bytes mla_decode_run_fp8 needs for a plan (H 16 or 32)."""
    plan_host = np.ascontiguousarray(plan_host, dtype=np.int32)
    n = ctypes.c_size_t(0)
    st = _lib.mla_decode_fp8_workspace_bytes(plan_host.ctypes.data, ctypes.byref(n))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_fp8_workspace_bytes")
    return int(n.value)


def decode_run_fp8(plan_host, plan_dev, q_nope, q_rope, kv_cache, kv_scale, kv_indptr, kv_indices, sm_scale,
                   out, lse, workspace, stream=None) -> None:
    """Decode over an FP8 cache: kv_cache uint8 [num_slots, 576] E4M3 codes (value = code x kv_scale);
    other tensors as for decode_run; workspace of decode_fp8_workspace_bytes(plan) bytes, zero-filled once."""
    out_dtype = _out_dtype(out, "mla_decode_run_fp8")
    plan_host = np.ascontiguousarray(plan_host, dtype=np.int32)
    _check_csr(plan_host, kv_indptr, kv_indices, "mla_decode_run_fp8")
    st = _lib.mla_decode_run_fp8(plan_host.ctypes.data, _ptr(plan_dev), _ptr(q_nope), _ptr(q_rope), _ptr(kv_cache),
                                 int(kv_cache.shape[0]), float(kv_scale), _ptr(kv_indptr), _ptr(kv_indices),
                                 float(sm_scale), _ptr(out), out_dtype, _ptr(lse), _ptr(workspace),
                                 int(workspace.numel() * workspace.element_size()), _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_run_fp8")


def decode_run_fp8_rows(plan_host, plan_dev, q_nope, q_rope, kv_cache, kv_scales, kv_indptr, kv_indices, sm_scale, out,
                        lse, workspace, stream=None) -> None:
    """Decode over an FP8 cache with a scale for every row: kv_cache uint8 [num_slots, 576] E4M3 codes, kv_scales
    float32 [num_slots] (value = code x kv_scales[slot]); other tensors as for decode_run, in their types and shapes;
    workspace of decode_fp8_workspace_bytes(plan) bytes, zero-filled once."""
    import torch
    w = "mla_decode_run_fp8_rows"
    plan_host = np.ascontiguousarray(plan_host, dtype=np.int32)
    if plan_host.size < 16:
        raise ValueError(f"{w}: plan_host is the int32 array of decode_plan")
    _check_csr(plan_host, kv_indptr, kv_indices, w)
    B, H = int(plan_host[_H_BATCH]), int(plan_host[_H_HEADS])
    N = _sizes(w, "kv_cache", kv_cache, 2)[0]
    _need(w, "plan_dev", plan_dev, torch.int32, (plan_host.size,))
    _need(w, "q_nope", q_nope, torch.bfloat16, (B, H, 512))
    _need(w, "q_rope", q_rope, torch.bfloat16, (B, H, 64))
    _need(w, "kv_cache", kv_cache, torch.uint8, (N, 576))
    _need(w, "kv_scales", kv_scales, torch.float32, (N,))
    _need(w, "kv_indptr", kv_indptr, torch.int32, (B + 1,))
    if kv_indices is not None:
        _need(w, "kv_indices", kv_indices, torch.int32, (kv_indices.numel(),))
    out_dtype = _out_dtype(out, w)
    _need(w, "out", out, out.dtype, (B, H, 512))
    if lse is not None:
        _need(w, "lse", lse, torch.float32, (B, H))
    _need(w, "workspace", workspace, torch.uint8, (workspace.numel(),))
    st = _launch_stream(w, stream, plan_dev, q_nope, q_rope, kv_cache, kv_scales, kv_indptr, kv_indices, out, lse,
                        workspace)
    st = _lib.mla_decode_run_fp8_rows(_host_ptr(plan_host), plan_dev.data_ptr(), q_nope.data_ptr(), q_rope.data_ptr(),
                                      kv_cache.data_ptr(), N, kv_scales.data_ptr(), kv_indptr.data_ptr(),
                                      _ptr(kv_indices), float(sm_scale), out.data_ptr(), out_dtype, _ptr(lse),
                                      workspace.data_ptr(), workspace.numel(), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def append_kv_fp8(kv_cache, slots, rows, kv_scale, workspace=None, stream=None) -> None:
    """kv_cache[slots[b]] = E4M3(rows[b] / kv_scale): uint8 [num_slots, 576] <- bf16 [B, 576]."""
    st = _lib.mla_append_kv_fp8(_ptr(kv_cache), int(kv_cache.shape[0]), _ptr(slots), _ptr(rows), int(rows.shape[0]),
                                float(kv_scale), _ptr(workspace), _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_append_kv_fp8")


def decode_run_multi_query(plan_host, plan_dev, q_len, q_nope, q_rope, kv_cache, kv_indptr, kv_indices, sm_scale,
                           out, lse, workspace, stream=None) -> None:
    """q_len draft tokens per request in one pass: q [B, q_len, H, 576 split], out [B, q_len, H, 512]."""
    out_dtype = _out_dtype(out, "mla_decode_run_multi_query")
    plan_host = np.ascontiguousarray(plan_host, dtype=np.int32)
    _check_csr(plan_host, kv_indptr, kv_indices, "mla_decode_run_multi_query")
    st = _lib.mla_decode_run_multi_query(plan_host.ctypes.data, _ptr(plan_dev), int(q_len), _ptr(q_nope),
                                         _ptr(q_rope), _ptr(kv_cache), int(kv_cache.shape[0]), _ptr(kv_indptr),
                                         _ptr(kv_indices), float(sm_scale), _ptr(out), out_dtype, _ptr(lse),
                                         _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                                         _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_run_multi_query")


def decode_run_tree(plan_host, plan_dev, parents, tree_masks, q_nope, q_rope, kv_cache, kv_indptr, kv_indices,
                    sm_scale, out, lse, workspace, stream=None) -> None:
    """A tree of W draft tokens per request in one pass: parents device int32 [B, W] (each draft's parent, an
    earlier draft, or -1), tree_masks device int64 [B, W] scratch; q [B, W, H, 576 split], out [B, W, H, 512]."""
    out_dtype = _out_dtype(out, "mla_decode_run_tree")
    plan_host = np.ascontiguousarray(plan_host, dtype=np.int32)
    _check_csr(plan_host, kv_indptr, kv_indices, "mla_decode_run_tree")
    W = int(parents.shape[-1])
    if tree_masks.numel() < parents.numel() or tree_masks.element_size() != 8:
        raise MLAError(1, "mla_decode_run_tree: tree_masks must hold one 8-byte word per draft")
    st = _lib.mla_decode_run_tree(plan_host.ctypes.data, _ptr(plan_dev), W, _ptr(parents), _ptr(tree_masks),
                                  _ptr(q_nope), _ptr(q_rope), _ptr(kv_cache), int(kv_cache.shape[0]),
                                  _ptr(kv_indptr), _ptr(kv_indices), float(sm_scale), _ptr(out), out_dtype,
                                  _ptr(lse), _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                                  _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_run_tree")


def merge_two_states(o_a, lse_a, o_b, lse_b, out, lse, stream=None) -> None:
    """Row-wise LSE merge of two fp32 states [..., 512] / [...] into out (fp32 or bf16) and lse."""
    out_dtype = _out_dtype(out, "mla_merge_two_states")
    rows = int(lse_a.numel())
    st = _lib.mla_merge_two_states(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), rows, _ptr(out), out_dtype,
                                   _ptr(lse), _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_merge_two_states")


def step_staging_bytes(batch: int, num_heads: int, nnz: int, plan_words: int, out_dtype: int) -> int:
    return int(_lib.mla_step_staging_bytes(batch, num_heads, nnz, plan_words, out_dtype))


def decode_step_host(q_nope, q_rope, kv_indptr, kv_indices, kv_cache, sm_scale, out, lse, plan, staging, workspace,
                     stream=None, copy_in_stream=None, copy_out_stream=None) -> None:
    """One step from host tensors (pinned for asynchronous copies): plan, copy in, run, copy out on `stream`.
    `plan` is a host int32 tensor with room for the plan words."""
    out_dtype = _out_dtype(out, "mla_decode_step_host")
    B, H = int(q_nope.shape[0]), int(q_nope.shape[1])
    if kv_indptr.numel() != B + 1 or kv_indices.numel() < int(kv_indptr[-1]):
        raise ValueError("mla_decode_step_host: kv_indptr must hold batch + 1 entries and kv_indices the "
                         "kv_indptr[batch] slots it names")
    st = _lib.mla_decode_step_host(_ptr(q_nope), _ptr(q_rope), _ptr(kv_indptr), _ptr(kv_indices), B, H,
                                   _ptr(kv_cache), int(kv_cache.shape[0]), float(sm_scale), _ptr(out), out_dtype,
                                   _ptr(lse), _ptr(plan), int(plan.numel()), _ptr(staging), int(staging.numel()),
                                   _ptr(workspace), int(workspace.numel()), _stream_handle(stream),
                                   None if copy_in_stream is None else _stream_handle(copy_in_stream),
                                   None if copy_out_stream is None else _stream_handle(copy_out_stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_decode_step_host")


# ---- the prompt side: rotary positions, latent expansion, expanded attention ----

def _need(where, name, t, dtype, shape, dense=True) -> None:
    """The ABI passes no lengths and no types: a tensor of another type, shape, layout or device is refused
    here, before any launch.  dense: contiguous; else only the last dimension is."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and (t.is_contiguous() or not dense and t.stride(-1) == 1):
        return
    if t.dtype is not dtype:
        raise ValueError(f"{where}: {name} is {t.dtype}, {dtype} is wanted")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, {tuple(shape)} is wanted")
    if t.numel() and not (t.is_contiguous() if dense else (t.stride(-1) == 1 or t.shape[-1] == 1)):
        raise ValueError(f"{where}: {name} is not laid out {'densely' if dense else 'with its last dimension together'}")
    if not t.is_cuda:
        raise ValueError(f"{where}: {name} is not on a CUDA device")


def _sizes(where, name, t, dims):
    """The shape of a tensor that sets the sizes of a call."""
    if t.dim() != dims:
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, {dims} dimensions are wanted")
    return t.shape


def _status_word(where, workspace) -> None:
    if workspace is not None and workspace.numel() * workspace.element_size() < 4:
        raise ValueError(f"{where}: workspace has no room for the status word")


def _current(stream):
    """The current device, and the handle of `stream` or of the device's current stream."""
    import torch
    try:                                             # what current_device and current_stream look up, without
        cur = torch._C._cuda_getDevice()             # their objects: a third of a small call's host time
        return cur, torch._C._cuda_getCurrentRawStream(cur) if stream is None else _stream_handle(stream) or 0
    except AttributeError:
        return torch.cuda.current_device(), _stream_handle(stream) or 0


def _launch_stream(where, stream, *tensors):
    """The stream to launch on (the current one when none is given).  Every tensor has to be on the current
    device: the launch goes there."""
    cur, raw = _current(stream)
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"{where}: a tensor is on device {t.device}, the current device is cuda:{cur}")
    return raw or None


_ROPE_SCALING = {"none": 0, "linear": 1, "yarn": 2}


def rope_frequencies(theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_positions: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0) -> np.ndarray:
    """Rotary frequencies of the 64-wide part as 64-bit fractions of a turn per position: uint64 numpy [32].
    scaling: "none", "linear" (positions interpolated by factor) or "yarn"."""
    freqs = np.zeros(32, dtype=np.uint64)
    if scaling not in _ROPE_SCALING:
        raise MLAError(2, f"mla_rope_frequencies: scaling {scaling!r}")
    st = _lib.mla_rope_frequencies(float(theta), _ROPE_SCALING[scaling], float(factor), int(original_positions),
                                   float(beta_fast), float(beta_slow), freqs.ctypes.data)
    if st != MLA_OK:
        raise MLAError(st, "mla_rope_frequencies")
    return freqs


def _host_ptr(a) -> int:
    """Address of a numpy array (through the buffer protocol: a third of `ctypes.data`'s time)."""
    try:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    except TypeError:                                # a read-only array
        return a.ctypes.data


def _freqs_ptr(where, freqs):
    if not isinstance(freqs, np.ndarray) or freqs.dtype != np.uint64 or freqs.shape != (32,) or \
            not freqs.flags.c_contiguous:
        raise ValueError(f"{where}: freqs is the uint64 array of rope_frequencies")
    return _host_ptr(freqs)


def rope_query(q, positions, freqs, q_rope, q_nope=None, amplitude: float = 1.0, interleaved: bool = True,
               stream=None) -> None:
    """Rotate the last 64 values of every head: q bf16 [T, H, nope + 64] (any strides that are multiples of 8),
    positions int32 [T] -> q_rope bf16 [T, H, 64] (a dense tensor, or q[..., nope:] itself to rotate in place);
    q_nope: optional dense bf16 [T, H, nope] that receives the rest of each head."""
    import torch
    w = "mla_rope_query"
    bf = torch.bfloat16
    T, H, D = _sizes(w, "q", q, 3)
    nope = D - 64
    _need(w, "q", q, bf, (T, H, D), dense=False)
    if nope < 0:
        raise ValueError(f"{w}: q has {D} values a head, at least the 64 rotary ones are wanted")
    _need(w, "positions", positions, torch.int32, (T,))
    _need(w, "q_rope", q_rope, bf, (T, H, 64), dense=False)
    if q_nope is not None:
        _need(w, "q_nope", q_nope, bf, (T, H, nope))
    fr, st = _freqs_ptr(w, freqs), _launch_stream(w, stream, q, positions, q_rope, q_nope)
    if T == 0 or H == 0:
        return
    (qt, qh, _), (rt, rh, _) = q.stride(), q_rope.stride()
    st = _lib.mla_rope_query(q.data_ptr(), qt, qh, positions.data_ptr(), T, H, nope, fr, amplitude,
                             1 if interleaved else 0, q_rope.data_ptr(), rt, rh, _ptr(q_nope), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def _rope_append(w, cache_dtype, kv_cache, slots, rows, positions, freqs, norm_weight, workspace, stream,
                 kv_scales=None):
    import torch
    _status_word(w, workspace)
    T = _sizes(w, "rows", rows, 2)[0]
    N = _sizes(w, "kv_cache", kv_cache, 2)[0]
    _need(w, "kv_cache", kv_cache, cache_dtype, (N, 576))
    _need(w, "rows", rows, torch.bfloat16, (T, 576), dense=False)
    _need(w, "slots", slots, torch.int32, (T,))
    _need(w, "positions", positions, torch.int32, (T,))
    if norm_weight is not None:
        _need(w, "norm_weight", norm_weight, torch.bfloat16, (512,))
    return (N, T, rows.stride(0), _freqs_ptr(w, freqs),
            _launch_stream(w, stream, kv_cache, rows, slots, positions, norm_weight, workspace, kv_scales))


def rope_append_kv(kv_cache, slots, rows, positions, freqs, norm_weight=None, eps: float = 1e-6,
                   amplitude: float = 1.0, interleaved: bool = True, workspace=None, stream=None) -> None:
    """kv_cache[slots[t]] = [rms_norm(rows[t, :512]) * norm_weight, rotated rows[t, 512:]]: bf16 [num_slots, 576]
    <- bf16 [T, 576] (rows may be a slice of a wider projection); norm_weight bf16 [512] or None (no norm)."""
    import torch
    w = "mla_rope_append_kv"
    N, T, rs, fr, st = _rope_append(w, torch.bfloat16, kv_cache, slots, rows, positions, freqs, norm_weight,
                                    workspace, stream)
    st = _lib.mla_rope_append_kv(kv_cache.data_ptr(), N, slots.data_ptr(), rows.data_ptr(), rs,
                                 positions.data_ptr(), T, _ptr(norm_weight), eps, fr, amplitude,
                                 1 if interleaved else 0, _ptr(workspace), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def rope_append_kv_fp8(kv_cache, slots, rows, positions, freqs, kv_scale, norm_weight=None, eps: float = 1e-6,
                       amplitude: float = 1.0, interleaved: bool = True, workspace=None, stream=None) -> None:
    """rope_append_kv into an FP8 cache: uint8 [num_slots, 576] E4M3 codes of the values / kv_scale."""
    import torch
    w = "mla_rope_append_kv_fp8"
    N, T, rs, fr, st = _rope_append(w, torch.uint8, kv_cache, slots, rows, positions, freqs, norm_weight, workspace,
                                    stream)
    st = _lib.mla_rope_append_kv_fp8(kv_cache.data_ptr(), N, slots.data_ptr(), rows.data_ptr(), rs,
                                     positions.data_ptr(), T, _ptr(norm_weight), eps, fr, amplitude,
                                     1 if interleaved else 0, kv_scale, _ptr(workspace), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def rope_append_kv_fp8_rows(kv_cache, kv_scales, slots, rows, positions, freqs, norm_weight=None, eps: float = 1e-6,
                            amplitude: float = 1.0, interleaved: bool = True, workspace=None, stream=None) -> None:
    """rope_append_kv into an FP8 cache with a scale for every row: uint8 [num_slots, 576] E4M3 codes and float32
    kv_scales [num_slots], the row's largest magnitude / 448 (value = code x scale)."""
    import torch
    w = "mla_rope_append_kv_fp8_rows"
    N, T, rs, fr, st = _rope_append(w, torch.uint8, kv_cache, slots, rows, positions, freqs, norm_weight, workspace,
                                    stream, kv_scales)
    _need(w, "kv_scales", kv_scales, torch.float32, (N,))
    st = _lib.mla_rope_append_kv_fp8_rows(kv_cache.data_ptr(), kv_scales.data_ptr(), N, slots.data_ptr(),
                                          rows.data_ptr(), rs, positions.data_ptr(), T, _ptr(norm_weight), eps, fr,
                                          amplitude, 1 if interleaved else 0, _ptr(workspace), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def _expand(w, cache_dtype, kv_cache, kv_indices, w_kc, w_vc, k_nope, k_rope, v, workspace, stream,
            kv_scales=None):
    import torch
    _status_word(w, workspace)
    bf = torch.bfloat16
    N = _sizes(w, "kv_cache", kv_cache, 2)[0]
    T = _sizes(w, "kv_indices", kv_indices, 1)[0]
    H = _sizes(w, "w_kc", w_kc, 3)[0]
    _need(w, "kv_cache", kv_cache, cache_dtype, (N, 576))
    _need(w, "kv_indices", kv_indices, torch.int32, (T,))
    _need(w, "w_kc", w_kc, bf, (H, 128, 512))
    _need(w, "w_vc", w_vc, bf, (H, 512, 128))
    _need(w, "k_nope", k_nope, bf, (T, H, 128))
    _need(w, "k_rope", k_rope, bf, (T, 64))
    _need(w, "v", v, bf, (T, H, 128))
    return N, T, H, _launch_stream(w, stream, kv_cache, kv_indices, w_kc, w_vc, k_nope, k_rope, v, workspace, kv_scales)


def expand_kv(kv_cache, kv_indices, w_kc, w_vc, k_nope, k_rope, v, workspace=None, stream=None) -> None:
    """Per-head keys and values of the cached rows kv_indices int32 [T]: k_nope[t,h,:] = c_t . w_kc[h]^T and
    v[t,h,:] = c_t . w_vc[h] (bf16 [T,H,128]), k_rope[t,:] the rows' rope keys (bf16 [T,64])."""
    import torch
    w = "mla_expand_kv"
    N, T, H, st = _expand(w, torch.bfloat16, kv_cache, kv_indices, w_kc, w_vc, k_nope, k_rope, v, workspace, stream)
    st = _lib.mla_expand_kv(kv_cache.data_ptr(), N, kv_indices.data_ptr(), T, w_kc.data_ptr(), w_vc.data_ptr(), H,
                            k_nope.data_ptr(), k_rope.data_ptr(), v.data_ptr(), _ptr(workspace), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def expand_kv_fp8(kv_cache, kv_scale, kv_indices, w_kc, w_vc, k_nope, k_rope, v, workspace=None,
                  stream=None) -> None:
    """expand_kv from an FP8 cache: uint8 [num_slots, 576] E4M3 codes (value = code x kv_scale)."""
    import torch
    w = "mla_expand_kv_fp8"
    N, T, H, st = _expand(w, torch.uint8, kv_cache, kv_indices, w_kc, w_vc, k_nope, k_rope, v, workspace, stream)
    st = _lib.mla_expand_kv_fp8(kv_cache.data_ptr(), N, kv_scale, kv_indices.data_ptr(), T, w_kc.data_ptr(),
                                w_vc.data_ptr(), H, k_nope.data_ptr(), k_rope.data_ptr(), v.data_ptr(),
                                _ptr(workspace), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def expand_kv_fp8_rows(kv_cache, kv_scales, kv_indices, w_kc, w_vc, k_nope, k_rope, v, workspace=None,
                       stream=None) -> None:
    """expand_kv from an FP8 cache with a scale for every row: float32 kv_scales [num_slots]."""
    import torch
    w = "mla_expand_kv_fp8_rows"
    N, T, H, st = _expand(w, torch.uint8, kv_cache, kv_indices, w_kc, w_vc, k_nope, k_rope, v, workspace, stream,
                          kv_scales)
    _need(w, "kv_scales", kv_scales, torch.float32, (N,))
    st = _lib.mla_expand_kv_fp8_rows(kv_cache.data_ptr(), kv_scales.data_ptr(), N, kv_indices.data_ptr(), T,
                                     w_kc.data_ptr(), w_vc.data_ptr(), H, k_nope.data_ptr(), k_rope.data_ptr(),
                                     v.data_ptr(), _ptr(workspace), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def prefill_plan(q_indptr_host, kv_indptr_host, num_heads: int, causal: bool = True, num_sms: int = 0):
    """Host plan of the expanded attention.  Returns (plan words as int32 numpy array, workspace bytes)."""
    qp = np.ascontiguousarray(np.asarray(q_indptr_host), dtype=np.int32)
    kp = np.ascontiguousarray(np.asarray(kv_indptr_host), dtype=np.int32)
    if qp.ndim != 1 or qp.shape != kp.shape or qp.shape[0] < 1:
        raise ValueError("mla_prefill_plan: q_indptr and kv_indptr must both hold batch + 1 entries")
    need, ws = ctypes.c_size_t(0), ctypes.c_size_t(0)
    plan = np.zeros(0, dtype=np.int32)
    for _ in range(2):                               # the sizes, then the words
        st = _lib.mla_prefill_plan(qp.ctypes.data, kp.ctypes.data, qp.shape[0] - 1, int(num_heads), int(bool(causal)),
                                   int(num_sms), plan.ctypes.data if plan.size else None, plan.size,
                                   ctypes.byref(need), ctypes.byref(ws))
        if st != MLA_OK:
            raise MLAError(st, "mla_prefill_plan")
        if not plan.size:
            plan = np.zeros(need.value, dtype=np.int32)
    return plan, int(ws.value)


_P_HEADS, _P_Q, _P_KV, _P_WORDS = 3, 5, 6, 11        # prefill plan header words


def prefill_run(plan_host, plan_dev, q, k_nope, k_rope, v, sm_scale: float, out, lse, workspace, stream=None) -> None:
    """Attention over expanded keys: q bf16 [Tq,H,192], k_nope and v bf16 [Tk,H,128], k_rope bf16 [Tk,64] (strides
    that are multiples of 8), out bf16 [Tq,H,128], lse fp32 [Tq,H] or None, workspace uint8 (zero-filled once)."""
    import torch
    w, bf = "mla_prefill_run", torch.bfloat16
    if not isinstance(plan_host, np.ndarray) or plan_host.dtype != np.int32 or plan_host.size < 16 or \
            not plan_host.flags.c_contiguous:
        raise ValueError(f"{w}: plan_host is the int32 array of prefill_plan")
    head = plan_host[:16].tolist()
    if head[_P_WORDS] != plan_host.size:             # (plan_dev has as many; the kernel reads what the header counts)
        raise ValueError(f"{w}: plan_host has {plan_host.size} words, its header counts {head[_P_WORDS]}")
    H, nq, nk = head[_P_HEADS], head[_P_Q], head[_P_KV]
    _need(w, "plan_dev", plan_dev, torch.int32, (plan_host.shape[0],))
    _need(w, "q", q, bf, (nq, H, 192), dense=False)
    _need(w, "k_nope", k_nope, bf, (nk, H, 128), dense=False)
    _need(w, "k_rope", k_rope, bf, (nk, 64), dense=False)
    _need(w, "v", v, bf, (nk, H, 128), dense=False)
    _need(w, "out", out, bf, (nq, H, 128))
    if lse is not None:
        _need(w, "lse", lse, torch.float32, (nq, H))
    _need(w, "workspace", workspace, torch.uint8, (workspace.numel(),))
    st = _launch_stream(w, stream, plan_dev, q, k_nope, k_rope, v, out, lse, workspace)
    (qt, qh, _), (kt, kh, _), (vt, vh, _) = q.stride(), k_nope.stride(), v.stride()
    st = _lib.mla_prefill_run(_host_ptr(plan_host), plan_dev.data_ptr(), q.data_ptr(), qt, qh, k_nope.data_ptr(), kt,
                              kh, k_rope.data_ptr(), k_rope.stride(0), v.data_ptr(), vt, vh, sm_scale,
                              out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.numel(), st)
    if st != MLA_OK:
        raise MLAError(st, w)


# ---- between two steps: drafts verified, lists of rows rewritten, rows moved ----

def verify_drafts(target_probs, tokens, uniforms, path, accepted, next_token, draft_probs=None, parents=None,
                  workspace=None, stream=None) -> None:
    """Which drafts of a speculative step hold, and the token that follows them: target_probs fp32 [B, W, V] (row i:
    the distribution after draft i; draft 0 is the last token itself), tokens int32 and uniforms fp32 [B, W] (entry 0
    draws the next token) -> path int32 [B, W] (accepted drafts, then -1), accepted and next_token int32 [B].
    draft_probs fp32 [B, W, V]: what the drafts of a chain were sampled from; parents int32 [B, W]: a tree of chosen
    drafts; neither: a chain of chosen drafts.  Batch and row strides are free, the vocabulary lies together."""
    import torch
    w = "mla_verify_drafts"
    _status_word(w, workspace)
    f32, i32 = torch.float32, torch.int32
    B, W, V = _sizes(w, "target_probs", target_probs, 3)
    _need(w, "target_probs", target_probs, f32, (B, W, V), dense=False)
    _need(w, "tokens", tokens, i32, (B, W))
    _need(w, "uniforms", uniforms, f32, (B, W))
    _need(w, "path", path, i32, (B, W))
    _need(w, "accepted", accepted, i32, (B,))
    _need(w, "next_token", next_token, i32, (B,))
    db = dr = 0
    if draft_probs is not None:
        _need(w, "draft_probs", draft_probs, f32, (B, W, V), dense=False)
        db, dr, _ = draft_probs.stride()
    if parents is not None:
        _need(w, "parents", parents, i32, (B, W))
    st = _launch_stream(w, stream, target_probs, tokens, uniforms, path, accepted, next_token, draft_probs, parents,
                        workspace)
    tb, tr, _ = target_probs.stride()
    st = _lib.mla_verify_drafts(target_probs.data_ptr(), tb, tr, _ptr(draft_probs), db, dr, tokens.data_ptr(),
                                _ptr(parents), uniforms.data_ptr(), B, W, V, path.data_ptr(), accepted.data_ptr(),
                                next_token.data_ptr(), _ptr(workspace), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def slots_workspace_bytes(num_slots: int) -> int:
    """Workspace bytes of repack_requests and compact_cache for a pool of num_slots rows (zero-filled once)."""
    n = int(_lib.mla_slots_workspace_bytes(int(num_slots)))
    if n == 0:
        raise MLAError(1, "mla_slots_workspace_bytes")
    return n


def repack_requests(kv_indptr, kv_indices, sources, new_indptr, new_indices, num_slots: int, workspace, path=None,
                    accepted=None, freed=None, freed_count=None, stream=None) -> None:
    """The lists of the next step's requests: request r continues request sources[r] (int32 [B'], -1: no rows) of
    kv_indptr int32 [B + 1] / kv_indices int32, with path int32 [B, W] and accepted int32 [B] of verify_drafts cut to
    the accepted of its last W rows -> new_indptr int32 [B' + 1], new_indices int32 (its size is the room).  freed
    int32 and freed_count int32 [1] take the slots that no new list holds, ascending, and their number."""
    import torch
    w, i32 = "mla_repack_requests", torch.int32
    B1 = _sizes(w, "kv_indptr", kv_indptr, 1)[0]
    N1 = _sizes(w, "sources", sources, 1)[0]
    if B1 < 1:
        raise ValueError(f"{w}: kv_indptr must hold batch + 1 entries")
    _need(w, "kv_indptr", kv_indptr, i32, (B1,))
    _need(w, "kv_indices", kv_indices, i32, (kv_indices.numel(),))
    _need(w, "sources", sources, i32, (N1,))
    _need(w, "new_indptr", new_indptr, i32, (N1 + 1,))
    _need(w, "new_indices", new_indices, i32, (new_indices.numel(),))
    _need(w, "workspace", workspace, torch.uint8, (workspace.numel(),))
    W = 0
    if (path is None) != (accepted is None) or (freed is None) != (freed_count is None):
        raise ValueError(f"{w}: path goes with accepted, freed with freed_count")
    if path is not None:
        W = _sizes(w, "path", path, 2)[1]
        _need(w, "path", path, i32, (B1 - 1, W))
        _need(w, "accepted", accepted, i32, (B1 - 1,))
    if freed is not None:
        _need(w, "freed", freed, i32, (freed.numel(),))
        _need(w, "freed_count", freed_count, i32, (1,))
    st = _launch_stream(w, stream, kv_indptr, kv_indices, sources, new_indptr, new_indices, path, accepted, freed,
                        freed_count, workspace)
    st = _lib.mla_repack_requests(kv_indptr.data_ptr(), kv_indices.data_ptr(), kv_indices.numel(), B1 - 1,
                                  sources.data_ptr(), N1, _full(path), _full(accepted), W, new_indptr.data_ptr(),
                                  new_indices.data_ptr(), new_indices.numel(), int(num_slots), _full(freed),
                                  0 if freed is None else freed.numel(), _full(freed_count), workspace.data_ptr(),
                                  workspace.numel(), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def _full(t) -> Optional[int]:
    """Address of an optional tensor; that of an empty one is not null (null means it is not there)."""
    return None if t is None else t.data_ptr() or 16


def _layers(w, name, cache, scales):
    """(slots, rows from a layer to the next, layers, bytes of a row) of a cache [N, 576] or [L, N, 576] in bf16 or
    E4M3 codes, and of its scales [N] or [L, N]."""
    import torch
    dt, shape = cache.dtype, cache.shape
    codes = dt is torch.uint8
    if not (codes or dt is torch.bfloat16) or len(shape) not in (2, 3) or shape[-1] != 576:
        raise ValueError(f"{w}: {name} is {dt} {tuple(shape)}, bfloat16 or uint8 [.., slots, 576] is wanted")
    L, N = (1, shape[0]) if len(shape) == 2 else shape[:2]
    rows, dense = N, cache.is_contiguous()
    if not dense:
        if N and L and (cache.stride(-1) != 1 or (N > 1 and cache.stride(-2) != 576) or (L > 1 and cache.stride(0) % 576)):
            raise ValueError(f"{w}: {name}'s rows do not lie one after another")
        rows = N if L <= 1 else cache.stride(0) // 576
    if scales is not None:
        if not codes:
            raise ValueError(f"{w}: {name} has scales, its rows are not 8-bit")
        _need(w, name + "'s scales", scales, torch.float32, shape[:-1], dense=False)
        if L > 1 and scales.stride(0) != rows:
            raise ValueError(f"{w}: {name}'s scales lie {scales.stride(0)} apart a layer, its rows {rows}")
    return N, rows, L, 576 if codes else 1152


def copy_rows(src_cache, src_slots, dst_cache, dst_slots, src_scales=None, dst_scales=None, workspace=None,
              stream=None) -> None:
    """dst_cache[.., dst_slots[i]] = src_cache[.., src_slots[i]] in every layer: caches [N, 576] or [L, N, 576] of one
    type (bf16 or E4M3 codes), slots int32 [n]; float32 scales [N] or [L, N] go with their rows.  Both caches may be the
    same one when no destination is also a source."""
    import torch
    w = "mla_copy_rows"
    _status_word(w, workspace)
    sn, sr, L, nbytes = _layers(w, "src_cache", src_cache, src_scales)
    if dst_cache is src_cache and dst_scales is src_scales:
        dn, dr = sn, sr
    else:
        dn, dr, dl, dbytes = _layers(w, "dst_cache", dst_cache, dst_scales)
        if L != dl or nbytes != dbytes:
            raise ValueError(f"{w}: the caches differ in layers or type")
        if (src_scales is None) != (dst_scales is None):
            raise ValueError(f"{w}: src_scales goes with dst_scales")
    n = _sizes(w, "src_slots", src_slots, 1)[0]
    _need(w, "src_slots", src_slots, torch.int32, (n,))
    _need(w, "dst_slots", dst_slots, torch.int32, (n,))
    st = _launch_stream(w, stream, src_cache, src_slots, dst_cache, dst_slots, src_scales, dst_scales, workspace)
    if n and (not sn or not dn):
        raise ValueError(f"{w}: a cache has no slots")
    st = _lib.mla_copy_rows(src_cache.data_ptr(), _ptr(src_scales), sn, sr, src_slots.data_ptr(), dst_cache.data_ptr(),
                            _ptr(dst_scales), dn, dr, dst_slots.data_ptr(), n, L, nbytes, _ptr(workspace), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def compact_cache(kv_cache, kv_indptr, kv_indices, new_indices, live_count, workspace, kv_scales=None,
                  stream=None) -> None:
    """Move the rows that kv_indices[: kv_indptr[-1]] names into the lowest slots, in every layer, and rewrite the
    lists into new_indices (kv_indices itself will do): kv_cache [N, 576] or [L, N, 576], live_count int32 [1] takes
    the number of live slots, workspace of slots_workspace_bytes(N) bytes."""
    import torch
    w, i32 = "mla_compact_cache", torch.int32
    N, rows, L, nbytes = _layers(w, "kv_cache", kv_cache, kv_scales)
    B1 = _sizes(w, "kv_indptr", kv_indptr, 1)[0]
    if B1 < 1:
        raise ValueError(f"{w}: kv_indptr must hold batch + 1 entries")
    n = kv_indices.numel()
    _need(w, "kv_indptr", kv_indptr, i32, (B1,))
    _need(w, "kv_indices", kv_indices, i32, (n,))
    _need(w, "new_indices", new_indices, i32, (n,))
    _need(w, "live_count", live_count, i32, (1,))
    _need(w, "workspace", workspace, torch.uint8, (workspace.numel(),))
    st = _launch_stream(w, stream, kv_cache, kv_indptr, kv_indices, new_indices, live_count, workspace, kv_scales)
    st = _lib.mla_compact_cache(kv_cache.data_ptr(), _ptr(kv_scales), N, rows, L, nbytes, kv_indptr.data_ptr(), B1 - 1,
                                kv_indices.data_ptr(), n, new_indices.data_ptr(), live_count.data_ptr(),
                                workspace.data_ptr(), workspace.numel(), st)
    if st != MLA_OK:
        raise MLAError(st, w)


def check_errors(workspace, stream=None) -> int:
    """Synchronise, read and clear the device status; returns the status code."""
    return int(_lib.mla_check_errors(_ptr(workspace), _stream_handle(stream)))


def probe_wait_limit(workspace, stream=None) -> None:
    """Launch the bounded-wait diagnostic: a wait that nothing completes gives up
    after the kernels' wait limit and leaves MLA_ERR_TIMEOUT in the status word."""
    st = _lib.mla_probe_wait_limit(_ptr(workspace), _stream_handle(stream))
    if st != MLA_OK:
        raise MLAError(st, "mla_probe_wait_limit")


class Decoder:
    """Convenience holder: plan once per batch shape, then run on device tensors."""

    def __init__(self, kv_indptr_host, num_heads: int, device="cuda", num_sms: int = 0):
        import torch
        self.plan_host, self.workspace_bytes = decode_plan(kv_indptr_host, num_heads, num_sms)
        self.plan_dev = torch.from_numpy(self.plan_host).to(device)
        self.workspace = torch.zeros(max(self.workspace_bytes, 256), dtype=torch.uint8, device=device)
        self.num_heads = num_heads
        self.batch = int(np.asarray(kv_indptr_host).shape[0]) - 1
        self.nnz = int(np.asarray(kv_indptr_host)[-1])

    @property
    def header(self):
        return self.plan_host[:16]

    def run(self, q_nope, q_rope, kv_cache, kv_indptr, kv_indices, sm_scale, out, lse, stream=None):
        decode_run(self.plan_host, self.plan_dev, q_nope, q_rope, kv_cache, kv_indptr, kv_indices,
                   sm_scale, out, lse, self.workspace, stream)

    def attend(self, q_nope, q_rope, kv_cache, kv_indptr, kv_indices, sm_scale, out, lse, stream=None):
        decode_attend(self.plan_host, self.plan_dev, q_nope, q_rope, kv_cache, kv_indptr, kv_indices,
                      sm_scale, out, lse, self.workspace, stream)

    def merge(self, out, lse, stream=None):
        decode_merge(self.plan_host, self.plan_dev, out, lse, self.workspace, stream)

    @property
    def has_merge(self) -> bool:
        return int(self.plan_host[10]) > 0

    def check(self, stream=None) -> int:
        return check_errors(self.workspace, stream)


class Prefiller:
    """Convenience holder: plan a batch's prompt attention once, then run it on device tensors.  Ready on every stream
    once it is made; its runs share one workspace, so they follow one another (on one stream, or ordered by events).  It
    may be dropped while a torch stream still runs it; one made elsewhere (a handle, an ExternalStream) has to be done."""

    def __init__(self, q_indptr_host, kv_indptr_host, num_heads: int, causal: bool = True, device="cuda",
                 num_sms: int = 0):
        import torch
        self.plan_host, self.workspace_bytes = prefill_plan(q_indptr_host, kv_indptr_host, num_heads, causal, num_sms)
        self.plan_dev = torch.from_numpy(self.plan_host).to(device)
        self.workspace = torch.zeros(self.workspace_bytes, dtype=torch.uint8, device=device)
        home = torch.cuda.current_stream(self.workspace.device)
        home.synchronize()                           # a run on another stream does not wait for the zeros
        self._streams = {home.cuda_stream}

    def run(self, q, k_nope, k_rope, v, sm_scale, out, lse=None, stream=None):
        cur, handle = _current(stream)
        if handle not in self._streams:
            import torch
            where = torch.cuda.current_stream(cur) if stream is None else stream
            # The allocator keeps plan and workspace until a stream of torch's own is done with them.  It may not be told
            # of a stream that others made (torch numbers it by its handle): that may be gone when they are freed.
            if isinstance(where, torch.cuda.Stream) and (handle == 0 or where.stream_id != handle):
                for t in (self.plan_dev, self.workspace):
                    t.record_stream(where)
            self._streams.add(handle)
        prefill_run(self.plan_host, self.plan_dev, q, k_nope, k_rope, v, sm_scale, out, lse, self.workspace, handle)

    def check(self, stream=None) -> int:
        return check_errors(self.workspace, stream)
