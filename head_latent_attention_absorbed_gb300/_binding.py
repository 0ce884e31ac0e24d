"""ctypes binding of the C ABI in ``include/mla.h``.

Argument marshalling only: every step of the decode runs in the CUDA library.
Tensors are torch tensors on a CUDA device (PyTorch provides device memory and
streams); their data pointers, sizes and the current stream are passed through.
If the shared library is missing the calls raise: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmla_gb300.so")
CHECK_LIB_PATH = os.path.join(PKG, "libmla_gb300_check.so")   # the checked build

MLA_F32, MLA_BF16, MLA_FP8_E4M3 = 0, 1, 2
MLA_DEV_LENGTH_OUT_OF_RANGE = 1
MLA_DEV_PIPELINE_TIMEOUT = 2
MLA_DEV_BOUNDS = 4
MLA_DEV_PAGE_OUT_OF_RANGE = 8
MLA_DEV_POOL_EXHAUSTED = 16
STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED",
          3: "MLA_ERR_WORKSPACE", 4: "MLA_ERR_CUDA"}
EXPORTED = ("mla_absorb_q", "mla_decode_num_splits", "mla_decode_workspace_bytes",
            "mla_decode_attn", "mla_decode_split", "mla_decode_combine",
            "mla_decode_attn_noalloc", "mla_decode_attn_multi", "mla_decode_multi_num_splits",
            "mla_decode_multi_workspace_bytes", "mla_decode_step", "mla_decode_step_multi",
            "mla_out_proj", "mla_cache_append",
            "mla_wo_proj", "mla_materialize_wkq", "mla_materialize_wov",
            "mla_absorb_q_materialized", "mla_ov_proj",
            "mla_status_string", "mla_last_error_message", "mla_test_set_split_hooks",
            "mla_set_launch_overlap", "mla_decode_plan", "mla_test_set_split_debug",
            "mla_test_set_split_form", "mla_built_with_checks", "mla_debug_bounds_word",
            "mla_set_split_parts", "mla_decode_heads_per_cta",
            "mla_pages_extend", "mla_pages_release", "mla_cache_append_paged",
            "mla_paged_num_splits", "mla_paged_workspace_bytes", "mla_decode_attn_paged",
            "mla_page_index", "mla_select_workspace_bytes", "mla_select_pages",
            "mla_sparse_workspace_bytes", "mla_decode_attn_sparse")


class MlaDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("d_c", ctypes.c_int32),
                ("d_rope", ctypes.c_int32), ("d_nope", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("s_max", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class MlaPaging(ctypes.Structure):
    _fields_ = [("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("table_stride", ctypes.c_int32)]


class MlaError(RuntimeError):
    def __init__(self, code: int, detail: str):
        super().__init__(f"{STATUS.get(code, code)}: {detail}")
        self.code = code


_lib = None


def load(path: Optional[str] = None):
    """Load the shared library (once) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library {p} is not built; run __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(MlaDims)
    lib.mla_absorb_q.argtypes = [D, P, P, P, P, ctypes.c_double, P, P, P]
    lib.mla_absorb_q.restype = ctypes.c_int
    lib.mla_decode_num_splits.argtypes = [D, I32]
    lib.mla_decode_num_splits.restype = I32
    lib.mla_decode_workspace_bytes.argtypes = [D, I32]
    lib.mla_decode_workspace_bytes.restype = SZ
    lib.mla_decode_attn.argtypes = [D, P, P, P, P, ctypes.c_float, I32, P, SZ, P, P, P, P]
    lib.mla_decode_attn.restype = ctypes.c_int
    lib.mla_decode_split.argtypes = [D, P, P, P, P, ctypes.c_float, I32, P, SZ, P, P]
    lib.mla_decode_split.restype = ctypes.c_int
    lib.mla_decode_combine.argtypes = [D, P, I32, P, SZ, P, P, P]
    lib.mla_decode_combine.restype = ctypes.c_int
    lib.mla_decode_attn_multi.argtypes = [D, I32, P, P, P, P, ctypes.c_float, I32, P, SZ, P, P, P,
                                          P]
    lib.mla_decode_attn_multi.restype = ctypes.c_int
    lib.mla_decode_multi_num_splits.argtypes = [D, I32, I32]
    lib.mla_decode_multi_num_splits.restype = I32
    lib.mla_decode_multi_workspace_bytes.argtypes = [D, I32, I32]
    lib.mla_decode_multi_workspace_bytes.restype = SZ
    lib.mla_decode_attn_noalloc.argtypes = [D, P, P, P, P, ctypes.c_float, I32, P, P, P, P]
    lib.mla_decode_attn_noalloc.restype = ctypes.c_int
    lib.mla_decode_step.argtypes = [D, P, P, P, P, ctypes.c_double, P, P, ctypes.c_float, I32, P,
                                    P, SZ, P, P, P, P, P, P, P]
    lib.mla_decode_step.restype = ctypes.c_int
    lib.mla_decode_step_multi.argtypes = [D, I32, P, P, P, P, ctypes.c_double, P, P, ctypes.c_float,
                                          I32, P, P, SZ, P, P, P, P, P, P, P]
    lib.mla_decode_step_multi.restype = ctypes.c_int
    lib.mla_cache_append.argtypes = [D, I32, P, P, P, ctypes.c_double, P, P, P]
    lib.mla_cache_append.restype = ctypes.c_int
    lib.mla_wo_proj.argtypes = [D, I32, P, P, P, P]
    lib.mla_wo_proj.restype = ctypes.c_int
    lib.mla_materialize_wkq.argtypes = [D, I32, P, P, P, P]
    lib.mla_materialize_wkq.restype = ctypes.c_int
    lib.mla_materialize_wov.argtypes = [D, I32, P, P, P, P]
    lib.mla_materialize_wov.restype = ctypes.c_int
    lib.mla_absorb_q_materialized.argtypes = [D, I32, P, P, P, P, ctypes.c_double, P, P, P]
    lib.mla_absorb_q_materialized.restype = ctypes.c_int
    lib.mla_ov_proj.argtypes = [D, I32, P, P, P, P]
    lib.mla_ov_proj.restype = ctypes.c_int
    lib.mla_out_proj.argtypes = [D, P, P, P, P]
    lib.mla_out_proj.restype = ctypes.c_int
    lib.mla_status_string.argtypes = [ctypes.c_int]
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_last_error_message.argtypes = []
    lib.mla_last_error_message.restype = ctypes.c_char_p
    lib.mla_test_set_split_hooks.argtypes = [ctypes.c_uint64, I32]
    lib.mla_test_set_split_hooks.restype = None
    lib.mla_set_launch_overlap.argtypes = [I32]
    lib.mla_set_launch_overlap.restype = None
    lib.mla_test_set_split_debug.argtypes = [P]
    lib.mla_test_set_split_debug.restype = None
    lib.mla_test_set_split_form.argtypes = [I32]
    lib.mla_test_set_split_form.restype = None
    lib.mla_set_split_parts.argtypes = [I32]
    lib.mla_set_split_parts.restype = ctypes.c_int
    lib.mla_decode_heads_per_cta.argtypes = [D]
    lib.mla_decode_heads_per_cta.restype = I32
    lib.mla_built_with_checks.argtypes = []
    lib.mla_built_with_checks.restype = I32
    lib.mla_debug_bounds_word.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
    lib.mla_debug_bounds_word.restype = ctypes.c_int
    lib.mla_decode_plan.argtypes = [D, I32, ctypes.POINTER(I32), ctypes.POINTER(I32),
                                    ctypes.POINTER(I32)]
    lib.mla_decode_plan.restype = ctypes.c_int
    G = ctypes.POINTER(MlaPaging)
    F = ctypes.c_float
    lib.mla_pages_extend.argtypes = [I32, G, P, P, I32, P, P, P, P, P, P, P, P, P, P]
    lib.mla_pages_extend.restype = ctypes.c_int
    lib.mla_pages_release.argtypes = [I32, G, P, P, P, P, P, P, P]
    lib.mla_pages_release.restype = ctypes.c_int
    lib.mla_cache_append_paged.argtypes = [D, G, I32, I32, P, P, P, ctypes.c_double, P, P, P]
    lib.mla_cache_append_paged.restype = ctypes.c_int
    lib.mla_paged_num_splits.argtypes = [D, G, I32, I32, I32]
    lib.mla_paged_num_splits.restype = I32
    lib.mla_paged_workspace_bytes.argtypes = [D, G, I32, I32, I32]
    lib.mla_paged_workspace_bytes.restype = SZ
    lib.mla_decode_attn_paged.argtypes = [D, G, I32, I32, P, P, P, P, P, F, I32, P, SZ, P, P, P, P]
    lib.mla_decode_attn_paged.restype = ctypes.c_int
    lib.mla_page_index.argtypes = [D, G, I32, P, P, P, P, P, P, P, P]
    lib.mla_page_index.restype = ctypes.c_int
    lib.mla_select_workspace_bytes.argtypes = [D, G, I32]
    lib.mla_select_workspace_bytes.restype = SZ
    lib.mla_select_pages.argtypes = [D, G, I32, I32, P, P, P, P, P, P, I32, I32, I32, P, SZ, P, P,
                                     P, P]
    lib.mla_select_pages.restype = ctypes.c_int
    lib.mla_sparse_workspace_bytes.argtypes = [D, G, I32, I32, I32, I32]
    lib.mla_sparse_workspace_bytes.restype = SZ
    lib.mla_decode_attn_sparse.argtypes = [D, G, I32, I32, P, P, P, P, P, P, P, F, I32, I32, I32,
                                           I32, P, SZ, P, P, P, P, P, P]
    lib.mla_decode_attn_sparse.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def set_launch_overlap(enable: bool) -> None:
    """Programmatic dependent launch on (default) or off for later launches."""
    load().mla_set_launch_overlap(1 if enable else 0)


def set_split_parts(parts: int) -> None:
    """0: the library's choice (one bf16 part of the query and P at multiples of
    64 heads); 2: hi + lo parts everywhere."""
    _check(load().mla_set_split_parts(int(parts)))


def heads_per_cta(d: "MlaDims") -> int:
    """Heads per split CTA under the current set_split_parts (64: one part)."""
    return int(load().mla_decode_heads_per_cta(ctypes.byref(d)))


def _check(code: int):
    if code != 0:
        raise MlaError(code, load().mla_last_error_message().decode())


def dims(batch: int, heads: int, s_max: int, dtype: int, d_c: int = 512, d_rope: int = 64,
         d_nope: int = 128, d_v: int = 128) -> MlaDims:
    return MlaDims(batch, heads, d_c, d_rope, d_nope, d_v, s_max, dtype)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream) -> int:
    """The raw cudaStream_t of ``stream``, default the current device's current
    stream (read without building a torch.cuda.Stream object: that costs a few
    microseconds per call, as much as a kernel launch)."""
    import torch
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def dtype_code(torch_dtype) -> int:
    import torch
    if torch_dtype == torch.bfloat16:
        return MLA_BF16
    if torch_dtype == torch.float32:
        return MLA_F32
    if torch_dtype == torch.float8_e4m3fn:   # an E4M3 cache; queries and weights bf16
        return MLA_FP8_E4M3
    raise TypeError(f"unsupported dtype {torch_dtype}")


def _require(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _cuda_contig(*ts):
    for t in ts:
        if t is not None:
            _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")


def _cuda_or_pinned(*ts):
    for t in ts:
        if t is not None:
            _require(t.is_contiguous() and (t.is_cuda or t.is_pinned()),
                     "tensors must be contiguous CUDA tensors or pinned host tensors")


def num_splits(d: MlaDims, requested: int = 0) -> int:
    return int(load().mla_decode_num_splits(ctypes.byref(d), int(requested)))


def plan(d: MlaDims, requested: int = 0):
    """(splits, chunk rows, persistent) of the split for `requested` chunks."""
    sp, ch, pe = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(load().mla_decode_plan(ctypes.byref(d), int(requested), ctypes.byref(sp),
                                  ctypes.byref(ch), ctypes.byref(pe)))
    return sp.value, ch.value, bool(pe.value)


def workspace_bytes(d: MlaDims, requested: int = 0) -> int:
    return int(load().mla_decode_workspace_bytes(ctypes.byref(d), int(requested)))


def absorb_q(d: MlaDims, q_nope, q_rope, w_uk, positions, q_abs, q_pe, rope_base: float = 10000.0,
             stream=None) -> None:
    """q_abs = q_nope . W_UK per head; q_pe = RoPE(q_rope, positions)."""
    _cuda_contig(q_nope, q_rope, w_uk, positions, q_abs, q_pe)
    _check(load().mla_absorb_q(ctypes.byref(d), _ptr(q_nope), _ptr(q_rope), _ptr(w_uk),
                               _ptr(positions), float(rope_base), _ptr(q_abs), _ptr(q_pe),
                               _stream(stream)))


def decode_attn(d: MlaDims, q_abs, q_pe, cache, lengths, o_c, workspace, softmax_scale: float,
                num_splits_requested: int = 0, lse=None, dev_status=None, stream=None) -> None:
    """Split-KV attention over the latent cache followed by the LSE combine."""
    _cuda_contig(q_abs, q_pe, cache, lengths, o_c, workspace, lse, dev_status)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().mla_decode_attn(ctypes.byref(d), _ptr(q_abs), _ptr(q_pe), _ptr(cache),
                                  _ptr(lengths), float(softmax_scale), int(num_splits_requested),
                                  _ptr(workspace), nbytes, _ptr(o_c), _ptr(lse),
                                  _ptr(dev_status), _stream(stream)))


def decode_split(d: MlaDims, q_abs, q_pe, cache, lengths, workspace, softmax_scale: float,
                 num_splits_requested: int = 0, dev_status=None, stream=None) -> None:
    """First half of decode_attn: per-chunk partial outputs into the workspace."""
    _cuda_contig(q_abs, q_pe, cache, lengths, workspace, dev_status)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().mla_decode_split(ctypes.byref(d), _ptr(q_abs), _ptr(q_pe), _ptr(cache),
                                   _ptr(lengths), float(softmax_scale),
                                   int(num_splits_requested), _ptr(workspace), nbytes,
                                   _ptr(dev_status), _stream(stream)))


def decode_combine(d: MlaDims, lengths, workspace, o_c, num_splits_requested: int = 0, lse=None,
                   stream=None) -> None:
    """Second half of decode_attn: log-sum-exp merge of the chunk partials."""
    _cuda_contig(lengths, workspace, o_c, lse)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().mla_decode_combine(ctypes.byref(d), _ptr(lengths), int(num_splits_requested),
                                     _ptr(workspace), nbytes, _ptr(o_c), _ptr(lse),
                                     _stream(stream)))


def query_dims(d: MlaDims, q_len: int) -> MlaDims:
    """The dims of the query side of a q_len-token step: batch B * q_len."""
    return MlaDims(d.batch * q_len, d.heads, d.d_c, d.d_rope, d.d_nope, d.d_v, d.s_max, d.dtype)


def multi_num_splits(d: MlaDims, q_len: int, requested: int = 0) -> int:
    """Chunks per sequence that decode_attn_multi uses (d: the cache's dims)."""
    return int(load().mla_decode_multi_num_splits(ctypes.byref(d), int(q_len), int(requested)))


def multi_workspace_bytes(d: MlaDims, q_len: int, requested: int = 0) -> int:
    """Workspace bytes decode_attn_multi needs (d: the cache's dims)."""
    return int(load().mla_decode_multi_workspace_bytes(ctypes.byref(d), int(q_len),
                                                       int(requested)))


def decode_attn_multi(d: MlaDims, q_len: int, q_abs, q_pe, cache, lengths, o_c, workspace,
                      softmax_scale: float, num_splits_requested: int = 0, lse=None,
                      dev_status=None, stream=None) -> None:
    """decode_attn for q_len new tokens per sequence, causal within the block.

    ``d`` describes the cache (B sequences); q_abs, q_pe, o_c and lse have
    B * q_len rows (row b * q_len + i is token i of sequence b).
    """
    _cuda_contig(q_abs, q_pe, cache, lengths, o_c, workspace, lse, dev_status)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().mla_decode_attn_multi(ctypes.byref(d), int(q_len), _ptr(q_abs), _ptr(q_pe),
                                        _ptr(cache), _ptr(lengths), float(softmax_scale),
                                        int(num_splits_requested), _ptr(workspace), nbytes,
                                        _ptr(o_c), _ptr(lse), _ptr(dev_status),
                                        _stream(stream)))


def decode_attn_noalloc(d: MlaDims, q_abs, q_pe, cache, lengths, o_c, softmax_scale: float,
                        num_splits_requested: int = 0, lse=None, dev_status=None,
                        stream=None) -> None:
    """decode_attn with the library's fixed scratch in place of a workspace.

    For hosts that cannot allocate device memory while decoding; the call
    allocates nothing.  Calls that overlap on the GPU share that scratch and race.
    """
    _cuda_contig(q_abs, q_pe, cache, lengths, o_c, lse, dev_status)
    _check(load().mla_decode_attn_noalloc(ctypes.byref(d), _ptr(q_abs), _ptr(q_pe), _ptr(cache),
                                          _ptr(lengths), float(softmax_scale),
                                          int(num_splits_requested), _ptr(o_c), _ptr(lse),
                                          _ptr(dev_status), _stream(stream)))


def decode_step(d: MlaDims, q_nope, q_rope, w_uk, positions, cache, lengths, w_uv, workspace,
                q_abs, q_pe, o_c, out, softmax_scale: float, rope_base: float = 10000.0,
                num_splits_requested: int = 0, lse=None, dev_status=None, stream=None) -> None:
    """absorb_q, decode_attn and out_proj in one call (bf16: fused combine + W_UV).

    q_nope, q_rope, positions, lengths and out may be pinned host tensors: the
    kernels then read and write them over the host link, with no copies.
    """
    _cuda_contig(w_uk, cache, w_uv, workspace, q_abs, q_pe, o_c, lse, dev_status)
    _cuda_or_pinned(q_nope, q_rope, positions, lengths, out)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().mla_decode_step(ctypes.byref(d), _ptr(q_nope), _ptr(q_rope), _ptr(w_uk),
                                  _ptr(positions), float(rope_base), _ptr(cache), _ptr(lengths),
                                  float(softmax_scale), int(num_splits_requested), _ptr(w_uv),
                                  _ptr(workspace), nbytes, _ptr(q_abs), _ptr(q_pe), _ptr(o_c),
                                  _ptr(lse), _ptr(out), _ptr(dev_status), _stream(stream)))


def decode_step_multi(d: MlaDims, q_len: int, q_nope, q_rope, w_uk, positions, cache, lengths,
                      w_uv, workspace, q_abs, q_pe, o_c, out, softmax_scale: float,
                      rope_base: float = 10000.0, num_splits_requested: int = 0, lse=None,
                      dev_status=None, stream=None) -> None:
    """decode_step for q_len tokens per sequence (d: the cache's dims; the query
    side has B * q_len rows).  The step's inputs and out may be pinned host tensors."""
    _cuda_contig(w_uk, cache, w_uv, workspace, q_abs, q_pe, o_c, lse, dev_status)
    _cuda_or_pinned(q_nope, q_rope, positions, lengths, out)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().mla_decode_step_multi(ctypes.byref(d), int(q_len), _ptr(q_nope), _ptr(q_rope),
                                        _ptr(w_uk), _ptr(positions), float(rope_base),
                                        _ptr(cache), _ptr(lengths), float(softmax_scale),
                                        int(num_splits_requested), _ptr(w_uv), _ptr(workspace),
                                        nbytes, _ptr(q_abs), _ptr(q_pe), _ptr(o_c), _ptr(lse),
                                        _ptr(out), _ptr(dev_status), _stream(stream)))


def step_call(d: MlaDims, q_len: int, q_nope, q_rope, w_uk, positions, cache, lengths, w_uv,
              workspace, q_abs, q_pe, o_c, out, softmax_scale: float, rope_base: float,
              num_splits_requested: int, lse, dev_status):
    """The checked arguments of mla_decode_step (q_len 1) or mla_decode_step_multi,
    converted once: returns (function, arguments without the stream), for callers
    that make the same call every step (HostStep.launch).  The tensors must stay
    alive and in place while the arguments are used."""
    _cuda_contig(w_uk, cache, w_uv, workspace, q_abs, q_pe, o_c, lse, dev_status)
    _cuda_or_pinned(q_nope, q_rope, positions, lengths, out)
    nbytes = workspace.numel() * workspace.element_size()
    lib = load()
    tail = (_ptr(q_nope), _ptr(q_rope), _ptr(w_uk), _ptr(positions), float(rope_base),
            _ptr(cache), _ptr(lengths), float(softmax_scale), int(num_splits_requested),
            _ptr(w_uv), _ptr(workspace), nbytes, _ptr(q_abs), _ptr(q_pe), _ptr(o_c), _ptr(lse),
            _ptr(out), _ptr(dev_status))
    if q_len == 1:
        return lib.mla_decode_step, (ctypes.byref(d),) + tail
    return lib.mla_decode_step_multi, (ctypes.byref(d), int(q_len)) + tail


def out_proj(d: MlaDims, o_c, w_uv, out, stream=None) -> None:
    """o = W_UV . o_c per head."""
    _cuda_contig(o_c, w_uv, out)
    _check(load().mla_out_proj(ctypes.byref(d), _ptr(o_c), _ptr(w_uv), _ptr(out), _stream(stream)))


def cache_append(d: MlaDims, x, w_kva, positions, cache, rope_base: float = 10000.0,
                 dev_status=None, stream=None) -> None:
    """Write the new token of each sequence into the cache at positions[b]."""
    _cuda_contig(x, w_kva, positions, cache, dev_status)
    _check(load().mla_cache_append(ctypes.byref(d), int(x.shape[-1]), _ptr(x), _ptr(w_kva),
                                   _ptr(positions), float(rope_base), _ptr(cache),
                                   _ptr(dev_status), _stream(stream)))


def wo_proj(d: MlaDims, o, w_o, y, stream=None) -> None:
    """y = concat_h(o[:, h, :]) . W_O^T."""
    _cuda_contig(o, w_o, y)
    _check(load().mla_wo_proj(ctypes.byref(d), int(w_o.shape[0]), _ptr(o), _ptr(w_o), _ptr(y),
                              _stream(stream)))


def materialize_wkq(d: MlaDims, w_q_nope, w_uk, w_kq, stream=None) -> None:
    """W^KQ[h*512 + c, i] = sum_d w_uk[h, d, c] w_q_nope[h, d, i] (once per model)."""
    _cuda_contig(w_q_nope, w_uk, w_kq)
    _check(load().mla_materialize_wkq(ctypes.byref(d), int(w_q_nope.shape[-1]), _ptr(w_q_nope),
                                      _ptr(w_uk), _ptr(w_kq), _stream(stream)))


def materialize_wov(d: MlaDims, w_o, w_uv, w_ov, stream=None) -> None:
    """W^OV[n, h*512 + c] = sum_e w_o[n, h*128 + e] w_uv[h, e, c] (once per model)."""
    _cuda_contig(w_o, w_uv, w_ov)
    _check(load().mla_materialize_wov(ctypes.byref(d), int(w_o.shape[0]), _ptr(w_o), _ptr(w_uv),
                                      _ptr(w_ov), _stream(stream)))


def absorb_q_materialized(d: MlaDims, x, w_kq, q_rope, positions, q_abs, q_pe,
                          rope_base: float = 10000.0, stream=None) -> None:
    """q_abs = W^KQ x per head; q_pe = RoPE(q_rope, positions)."""
    _cuda_contig(x, w_kq, q_rope, positions, q_abs, q_pe)
    _check(load().mla_absorb_q_materialized(ctypes.byref(d), int(x.shape[-1]), _ptr(x),
                                            _ptr(w_kq), _ptr(q_rope), _ptr(positions),
                                            float(rope_base), _ptr(q_abs), _ptr(q_pe),
                                            _stream(stream)))


def ov_proj(d: MlaDims, o_c, w_ov, y, stream=None) -> None:
    """y = W^OV . concat_h(o_c[:, h, :])."""
    _cuda_contig(o_c, w_ov, y)
    _check(load().mla_ov_proj(ctypes.byref(d), int(w_ov.shape[0]), _ptr(o_c), _ptr(w_ov), _ptr(y),
                              _stream(stream)))


# ------------------------------------------------------------------- paged cache
#
# The paged calls check every tensor they hand over (device, layout, type, size):
# a wrong table or slot type would send a kernel outside its buffers.  The checks
# are spelled out in one expression per call, since a small call takes less time
# on the GPU than a loop of checks takes here (a decode step's block tables: 12 us
# of host time with a helper call per tensor, 7 us so); only a call that fails
# them goes through _explain for a message.

def paging(page_size: int, num_pages: int, table_stride: int) -> MlaPaging:
    """The pool's shape: rows per page, pages, and entries per block-table row."""
    return MlaPaging(page_size, num_pages, table_stride)


_I32 = _I64 = _I8 = _F32 = _BF16 = _ROW_TYPE = None
_device = _raw_stream = None


def _paged_lib():
    """The library; the first call fetches what the checks compare with."""
    global _I32, _I64, _I8, _F32, _BF16, _ROW_TYPE, _device, _raw_stream
    if _device is None:
        import torch
        _I32, _I64, _I8 = torch.int32, torch.int64, torch.int8
        _F32, _BF16 = torch.float32, torch.bfloat16
        _ROW_TYPE = {MLA_F32: torch.float32, MLA_BF16: torch.bfloat16,
                     MLA_FP8_E4M3: torch.float8_e4m3fn}
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _device = torch._C._cuda_getDevice
    return _lib if _lib is not None else load()


def _stream_on(dev: int, stream) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _explain(dev: int, **want):
    """Raises the ValueError of the first tensor that is not as wanted:
    name=(tensor, dtype, number of values)."""
    for name, (t, dtype, numel) in want.items():
        if t is None:
            continue
        _require(t.is_cuda and t.get_device() == dev,
                 f"{name} must be a CUDA tensor on the current device")
        _require(t.is_contiguous(), f"{name} must be contiguous")
        _require(t.dtype == dtype, f"{name} must be {dtype}, not {t.dtype}")
        _require(numel < 0 or t.numel() == numel, f"{name} must hold {numel} values, not {t.numel()}")
    raise ValueError("a tensor of this call is not as documented")


def _is(t, dev, dtype, numel) -> bool:
    return (t.get_device() == dev and t.dtype is dtype and t.numel() == numel
            and t.is_contiguous())


def _io_code(torch_dtype) -> int:
    """Query and output type of the paged calls."""
    _paged_lib()
    _require(torch_dtype is _BF16 or torch_dtype is _F32, "queries must be fp32 or bf16")
    return MLA_BF16 if torch_dtype is _BF16 else MLA_F32


def pages_extend(pg: MlaPaging, cached_lens, new_lens, block_table, free_list, num_free, lengths,
                 row_starts, slots, positions, num_free_out=None, dev_status=None,
                 stream=None) -> None:
    """Block tables and slot maps of one step from the requests' lengths.

    Takes pages from the free stack for the rows that new_lens adds, and writes
    lengths, row_starts, slots and positions (padded to slots.numel() with -1 and
    0).  All or nothing: see mla_pages_extend.  ``num_free`` is updated in place
    unless ``num_free_out`` is given.
    """
    lib = _paged_lib()
    dev, i32 = _device(), _I32
    out = num_free if num_free_out is None else num_free_out
    B, n = cached_lens.numel(), slots.numel()
    pages = pg.num_pages
    if not (cached_lens.get_device() == new_lens.get_device() == block_table.get_device()
            == free_list.get_device() == num_free.get_device() == out.get_device()
            == lengths.get_device() == row_starts.get_device() == slots.get_device()
            == positions.get_device() == dev
            and cached_lens.dtype is i32 and new_lens.dtype is i32 and block_table.dtype is i32
            and free_list.dtype is i32 and num_free.dtype is i32 and out.dtype is i32
            and lengths.dtype is i32 and row_starts.dtype is i32 and slots.dtype is _I64
            and positions.dtype is i32
            and new_lens.numel() == B and lengths.numel() == B and row_starts.numel() == B + 1
            and positions.numel() == n and free_list.numel() == pages and num_free.numel() == 1
            and out.numel() == 1 and block_table.numel() == B * pg.table_stride
            and cached_lens.is_contiguous() and new_lens.is_contiguous()
            and block_table.is_contiguous() and free_list.is_contiguous()
            and lengths.is_contiguous() and row_starts.is_contiguous() and slots.is_contiguous()
            and positions.is_contiguous()
            and (dev_status is None or _is(dev_status, dev, i32, 1))):
        _explain(dev, cached_lens=(cached_lens, i32, B), new_lens=(new_lens, i32, B),
                 block_table=(block_table, i32, B * pg.table_stride),
                 free_list=(free_list, i32, pages), num_free=(num_free, i32, 1),
                 num_free_out=(out, i32, 1), lengths=(lengths, i32, B),
                 row_starts=(row_starts, i32, B + 1), slots=(slots, _I64, n),
                 positions=(positions, i32, n), dev_status=(dev_status, i32, 1))
    code = lib.mla_pages_extend(
        B, pg, cached_lens.data_ptr(), new_lens.data_ptr(), n, block_table.data_ptr(),
        free_list.data_ptr(), num_free.data_ptr(), out.data_ptr(), lengths.data_ptr(),
        row_starts.data_ptr(), slots.data_ptr(), positions.data_ptr(),
        None if dev_status is None else dev_status.data_ptr(), _stream_on(dev, stream))
    if code:
        _check(code)


def pages_release(pg: MlaPaging, finished, lengths, block_table, free_list, num_free,
                  dev_status=None, stream=None) -> None:
    """Push the pages of the requests with finished[b] != 0 back on the free stack."""
    lib = _paged_lib()
    dev, i32, B = _device(), _I32, finished.numel()
    if not (_is(finished, dev, i32, B) and _is(lengths, dev, i32, B)
            and _is(block_table, dev, i32, B * pg.table_stride)
            and _is(free_list, dev, i32, pg.num_pages) and _is(num_free, dev, i32, 1)
            and (dev_status is None or _is(dev_status, dev, i32, 1))):
        _explain(dev, finished=(finished, i32, B), lengths=(lengths, i32, B),
                 block_table=(block_table, i32, B * pg.table_stride),
                 free_list=(free_list, i32, pg.num_pages), num_free=(num_free, i32, 1),
                 dev_status=(dev_status, i32, 1))
    code = lib.mla_pages_release(B, pg, finished.data_ptr(), lengths.data_ptr(),
                                 block_table.data_ptr(), free_list.data_ptr(),
                                 num_free.data_ptr(),
                                 None if dev_status is None else dev_status.data_ptr(),
                                 _stream_on(dev, stream))
    if code:
        _check(code)


def cache_append_paged(d: MlaDims, pg: MlaPaging, rows, positions, slots, cache,
                       rope_base: float = 10000.0, dev_status=None, stream=None) -> None:
    """Write latent rows [n, 576] (fp32 or bf16) into their slots, the RoPE key
    rotated at its position; a slot of -1 is skipped."""
    lib = _paged_lib()
    dev, n, row, kind = _device(), slots.numel(), d.d_c + d.d_rope, rows.dtype
    ct, cn = _ROW_TYPE.get(d.dtype), pg.num_pages * pg.page_size * row
    if not (rows.get_device() == positions.get_device() == slots.get_device()
            == cache.get_device() == dev
            and (kind is _BF16 or kind is _F32) and positions.dtype is _I32
            and slots.dtype is _I64 and cache.dtype is ct
            and rows.numel() == n * row and positions.numel() == n and cache.numel() == cn
            and rows.is_contiguous() and positions.is_contiguous() and slots.is_contiguous()
            and cache.is_contiguous()
            and (dev_status is None or _is(dev_status, dev, _I32, 1))):
        _explain(dev, rows=(rows, kind if kind is _BF16 else _F32, n * row),
                 positions=(positions, _I32, n), slots=(slots, _I64, n), cache=(cache, ct, cn),
                 dev_status=(dev_status, _I32, 1))
    code = lib.mla_cache_append_paged(
        d, pg, n, MLA_BF16 if kind is _BF16 else MLA_F32, rows.data_ptr(), positions.data_ptr(),
        slots.data_ptr(), rope_base, cache.data_ptr(),
        None if dev_status is None else dev_status.data_ptr(), _stream_on(dev, stream))
    if code:
        _check(code)


def paged_num_splits(d: MlaDims, pg: MlaPaging, io_dtype, q_len: int = 1,
                     requested: int = 0) -> int:
    """Chunks per sequence decode_attn_paged uses for queries of ``io_dtype``."""
    n = int(load().mla_paged_num_splits(d, pg, _io_code(io_dtype), int(q_len), int(requested)))
    _require(n > 0, load().mla_last_error_message().decode())
    return n


def paged_workspace_bytes(d: MlaDims, pg: MlaPaging, io_dtype, q_len: int = 1,
                          requested: int = 0) -> int:
    """Workspace bytes of decode_attn_paged for queries of ``io_dtype``."""
    n = int(load().mla_paged_workspace_bytes(d, pg, _io_code(io_dtype), int(q_len),
                                             int(requested)))
    _require(n > 0, load().mla_last_error_message().decode())
    return n


def decode_attn_paged(d: MlaDims, pg: MlaPaging, q_abs, q_pe, cache, block_table, lengths, o_c,
                      workspace, softmax_scale: float, q_len: int = 1,
                      num_splits_requested: int = 0, lse=None, dev_status=None,
                      stream=None) -> None:
    """decode_attn_multi over a paged cache; q_abs, q_pe and o_c all fp32 or all bf16."""
    lib = _paged_lib()
    dev, io, B, dc, dr = _device(), q_abs.dtype, d.batch, d.d_c, d.d_rope
    rows = B * q_len * d.heads
    ct, cn = _ROW_TYPE.get(d.dtype), pg.num_pages * pg.page_size * (dc + dr)
    if not (q_abs.get_device() == q_pe.get_device() == cache.get_device()
            == block_table.get_device() == lengths.get_device() == o_c.get_device()
            == workspace.get_device() == dev
            and (io is _BF16 or io is _F32) and q_pe.dtype is io and o_c.dtype is io
            and cache.dtype is ct and block_table.dtype is _I32 and lengths.dtype is _I32
            and q_abs.numel() == rows * dc and q_pe.numel() == rows * dr
            and o_c.numel() == rows * dc and cache.numel() == cn
            and block_table.numel() == B * pg.table_stride and lengths.numel() == B
            and q_abs.is_contiguous() and q_pe.is_contiguous() and cache.is_contiguous()
            and block_table.is_contiguous() and lengths.is_contiguous() and o_c.is_contiguous()
            and workspace.is_contiguous()
            and (lse is None or _is(lse, dev, _F32, rows))
            and (dev_status is None or _is(dev_status, dev, _I32, 1))):
        _io_code(io)
        _explain(dev, q_abs=(q_abs, io, rows * dc), q_pe=(q_pe, io, rows * dr),
                 o_c=(o_c, io, rows * dc), cache=(cache, ct, cn),
                 block_table=(block_table, _I32, B * pg.table_stride),
                 lengths=(lengths, _I32, B), workspace=(workspace, workspace.dtype, -1),
                 lse=(lse, _F32, rows), dev_status=(dev_status, _I32, 1))
    code = lib.mla_decode_attn_paged(
        d, pg, MLA_BF16 if io is _BF16 else MLA_F32, q_len, q_abs.data_ptr(), q_pe.data_ptr(),
        cache.data_ptr(), block_table.data_ptr(), lengths.data_ptr(), softmax_scale,
        num_splits_requested, workspace.data_ptr(), workspace.numel() * workspace.itemsize,
        o_c.data_ptr(), None if lse is None else lse.data_ptr(),
        None if dev_status is None else dev_status.data_ptr(), _stream_on(dev, stream))
    if code:
        _check(code)


def page_index(d: MlaDims, pg: MlaPaging, cache, block_table, first_rows, lengths, max_new: int,
               codes, scales, dev_status=None, stream=None) -> None:
    """Index rows (int8 mean row and scale, by page number) of the pages that hold
    rows [first_rows[b], lengths[b]) of each sequence."""
    lib = _paged_lib()
    dev, i32, B, row, pages = _device(), _I32, d.batch, d.d_c + d.d_rope, pg.num_pages
    ct = _ROW_TYPE.get(d.dtype)
    if not (cache.get_device() == block_table.get_device() == first_rows.get_device()
            == lengths.get_device() == codes.get_device() == scales.get_device() == dev
            and cache.dtype is ct and block_table.dtype is i32 and first_rows.dtype is i32
            and lengths.dtype is i32 and codes.dtype is _I8 and scales.dtype is _F32
            and cache.numel() == pages * pg.page_size * row
            and block_table.numel() == B * pg.table_stride and first_rows.numel() == B
            and lengths.numel() == B and codes.numel() == pages * row and scales.numel() == pages
            and cache.is_contiguous() and block_table.is_contiguous()
            and first_rows.is_contiguous() and lengths.is_contiguous() and codes.is_contiguous()
            and scales.is_contiguous()
            and (dev_status is None or _is(dev_status, dev, i32, 1))):
        _explain(dev, cache=(cache, ct, pages * pg.page_size * row),
                 block_table=(block_table, i32, B * pg.table_stride),
                 first_rows=(first_rows, i32, B), lengths=(lengths, i32, B),
                 codes=(codes, _I8, pages * row), scales=(scales, _F32, pages),
                 dev_status=(dev_status, i32, 1))
    code = lib.mla_page_index(
        d, pg, max_new, cache.data_ptr(), block_table.data_ptr(), first_rows.data_ptr(),
        lengths.data_ptr(), codes.data_ptr(), scales.data_ptr(),
        None if dev_status is None else dev_status.data_ptr(), _stream_on(dev, stream))
    if code:
        _check(code)


def select_workspace_bytes(d: MlaDims, pg: MlaPaging, q_len: int = 1) -> int:
    n = int(load().mla_select_workspace_bytes(d, pg, int(q_len)))
    _require(n > 0, load().mla_last_error_message().decode())
    return n


def _check_selection(dev, d, pg, q_abs, q_pe, block_table, lengths, codes, scales, sel_table,
                     sel_lengths, workspace, q_len, dev_status) -> int:
    """The checks select_pages and decode_attn_sparse share; returns io_dtype."""
    i32, io, B, dc, dr, pages = _I32, q_abs.dtype, d.batch, d.d_c, d.d_rope, pg.num_pages
    R = B * q_len
    rows = R * d.heads
    top = sel_table.shape[1] if sel_table.dim() == 2 else -1
    if not (q_abs.get_device() == q_pe.get_device() == block_table.get_device()
            == lengths.get_device() == codes.get_device() == scales.get_device()
            == sel_table.get_device() == sel_lengths.get_device() == workspace.get_device() == dev
            and (io is _BF16 or io is _F32) and q_pe.dtype is io and block_table.dtype is i32
            and lengths.dtype is i32 and codes.dtype is _I8 and scales.dtype is _F32
            and sel_table.dtype is i32 and sel_lengths.dtype is i32 and top >= 0
            and q_abs.numel() == rows * dc and q_pe.numel() == rows * dr
            and block_table.numel() == B * pg.table_stride and lengths.numel() == B
            and codes.numel() == pages * (dc + dr) and scales.numel() == pages
            and sel_table.numel() == R * top and sel_lengths.numel() == R
            and q_abs.is_contiguous() and q_pe.is_contiguous() and block_table.is_contiguous()
            and lengths.is_contiguous() and codes.is_contiguous() and scales.is_contiguous()
            and sel_table.is_contiguous() and sel_lengths.is_contiguous()
            and workspace.is_contiguous()
            and (dev_status is None or _is(dev_status, dev, i32, 1))):
        _io_code(io)
        _require(top >= 0, "sel_table must have one row per token")
        _explain(dev, q_abs=(q_abs, io, rows * dc), q_pe=(q_pe, io, rows * dr),
                 block_table=(block_table, i32, B * pg.table_stride), lengths=(lengths, i32, B),
                 codes=(codes, _I8, pages * (dc + dr)), scales=(scales, _F32, pages),
                 sel_table=(sel_table, i32, R * top), sel_lengths=(sel_lengths, i32, R),
                 workspace=(workspace, workspace.dtype, -1), dev_status=(dev_status, i32, 1))
    return MLA_BF16 if io is _BF16 else MLA_F32


def select_pages(d: MlaDims, pg: MlaPaging, q_abs, q_pe, block_table, lengths, codes, scales,
                 sel_table, sel_lengths, workspace, q_len: int = 1, keep_first: int = 1,
                 keep_last: int = 1, dev_status=None, stream=None) -> None:
    """The pages each token attends: its first and last ones and the best by the
    index's score, sel_table.shape[1] in all, as a block table of their own."""
    lib = _paged_lib()
    dev = _device()
    io = _check_selection(dev, d, pg, q_abs, q_pe, block_table, lengths, codes, scales, sel_table,
                          sel_lengths, workspace, q_len, dev_status)
    code = lib.mla_select_pages(
        d, pg, io, q_len, q_abs.data_ptr(), q_pe.data_ptr(), block_table.data_ptr(),
        lengths.data_ptr(), codes.data_ptr(), scales.data_ptr(), sel_table.shape[1], keep_first,
        keep_last, workspace.data_ptr(), workspace.numel() * workspace.itemsize,
        sel_table.data_ptr(), sel_lengths.data_ptr(),
        None if dev_status is None else dev_status.data_ptr(), _stream_on(dev, stream))
    if code:
        _check(code)


def sparse_workspace_bytes(d: MlaDims, pg: MlaPaging, io_dtype, top_pages: int, q_len: int = 1,
                           requested: int = 0) -> int:
    """Workspace bytes of decode_attn_sparse for queries of ``io_dtype``."""
    n = int(load().mla_sparse_workspace_bytes(d, pg, _io_code(io_dtype), int(q_len),
                                              int(top_pages), int(requested)))
    _require(n > 0, load().mla_last_error_message().decode())
    return n


def decode_attn_sparse(d: MlaDims, pg: MlaPaging, q_abs, q_pe, cache, block_table, lengths, codes,
                       scales, sel_table, sel_lengths, o_c, workspace, softmax_scale: float,
                       q_len: int = 1, keep_first: int = 1, keep_last: int = 1,
                       num_splits_requested: int = 0, lse=None, dev_status=None,
                       stream=None) -> None:
    """select_pages, then decode_attn_paged over the pages kept."""
    lib = _paged_lib()
    dev = _device()
    io = _check_selection(dev, d, pg, q_abs, q_pe, block_table, lengths, codes, scales, sel_table,
                          sel_lengths, workspace, q_len, dev_status)
    rows = d.batch * q_len * d.heads
    ct, cn = _ROW_TYPE.get(d.dtype), pg.num_pages * pg.page_size * (d.d_c + d.d_rope)
    if not (_is(cache, dev, ct, cn) and _is(o_c, dev, q_abs.dtype, rows * d.d_c)
            and (lse is None or _is(lse, dev, _F32, rows))):
        _explain(dev, cache=(cache, ct, cn), o_c=(o_c, q_abs.dtype, rows * d.d_c),
                 lse=(lse, _F32, rows))
    code = lib.mla_decode_attn_sparse(
        d, pg, io, q_len, q_abs.data_ptr(), q_pe.data_ptr(), cache.data_ptr(),
        block_table.data_ptr(), lengths.data_ptr(), codes.data_ptr(), scales.data_ptr(),
        softmax_scale, sel_table.shape[1], keep_first, keep_last, num_splits_requested,
        workspace.data_ptr(), workspace.numel() * workspace.itemsize, sel_table.data_ptr(),
        sel_lengths.data_ptr(), o_c.data_ptr(), None if lse is None else lse.data_ptr(),
        None if dev_status is None else dev_status.data_ptr(), _stream_on(dev, stream))
    if code:
        _check(code)
