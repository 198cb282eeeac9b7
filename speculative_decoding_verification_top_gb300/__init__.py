"""GB300 (sm_103a) speculative-decoding verification: Python binding.

The compute lives in ``libspecverify.so`` (hand-written CUDA, C ABI declared
in ``include/spec_verify.h``).  This module only loads it with ctypes and
marshals arguments: every step of the verification runs in the library's
kernels.  There is no CPU fallback -- if the library is not built, every
call raises.

Entry points (same names as the C ABI):
    spec_verify_workspace_size, spec_verify_tree_workspace_size,
    spec_verify_workspace_init, spec_verify_sample, spec_verify_tree,
    spec_verify_last_error, spec_verify_intermediates,
    spec_verify_acceptance, spec_verify_sample_probs, spec_verify_tree_mask,
    spec_verify_status_string,
    spec_kv_append, spec_kv_read, spec_attn_workspace_size, spec_attn_tree,
    spec_attn_shared (the target pass's cache and attention, declared in
    ``include/spec_attn.h``),
    spec_rope_freqs, spec_rope, spec_kv_append_rope (rotary positions),
    spec_latent_append, spec_latent_workspace_size, spec_latent_attn (a latent
    cache and its attention), spec_verify_logprobs_workspace_size,
    spec_verify_logprobs
plus tensor-level helpers ``verify_sample`` / ``verify_sample_probs`` /
``verify_tree`` / ``acceptance`` / ``logprobs`` / ``kv_append`` / ``kv_read`` /
``attn_tree`` / ``attn_shared`` / ``rope_freqs`` / ``rope`` /
``kv_append_rope`` / ``latent_append`` / ``latent_attn`` that take
torch CUDA tensors, allocate outputs and a zeroed workspace, and raise on a
negative status.
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import os
import subprocess

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
LIB_PATH = os.path.join(_PKG, "libspecverify.so")
CSRC = os.path.join(_PKG, "csrc")
SOURCES = [os.path.join(CSRC, f)
           for f in ("api.cu", "rows.cu", "topp.cu", "final.cu", "noalloc.cu",
                     "accept.cu", "treemask.cu", "treesample.cu", "select.cu",
                     "kvcache.cu", "attn.cu", "attn_few.cu", "attn_wide.cu", "attn_api.cu",
                     "rope.cu", "latent.cu", "target_api.cu", "logprobs.cu")]
HEADERS = [os.path.join(CSRC, f) for f in ("common.cuh", "stream.cuh", "draw.cuh", "attn.cuh",
                                             "attn_plan.cuh", "tensor.cuh", "checks.cuh",
                                             "kvrows.cuh", "target.cuh", "logprobs.cuh", "util.cuh",
                                             "latent_plan.cuh", "wide.h")]
INCLUDE = os.path.join(_ROOT, "include")
HEADER = os.path.join(INCLUDE, "spec_verify.h")
ATTN_HEADER = os.path.join(INCLUDE, "spec_attn.h")
BUILD_DIR = os.path.join(_PKG, "_build")

SPEC_F32, SPEC_BF16, SPEC_E4M3 = 0, 1, 2
SPEC_STOCHASTIC, SPEC_GREEDY = 0, 1
SPEC_OK = 0
SPEC_DATA_ROW_NONFINITE = 1 << 1
SPEC_DATA_ROW_ALL_NEG_INF = 1 << 2
SPEC_DATA_TOKEN_RANGE = 1 << 3
SPEC_DATA_UNIFORM_RANGE = 1 << 4
SPEC_DATA_TREE_SHAPE = 1 << 5
SPEC_DATA_PROB_RANGE = 1 << 6
SPEC_DATA_PAGE_RANGE = 1 << 7
SPEC_DATA_STALL = 1 << 8
SPEC_MAX_K = 31
SPEC_MAX_TOP = 32
SPEC_ROPE_HALF, SPEC_ROPE_INTERLEAVED = 0, 1
SPEC_ROPE_PLAIN, SPEC_ROPE_LINEAR, SPEC_ROPE_TURNS, SPEC_ROPE_INDEX = 0, 1, 2, 3

EXPORTED = (
    "spec_verify_workspace_size",
    "spec_verify_tree_workspace_size",
    "spec_verify_workspace_init",
    "spec_verify_sample",
    "spec_verify_sample_topk",
    "spec_verify_sample_rows",
    "spec_verify_sample_finish",
    "spec_verify_sample_noalloc",
    "spec_verify_tree",
    "spec_verify_last_error",
    "spec_verify_intermediates",
    "spec_verify_acceptance",
    "spec_verify_sample_probs",
    "spec_verify_tree_mask",
    "spec_verify_tree_sample_workspace_size",
    "spec_verify_tree_sample",
    "spec_kv_append",
    "spec_kv_read",
    "spec_attn_workspace_size",
    "spec_attn_tree",
    "spec_attn_shared",
    "spec_rope_freqs",
    "spec_rope",
    "spec_kv_append_rope",
    "spec_latent_append",
    "spec_latent_workspace_size",
    "spec_latent_attn",
    "spec_verify_logprobs_workspace_size",
    "spec_verify_logprobs",
    "spec_verify_status_string",
)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden"]


class CacheDescriptor(ctypes.Structure):
    """struct spec_kv_cache of include/spec_attn.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("page", ctypes.c_int), ("D", ctypes.c_int), ("dtype", ctypes.c_int)]


class LatentDescriptor(ctypes.Structure):
    """struct spec_latent_cache of include/spec_attn.h."""
    _fields_ = [("data", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page", ctypes.c_int),
                ("C", ctypes.c_int), ("R", ctypes.c_int)]


class SpecVerifyError(RuntimeError):
    """A negative status from the library."""


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA sources for sm_103a (one nvcc per translation unit,
    in parallel) and link libspecverify.so in-tree."""
    newest = max(os.path.getmtime(p) for p in SOURCES + HEADERS + [HEADER, ATTN_HEADER])
    if not force and os.path.exists(LIB_PATH) and os.path.getmtime(LIB_PATH) >= newest:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    tag = "%d" % os.getpid()
    objs, procs = [], []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + "." + tag + ".o")
        cmd = ["nvcc", *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        objs.append(obj)
        procs.append(subprocess.Popen(cmd))
    if any(p.wait() != 0 for p in procs):
        raise RuntimeError("nvcc failed")
    tmp = LIB_PATH + "." + tag + ".tmp"
    subprocess.check_call(["nvcc", *ARCH, "-shared", *objs, "-o", tmp])
    os.replace(tmp, LIB_PATH)
    for obj in objs:
        os.unlink(obj)
    return LIB_PATH


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libspecverify.so is not built (run speculative_decoding_verification_top_gb300"
                ".build()); there is no fallback implementation")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.spec_verify_workspace_size.argtypes = [I, I, I, ctypes.POINTER(Z)]
        L.spec_verify_tree_workspace_size.argtypes = [I, I, I, ctypes.POINTER(Z)]
        L.spec_verify_workspace_init.argtypes = [P, Z, P]
        for name in ("spec_verify_sample", "spec_verify_sample_rows", "spec_verify_sample_finish"):
            getattr(L, name).argtypes = [P, P, P, P, I, I, I, F, F, I, I, P, P, P, Z, P]
        L.spec_verify_sample_topk.argtypes = [P, P, P, P, I, I, I, F, F, I, I, I, P, P, P, Z, P]
        L.spec_verify_sample_noalloc.argtypes = [P, P, P, P, I, I, I, F, F, I, I, P, P, P]
        L.spec_verify_tree.argtypes = [P, P, P, I, I, I, I, I, P, P, P, P, Z, P]
        L.spec_verify_last_error.argtypes = [P, Z, P]
        L.spec_verify_intermediates.argtypes = [P, Z, I, I, I, P, P, P, P, P]
        L.spec_verify_acceptance.argtypes = [P, P, I, I, I, F, F, I, I, P, P, P, Z, P]
        L.spec_verify_sample_probs.argtypes = [P, P, P, P, I, I, I, F, F, I, I, P, P, P, Z, P]
        L.spec_verify_tree_mask.argtypes = [P, P, I, I, P, P, P, P]
        L.spec_verify_tree_sample_workspace_size.argtypes = [I, I, I, ctypes.POINTER(Z)]
        L.spec_verify_tree_sample.argtypes = [P, P, P, P, P, I, I, I, I, F, F, I, I, P, P, P, P,
                                              Z, P]
        C, S = ctypes.POINTER(CacheDescriptor), ctypes.c_int64
        L.spec_kv_append.argtypes = [C, P, I, P, P, P, S, P, I, I, I, I, P]
        L.spec_kv_read.argtypes = [C, P, I, P, P, P, I, I, I, P]
        L.spec_attn_workspace_size.argtypes = [I, I, I, I, I, ctypes.POINTER(Z)]
        L.spec_attn_tree.argtypes = [C, P, I, P, P, S, P, P, P, I, I, I, F, F, I, I, P, P, P, Z, P]
        L.spec_attn_shared.argtypes = [C, P, I, P, I, P, P, S, P, P, P, I, I, I, F, F, I, I, P, P,
                                       P, Z, P]
        D, A = ctypes.c_double, ctypes.POINTER(LatentDescriptor)
        L.spec_rope_freqs.argtypes = [I, D, I, D, D, D, D, P]
        L.spec_rope.argtypes = [P, S, P, S, P, I, I, F, I, I, P, I, I, I, I, I, P]
        L.spec_kv_append_rope.argtypes = [C, P, I, P, P, P, S, P, P, P, I, F, I, P, S, P, S, I, I, I,
                                          I, I, P]
        L.spec_latent_append.argtypes = [A, P, I, P, P, S, P, S, P, P, P, F, I, I, I, I, I, P]
        L.spec_latent_workspace_size.argtypes = [I, I, I, I, ctypes.POINTER(Z)]
        L.spec_latent_attn.argtypes = [A, P, I, P, P, S, P, I, I, I, F, P, P, P, Z, P]
        L.spec_verify_logprobs_workspace_size.argtypes = [ctypes.POINTER(Z)]
        L.spec_verify_logprobs.argtypes = [P, P, P, I, I, I, I, F, I, I, P, P, P, P, P, P, Z, P]
        L.spec_verify_status_string.argtypes = [I]
        L.spec_verify_status_string.restype = ctypes.c_char_p
        for name in EXPORTED[:-1]:
            getattr(L, name).restype = I
        _lib = L
    return _lib


def _check(rc):
    if rc < 0:
        raise SpecVerifyError("%d: %s" % (rc, spec_verify_status_string(rc)))
    return rc


# ----------------------------------------------------- C ABI, same names

def spec_verify_workspace_size(B, k, V):
    out = ctypes.c_size_t(0)
    _check(lib().spec_verify_workspace_size(B, k, V, ctypes.byref(out)))
    return out.value


def spec_verify_tree_workspace_size(B, N, V):
    out = ctypes.c_size_t(0)
    _check(lib().spec_verify_tree_workspace_size(B, N, V, ctypes.byref(out)))
    return out.value


def spec_verify_workspace_init(workspace_ptr, nbytes, stream=0):
    return _check(lib().spec_verify_workspace_init(workspace_ptr, nbytes, stream))


def spec_verify_sample(target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V, temperature,
                       top_p, mode, dtype, out_tokens_ptr, out_num_ptr, workspace_ptr,
                       workspace_bytes, stream=0):
    return _check(lib().spec_verify_sample(
        target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V, float(temperature),
        float(top_p), mode, dtype, out_tokens_ptr, out_num_ptr, workspace_ptr,
        workspace_bytes, stream))


def spec_verify_sample_topk(target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V,
                            temperature, top_p, top_k, mode, dtype, out_tokens_ptr, out_num_ptr,
                            workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_verify_sample_topk(
        target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V, float(temperature),
        float(top_p), int(top_k), mode, dtype, out_tokens_ptr, out_num_ptr, workspace_ptr,
        workspace_bytes, stream))


def spec_verify_sample_rows(target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V,
                            temperature, top_p, mode, dtype, out_tokens_ptr, out_num_ptr,
                            workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_verify_sample_rows(
        target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V, float(temperature),
        float(top_p), mode, dtype, out_tokens_ptr, out_num_ptr, workspace_ptr,
        workspace_bytes, stream))


def spec_verify_sample_finish(target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V,
                              temperature, top_p, mode, dtype, out_tokens_ptr, out_num_ptr,
                              workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_verify_sample_finish(
        target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V, float(temperature),
        float(top_p), mode, dtype, out_tokens_ptr, out_num_ptr, workspace_ptr,
        workspace_bytes, stream))


def spec_verify_sample_noalloc(target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V,
                               temperature, top_p, mode, dtype, out_tokens_ptr, out_num_ptr,
                               stream=0):
    """spec_verify_sample without a workspace, for callers that cannot
    allocate device memory: the library's fixed 4 MiB per-device scratch is
    used instead (calls that overlap on the GPU race on it)."""
    return _check(lib().spec_verify_sample_noalloc(
        target_ptr, draft_ptr, tokens_ptr, uniforms_ptr, B, k, V, float(temperature),
        float(top_p), mode, dtype, out_tokens_ptr, out_num_ptr, stream))


def spec_verify_tree(target_ptr, parents_ptr, node_tokens_ptr, B, N, V, D, dtype,
                     out_tokens_ptr, out_num_ptr, out_path_ptr, workspace_ptr, workspace_bytes,
                     stream=0):
    return _check(lib().spec_verify_tree(
        target_ptr, parents_ptr, node_tokens_ptr, B, N, V, D, dtype, out_tokens_ptr,
        out_num_ptr, out_path_ptr, workspace_ptr, workspace_bytes, stream))


def spec_verify_last_error(workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_verify_last_error(workspace_ptr, workspace_bytes, stream))


def spec_verify_intermediates(workspace_ptr, workspace_bytes, B, k, V, P_ptr, Q_ptr, Z_ptr,
                              S_ptr, stream=0):
    return _check(lib().spec_verify_intermediates(workspace_ptr, workspace_bytes, B, k, V,
                                                  P_ptr, Q_ptr, Z_ptr, S_ptr, stream))


def spec_verify_acceptance(target_ptr, draft_ptr, B, k, V, temperature, top_p, top_k, dtype,
                           out_beta_ptr, out_tv_ptr, workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_verify_acceptance(
        target_ptr, draft_ptr, B, k, V, float(temperature), float(top_p), int(top_k), dtype,
        out_beta_ptr, out_tv_ptr, workspace_ptr, workspace_bytes, stream))


def spec_verify_sample_probs(target_ptr, draft_probs_ptr, tokens_ptr, uniforms_ptr, B, k, V,
                             temperature, top_p, top_k, dtype, out_tokens_ptr, out_num_ptr,
                             workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_verify_sample_probs(
        target_ptr, draft_probs_ptr, tokens_ptr, uniforms_ptr, B, k, V, float(temperature),
        float(top_p), int(top_k), dtype, out_tokens_ptr, out_num_ptr, workspace_ptr,
        workspace_bytes, stream))


def spec_verify_tree_mask(parents_ptr, pos0_ptr, B, N, out_mask_ptr, out_bias_ptr, out_pos_ptr,
                          stream=0):
    return _check(lib().spec_verify_tree_mask(parents_ptr, pos0_ptr, B, N, out_mask_ptr,
                                              out_bias_ptr, out_pos_ptr, stream))


def spec_verify_tree_sample_workspace_size(B, N, V):
    out = ctypes.c_size_t(0)
    _check(lib().spec_verify_tree_sample_workspace_size(B, N, V, ctypes.byref(out)))
    return out.value


def spec_verify_tree_sample(target_ptr, draft_ptr, parents_ptr, node_tokens_ptr, uniforms_ptr,
                            B, N, V, D, temperature, top_p, top_k, dtype, out_tokens_ptr,
                            out_num_ptr, out_path_ptr, workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_verify_tree_sample(
        target_ptr, draft_ptr, parents_ptr, node_tokens_ptr, uniforms_ptr, B, N, V, D,
        float(temperature), float(top_p), int(top_k), dtype, out_tokens_ptr, out_num_ptr,
        out_path_ptr, workspace_ptr, workspace_bytes, stream))


def spec_kv_append(cache, table_ptr, table_width, starts_ptr, k_ptr, v_ptr, token_stride, rows_ptr,
                   B, N, M, dtype, stream=0):
    """`cache`: a CacheDescriptor, here and below."""
    return _check(lib().spec_kv_append(cache, table_ptr, table_width, starts_ptr, k_ptr, v_ptr,
                                       token_stride, rows_ptr, B, N, M, dtype, stream))


def spec_kv_read(cache, table_ptr, table_width, starts_ptr, out_k_ptr, out_v_ptr, B, M, dtype,
                 stream=0):
    return _check(lib().spec_kv_read(cache, table_ptr, table_width, starts_ptr, out_k_ptr,
                                     out_v_ptr, B, M, dtype, stream))


def spec_attn_workspace_size(B, N, Hq, Hkv, D):
    out = ctypes.c_size_t(0)
    _check(lib().spec_attn_workspace_size(B, N, Hq, Hkv, D, ctypes.byref(out)))
    return out.value


def spec_attn_tree(cache, table_ptr, table_width, lens_ptr, q_ptr, q_stride, mask_ptr, pos_ptr,
                   slopes_ptr, B, N, Hq, scale, cap, window, dtype, out_ptr, out_lse_ptr,
                   workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_attn_tree(
        cache, table_ptr, table_width, lens_ptr, q_ptr, q_stride, mask_ptr, pos_ptr, slopes_ptr, B,
        N, Hq, float(scale), float(cap), window, dtype, out_ptr, out_lse_ptr, workspace_ptr,
        workspace_bytes, stream))


def spec_attn_shared(cache, shared_table_ptr, shared_len, table_ptr, table_width, lens_ptr, q_ptr,
                     q_stride, mask_ptr, pos_ptr, slopes_ptr, B, N, Hq, scale, cap, window, dtype,
                     out_ptr, out_lse_ptr, workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_attn_shared(
        cache, shared_table_ptr, shared_len, table_ptr, table_width, lens_ptr, q_ptr, q_stride,
        mask_ptr, pos_ptr, slopes_ptr, B, N, Hq, float(scale), float(cap), window, dtype, out_ptr,
        out_lse_ptr, workspace_ptr, workspace_bytes, stream))


def spec_rope_freqs(rot, base, scaling, factor, original, low, high, freqs_ptr):
    """`freqs_ptr`: host memory for rot / 2 uint64."""
    return _check(lib().spec_rope_freqs(rot, base, scaling, factor, original, low, high, freqs_ptr))


def spec_rope(x_ptr, x_stride, out_ptr, out_stride, freqs_ptr, rot, first, amplitude, layout, inverse,
              pos_ptr, B, N, H, D, dtype, stream=0):
    return _check(lib().spec_rope(x_ptr, x_stride, out_ptr, out_stride, freqs_ptr, rot, first,
                                  float(amplitude), layout, inverse, pos_ptr, B, N, H, D, dtype,
                                  stream))


def spec_kv_append_rope(cache, table_ptr, table_width, starts_ptr, k_ptr, v_ptr, token_stride, rows_ptr,
                        pos_ptr, freqs_ptr, rot, amplitude, layout, q_ptr, q_stride, out_q_ptr,
                        out_q_stride, B, N, M, Hq, dtype, stream=0):
    return _check(lib().spec_kv_append_rope(
        cache, table_ptr, table_width, starts_ptr, k_ptr, v_ptr, token_stride, rows_ptr, pos_ptr,
        freqs_ptr, rot, float(amplitude), layout, q_ptr, q_stride, out_q_ptr, out_q_stride, B, N, M, Hq,
        dtype, stream))


def spec_latent_append(cache, table_ptr, table_width, starts_ptr, c_ptr, c_stride, r_ptr, r_stride,
                       rows_ptr, pos_ptr, freqs_ptr, amplitude, layout, B, N, M, dtype, stream=0):
    """`cache`: a LatentDescriptor, here and below."""
    return _check(lib().spec_latent_append(
        cache, table_ptr, table_width, starts_ptr, c_ptr, c_stride, r_ptr, r_stride, rows_ptr, pos_ptr,
        freqs_ptr, float(amplitude), layout, B, N, M, dtype, stream))


def spec_latent_workspace_size(B, N, H, C):
    out = ctypes.c_size_t(0)
    _check(lib().spec_latent_workspace_size(B, N, H, C, ctypes.byref(out)))
    return out.value


def spec_latent_attn(cache, table_ptr, table_width, lens_ptr, q_ptr, q_stride, mask_ptr, B, N, H, scale,
                     out_ptr, out_lse_ptr, workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_latent_attn(
        cache, table_ptr, table_width, lens_ptr, q_ptr, q_stride, mask_ptr, B, N, H, float(scale), out_ptr,
        out_lse_ptr, workspace_ptr, workspace_bytes, stream))


def spec_verify_logprobs_workspace_size():
    out = ctypes.c_size_t(0)
    _check(lib().spec_verify_logprobs_workspace_size(ctypes.byref(out)))
    return out.value


def spec_verify_logprobs(target_ptr, tokens_ptr, rows_ptr, B, N, M, V, temperature, top, dtype,
                         out_logprob_ptr, out_entropy_ptr, out_rank_ptr, out_top_ids_ptr,
                         out_top_logprobs_ptr, workspace_ptr, workspace_bytes, stream=0):
    return _check(lib().spec_verify_logprobs(
        target_ptr, tokens_ptr, rows_ptr, B, N, M, V, float(temperature), top, dtype, out_logprob_ptr,
        out_entropy_ptr, out_rank_ptr, out_top_ids_ptr, out_top_logprobs_ptr, workspace_ptr,
        workspace_bytes, stream))


def spec_verify_status_string(status):
    return lib().spec_verify_status_string(int(status)).decode()


# ------------------------------------------------- torch tensor helpers

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    raise TypeError("logits must be torch.float32 or torch.bfloat16, got %s" % t.dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _made_on(stream):
    """Where a call's own tensors are made: on the stream that works on them, so
    that zeroing comes before that work and memory freed at return goes to later
    work of the same stream only."""
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


def _need(t, name, dtype, shape):
    if t.dtype != dtype or t.shape != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError("%s must be a contiguous CUDA %s tensor of shape %s, got %s %s"
                         % (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))


def _made(stream, make, *args, **kw):
    """make(...) on the call's stream (as _made_on)."""
    if stream is None:
        return make(*args, **kw)
    with _torch().cuda.stream(stream):
        return make(*args, **kw)


def _lies(t, name, dtype, shape, device):
    """_need for a tensor beside others on the device of index `device`."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d, got %s %s on %s"
                         % (name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device))


def _launch(device, stream):
    """The handle of the stream that a call on tensors of this device runs on: the
    given one, else the current one (by its handle: a Stream object takes 3 us)."""
    c = _torch()._C
    if c._cuda_getDevice() != device:
        raise ValueError("the tensors are on cuda:%d, which is not the current device" % device)
    return c._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _room(workspace, device):
    """A given workspace holds the bytes that it counts: not one of expanded elements."""
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on cuda:%d, got strides %s on %s"
                         % (device, workspace.stride(), workspace.device))


def new_workspace(nbytes, device):
    """A zero-filled workspace tensor (zeroing is the required first-use init)."""
    torch = _torch()
    return torch.zeros(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def verify_sample(target, draft, draft_tokens, uniforms, temperature=1.0, top_p=1.0,
                  mode=SPEC_STOCHASTIC, out_tokens=None, out_num=None, workspace=None,
                  stream=None, top_k=0):
    """Tensor-level spec_verify_sample.  Returns (out_tokens [B, k+1],
    out_num_accepted [B], workspace)."""
    torch = _torch()
    B, k1, V = target.shape
    k = k1 - 1
    dt = _dtype_code(target)
    _need(target, "target", target.dtype, (B, k + 1, V))
    if mode == SPEC_STOCHASTIC:
        _need(draft, "draft", target.dtype, (B, k, V))
        _need(uniforms, "uniforms", torch.float32, (B, k + 1))
    _need(draft_tokens, "draft_tokens", torch.int32, (B, k))
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if out_num is None:
        out_num = torch.empty((B,), dtype=torch.int32, device=dev)
    nbytes = spec_verify_workspace_size(B, k, V)
    if workspace is None:
        workspace = new_workspace(nbytes, dev)
    stoch = mode == SPEC_STOCHASTIC
    args = (_ptr(target), _ptr(draft) if stoch else None, _ptr(draft_tokens),
            _ptr(uniforms) if stoch else None, B, k, V, temperature, top_p)
    tail = (mode, dt, _ptr(out_tokens), _ptr(out_num), _ptr(workspace), workspace.numel(),
            _stream(stream))
    if top_k:
        spec_verify_sample_topk(*args, top_k, *tail)
    else:
        spec_verify_sample(*args, *tail)
    return out_tokens, out_num, workspace


def verify_sample_probs(target, draft_probs, draft_tokens, uniforms, temperature=1.0, top_p=1.0,
                        out_tokens=None, out_num=None, workspace=None, stream=None, top_k=0):
    """Tensor-level spec_verify_sample_probs (draft given as fp32
    probabilities [B, k, V]).  Returns (out_tokens, out_num_accepted,
    workspace)."""
    torch = _torch()
    B, k1, V = target.shape
    k = k1 - 1
    dt = _dtype_code(target)
    _need(target, "target", target.dtype, (B, k + 1, V))
    _need(draft_probs, "draft_probs", torch.float32, (B, k, V))
    _need(uniforms, "uniforms", torch.float32, (B, k + 1))
    _need(draft_tokens, "draft_tokens", torch.int32, (B, k))
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if out_num is None:
        out_num = torch.empty((B,), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = new_workspace(spec_verify_workspace_size(B, k, V), dev)
    spec_verify_sample_probs(_ptr(target), _ptr(draft_probs), _ptr(draft_tokens), _ptr(uniforms),
                             B, k, V, temperature, top_p, top_k, dt, _ptr(out_tokens),
                             _ptr(out_num),
                             _ptr(workspace), workspace.numel(), _stream(stream))
    return out_tokens, out_num, workspace


def verify_tree(target, parents, node_tokens, depth, out_tokens=None, out_num=None,
                out_path=None, workspace=None, stream=None):
    """Tensor-level spec_verify_tree.  Returns (out_tokens [B, D+1],
    out_num_accepted [B], out_path [B, D+1], workspace)."""
    torch = _torch()
    B, N, V = target.shape
    dt = _dtype_code(target)
    _need(target, "target", target.dtype, (B, N, V))
    _need(parents, "parents", torch.int32, (N,))
    _need(node_tokens, "node_tokens", torch.int32, (B, N))
    dev = target.device
    W = depth + 1
    if out_tokens is None:
        out_tokens = torch.empty((B, W), dtype=torch.int32, device=dev)
    if out_num is None:
        out_num = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_path is None:
        out_path = torch.empty((B, W), dtype=torch.int32, device=dev)
    nbytes = spec_verify_tree_workspace_size(B, N, V)
    if workspace is None:
        workspace = new_workspace(nbytes, dev)
    spec_verify_tree(_ptr(target), _ptr(parents), _ptr(node_tokens), B, N, V, depth, dt,
                     _ptr(out_tokens), _ptr(out_num), _ptr(out_path), _ptr(workspace),
                     workspace.numel(), _stream(stream))
    return out_tokens, out_num, out_path, workspace


def last_error(workspace, stream=None):
    return spec_verify_last_error(_ptr(workspace), workspace.numel(), _stream(stream))


def intermediates(workspace, B, k, V, stream=None):
    """(P [B, k], Q [B, k], Z [B, 2k+1], S [B]) of the last stochastic call."""
    torch = _torch()
    dev = workspace.device
    P = torch.empty((B, k), dtype=torch.float32, device=dev)
    Q = torch.empty((B, k), dtype=torch.float32, device=dev)
    Z = torch.empty((B, 2 * k + 1), dtype=torch.float32, device=dev)
    S = torch.empty((B,), dtype=torch.float32, device=dev)
    spec_verify_intermediates(_ptr(workspace), workspace.numel(), B, k, V, _ptr(P), _ptr(Q),
                              _ptr(Z), _ptr(S), _stream(stream))
    return P, Q, Z, S


def acceptance(target, draft, workspace, temperature=1.0, top_p=1.0, out_beta=None, out_tv=None,
               stream=None, top_k=0):
    """Tensor-level spec_verify_acceptance: (beta [B, k], tv [B, k]) of the
    last stochastic verify call made on `workspace` with these arguments."""
    torch = _torch()
    B, k1, V = target.shape
    k = k1 - 1
    dt = _dtype_code(target)
    _need(target, "target", target.dtype, (B, k + 1, V))
    _need(draft, "draft", target.dtype, (B, k, V))
    dev = target.device
    if out_beta is None:
        out_beta = torch.empty((B, k), dtype=torch.float32, device=dev)
    if out_tv is None:
        out_tv = torch.empty((B, k), dtype=torch.float32, device=dev)
    spec_verify_acceptance(_ptr(target), _ptr(draft), B, k, V, temperature, top_p, top_k, dt,
                           _ptr(out_beta), _ptr(out_tv), _ptr(workspace), workspace.numel(),
                           _stream(stream))
    return out_beta, out_tv


def tree_mask(parents, pos0=None, mask=True, bias=False, pos=True, stream=None):
    """Tensor-level spec_verify_tree_mask: parents [B, N] int32 (CUDA).
    Returns (mask [B, N, N] uint8 or None, bias [B, N, N] fp32 or None,
    pos [B, N] int32 or None)."""
    torch = _torch()
    B, N = parents.shape
    _need(parents, "parents", torch.int32, (B, N))
    if pos0 is not None:
        _need(pos0, "pos0", torch.int32, (B,))
    dev = parents.device
    m = torch.empty((B, N, N), dtype=torch.uint8, device=dev) if mask else None
    bs = torch.empty((B, N, N), dtype=torch.float32, device=dev) if bias else None
    p = torch.empty((B, N), dtype=torch.int32, device=dev) if pos else None
    spec_verify_tree_mask(_ptr(parents), _ptr(pos0), B, N, _ptr(m), _ptr(bs), _ptr(p),
                          _stream(stream))
    return m, bs, p


def verify_tree_sample(target, draft, parents, node_tokens, uniforms, depth, temperature=1.0,
                       top_p=1.0, top_k=0, workspace=None, stream=None):
    """Tensor-level spec_verify_tree_sample.  Returns (out_tokens [B, D+1],
    out_num_accepted [B], out_path [B, D+1], workspace)."""
    torch = _torch()
    B, N, V = target.shape
    dt = _dtype_code(target)
    _need(target, "target", target.dtype, (B, N, V))
    _need(draft, "draft", target.dtype, (B, N, V))
    _need(parents, "parents", torch.int32, (N,))
    _need(node_tokens, "node_tokens", torch.int32, (B, N))
    _need(uniforms, "uniforms", torch.float32, (B, N))
    dev = target.device
    W = depth + 1
    out_t = torch.empty((B, W), dtype=torch.int32, device=dev)
    out_n = torch.empty((B,), dtype=torch.int32, device=dev)
    out_p = torch.empty((B, W), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = new_workspace(spec_verify_tree_sample_workspace_size(B, N, V), dev)
    spec_verify_tree_sample(_ptr(target), _ptr(draft), _ptr(parents), _ptr(node_tokens),
                            _ptr(uniforms), B, N, V, depth, temperature, top_p, top_k, dt,
                            _ptr(out_t), _ptr(out_n), _ptr(out_p), _ptr(workspace),
                            workspace.numel(), _stream(stream))
    return out_t, out_n, out_p, workspace


LogProbs = collections.namedtuple("LogProbs", "logprob entropy rank top_ids top_logprobs")


def logprobs(target, tokens, rows=None, temperature=1.0, top=0, entropy=True, rank=True,
             workspace=None, stream=None):
    """Tensor-level spec_verify_logprobs: target logits [B, N, V], emitted
    tokens [B, M] int32 (verify_sample's out_tokens; -1: no entry) and, after
    verify_tree, rows = its out_path.  Returns LogProbs: logprob, entropy [B, M]
    fp32, rank [B, M] int32 (None where not asked for), and with top > 0 top_ids
    int32 and top_logprobs fp32 [B, M, top].  Data errors (last_error) are in the
    workspace: give one to read them."""
    torch = _torch()
    B, N, V = target.shape
    M = tokens.shape[1]
    if not (target.is_contiguous() and target.is_cuda):
        raise ValueError("target must be a contiguous CUDA tensor")
    device = target.get_device()
    _lies(tokens, "tokens", torch.int32, (B, M), device)
    if rows is not None:
        _lies(rows, "rows", torch.int32, (B, M), device)
    handle = _launch(device, stream)
    out = _made(stream, _new_logprobs, B, M, top, entropy, rank, target.device)
    if workspace is None:
        workspace = _made(stream, new_workspace, spec_verify_logprobs_workspace_size(), target.device)
    else:
        _room(workspace, device)
    spec_verify_logprobs(target.data_ptr(), tokens.data_ptr(), _ptr(rows), B, N, M, V, temperature, top,
                         _dtype_code(target), out.logprob.data_ptr(), _ptr(out.entropy), _ptr(out.rank),
                         _ptr(out.top_ids), _ptr(out.top_logprobs), workspace.data_ptr(),
                         workspace.numel(), handle)
    return out


def _new_logprobs(B, M, top, entropy, rank, device):
    empty, f, i = _torch().empty, _torch().float32, _torch().int32
    return LogProbs(empty((B, M), dtype=f, device=device),
                    empty((B, M), dtype=f, device=device) if entropy else None,
                    empty((B, M), dtype=i, device=device) if rank else None,
                    empty((B, M, top), dtype=i, device=device) if top else None,
                    empty((B, M, top), dtype=f, device=device) if top else None)


# ------------------------------------------- the target pass's cache and attention

class KVCache(collections.namedtuple("KVCache", "k v k_exp v_exp")):
    """A paged cache's tensors: k, v [num_pages, Hkv, page, D] bf16, or
    float8_e4m3fn with int8 exponents k_exp, v_exp [num_pages, Hkv, page]
    (else None).  Checked once, here; the calls pass its C descriptor."""

    def __new__(cls, k, v, k_exp=None, v_exp=None):
        torch = _torch()
        self = super().__new__(cls, k, v, k_exp, v_exp)
        n, H, page, D = k.shape
        e4m3 = k.dtype == torch.float8_e4m3fn
        if not e4m3 and k.dtype != torch.bfloat16:
            raise TypeError("a cache holds torch.bfloat16 or torch.float8_e4m3fn, got %s" % k.dtype)
        for t, name in ((k, "cache.k"), (v, "cache.v")):
            _need(t, name, k.dtype, (n, H, page, D))
        if e4m3:
            for t, name in ((k_exp, "cache.k_exp"), (v_exp, "cache.v_exp")):
                _need(t, name, torch.int8, (n, H, page))
        self.descriptor = CacheDescriptor(
            _ptr(k), _ptr(v), _ptr(k_exp) if e4m3 else None, _ptr(v_exp) if e4m3 else None, n, H,
            page, D, SPEC_E4M3 if e4m3 else SPEC_BF16)
        return self

    @classmethod
    def _make(cls, tensors):  # _replace comes here too
        return cls(*tensors)

    def __reduce__(self):  # a copy's descriptor is of the copy's tensors
        return type(self), tuple(self)


def new_cache(num_pages, Hkv, page, D, device, e4m3=False):
    """An empty (zeroed) cache of num_pages pages."""
    torch = _torch()
    shape = (num_pages, Hkv, page, D)
    if not e4m3:
        k, v = (torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in "kv")
        return KVCache(k, v, None, None)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
            for _ in "kv")
    ke, ve = (torch.zeros(shape[:3], dtype=torch.int8, device=device) for _ in "kv")
    return KVCache(k, v, ke, ve)


def _tokens(t, name, H, D, dtypes):
    """[B, N, H, D] with packed tokens; returns their stride in elements.
    Consecutive tokens may lie further apart (slices of a wider projection),
    evenly over the whole batch."""
    shape = t.shape
    if t.dtype not in dtypes or len(shape) != 4 or shape[2] != H or shape[3] != D or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor [B, N, %d, %d] of %s, got %s %s"
                         % (name, H, D, "/".join(map(str, dtypes)), t.dtype, tuple(t.shape)))
    if t.is_contiguous():
        return H * D
    B, N = t.shape[:2]
    s = t.stride()
    step = s[1] if N > 1 else s[0] if B > 1 else H * D
    if s[3] == 1 and (H == 1 or s[2] == D) and (B < 2 or s[0] == N * step) and step >= H * D:
        return step
    raise ValueError("%s: each token's heads must be contiguous and tokens evenly spaced, without "
                     "overlap (no expanded tokens), got strides %s" % (name, s))


def kv_append(cache, page_table, starts, k, v, rows=None, stream=None):
    """Tensor-level spec_kv_append: tokens k, v [B, N, Hkv, D] (fp32 or bf16)
    to positions starts[b] + t of a KVCache; rows [B, M] int32 picks the
    tokens (spec_verify_tree's out_path: the accepted nodes, -1 skipped)."""
    torch = _torch()
    c = cache.descriptor
    B, N = k.shape[:2]
    step = _tokens(k, "k", c.Hkv, c.D, (torch.bfloat16, torch.float32))
    if _tokens(v, "v", c.Hkv, c.D, (k.dtype,)) != step or v.shape != k.shape:
        raise ValueError("k and v must have one shape and token stride")
    _need(page_table, "page_table", torch.int32, (B, page_table.shape[1]))
    _need(starts, "starts", torch.int32, (B,))
    M = N
    if rows is not None:
        M = rows.shape[1]
        _need(rows, "rows", torch.int32, (B, M))
    spec_kv_append(c, _ptr(page_table), page_table.shape[1], _ptr(starts), _ptr(k), _ptr(v), step,
                   _ptr(rows), B, N, M, _dtype_code(k), _stream(stream))


def kv_read(cache, page_table, starts, count, dtype=None, stream=None):
    """Tensor-level spec_kv_read: (k, v) [B, count, Hkv, D] of the positions
    from starts[b] on, in bf16 (or fp32)."""
    torch = _torch()
    c = cache.descriptor
    B = starts.shape[0]
    _need(page_table, "page_table", torch.int32, (B, page_table.shape[1]))
    _need(starts, "starts", torch.int32, (B,))
    with _made_on(stream):
        k, v = (torch.empty((B, count, c.Hkv, c.D), dtype=dtype or torch.bfloat16,
                            device=starts.device) for _ in "kv")
    spec_kv_read(c, _ptr(page_table), page_table.shape[1], _ptr(starts), _ptr(k), _ptr(v), B, count,
                 _dtype_code(k), _stream(stream))
    return k, v


def _attn(call, q, cache, before, page_table, lens, mask, pos, slopes, scale, cap, window, out, lse,
          workspace, stream):
    torch = _torch()
    c = cache.descriptor
    B, N, Hq = q.shape[:3]
    step = _tokens(q, "q", Hq, c.D, (torch.bfloat16,))
    _need(page_table, "page_table", torch.int32, (B, page_table.shape[1]))
    _need(lens, "lens", torch.int32, (B,))
    if mask is not None:
        _need(mask, "mask", torch.uint8, (B, N, N))
    if pos is not None:
        _need(pos, "pos", torch.int32, (B, N))
    if slopes is not None:
        _need(slopes, "slopes", torch.float32, (Hq,))
    with _made_on(stream):
        if out is None:
            out = torch.empty((B, N, Hq, c.D), dtype=q.dtype, device=q.device)
        if lse is True:
            lse = torch.empty((B, N, Hq), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = new_workspace(spec_attn_workspace_size(B, N, Hq, c.Hkv, c.D), q.device)
    _need(out, "out", q.dtype, (B, N, Hq, c.D))
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, N, Hq))
    call(c, *before, _ptr(page_table), page_table.shape[1], _ptr(lens), _ptr(q), step, _ptr(mask),
         _ptr(pos), _ptr(slopes), B, N, Hq, c.D ** -0.5 if scale is None else scale, cap, window,
         SPEC_BF16, _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream))
    return out if lse is None else (out, lse)


def attn_tree(q, cache, page_table, lens, mask=None, pos=None, slopes=None, scale=None, cap=0.0,
              window=0, out=None, lse=None, workspace=None, stream=None):
    """Tensor-level spec_attn_tree: new tokens q [B, N, Hq, D] bf16 over a
    KVCache; mask and pos as tree_mask returns them (None: a chain); scale
    defaults to 1/sqrt(D).  Returns out [B, N, Hq, D], or (out, lse) with
    lse=True or a tensor.  With ``stream``, what the call allocates belongs to
    that stream.  Data errors (last_error) are in the workspace: give one to
    read them."""
    return _attn(spec_attn_tree, q, cache, (), page_table, lens, mask, pos, slopes, scale, cap,
                 window, out, lse, workspace, stream)


def attn_shared(q, cache, shared_table, shared_len, page_table, lens, mask=None, pos=None,
                slopes=None, scale=None, cap=0.0, window=0, out=None, lse=None, workspace=None,
                stream=None):
    """Tensor-level spec_attn_shared: attn_tree where every sequence's cache
    continues the shared_len positions of the pages shared_table lists."""
    torch = _torch()
    _need(shared_table, "shared_table", torch.int32, (shared_table.numel(),))
    if shared_table.numel() * cache.k.shape[2] < shared_len:
        raise ValueError("shared_table holds %d pages, %d positions need more"
                         % (shared_table.numel(), shared_len))
    return _attn(spec_attn_shared, q, cache, (_ptr(shared_table), shared_len), page_table, lens,
                 mask, pos, slopes, scale, cap, window, out, lse, workspace, stream)


# ------------------------------------------------------------- rotary positions

SCALINGS = {"plain": SPEC_ROPE_PLAIN, "linear": SPEC_ROPE_LINEAR, "turns": SPEC_ROPE_TURNS,
            "index": SPEC_ROPE_INDEX}


def rope_freqs(rot, base=10000.0, scaling="plain", factor=1.0, original=0, low=0.0, high=0.0,
               device="cuda"):
    """The frequencies of spec_rope_freqs, made once, as an int64 tensor [rot / 2]
    on `device`.  scaling: "plain", "linear", "turns" or "index" (the header's
    SPEC_ROPE_*)."""
    torch = _torch()
    if scaling not in SCALINGS:
        raise ValueError("scaling must be one of %s, got %r" % (", ".join(SCALINGS), scaling))
    host = torch.empty((max(int(rot), 2) // 2,), dtype=torch.int64)
    spec_rope_freqs(rot, base, SCALINGS[scaling], factor, original, low, high, _ptr(host))
    return host.to(device)


def _turn(freqs, interleaved, device):
    if (freqs.dtype != _torch().int64 or freqs.dim() != 1 or not freqs.is_contiguous() or
            freqs.get_device() != device):
        raise ValueError("freqs must be what rope_freqs returns, on cuda:%d" % device)
    return 2 * freqs.numel(), SPEC_ROPE_INTERLEAVED if interleaved else SPEC_ROPE_HALF


def _turned(x, out, name, H, D, stream):
    """out of a rotation of x [B, N, H, D] (None: a new tensor); both strides."""
    torch = _torch()
    step = _tokens(x, name, H, D, (torch.bfloat16, torch.float32))
    if out is None:
        return _made(stream, torch.empty_like, x, memory_format=torch.contiguous_format), step, H * D
    if out.shape != x.shape or out.get_device() != x.get_device():
        raise ValueError("out must have the shape and device of %s, got %s on %s"
                         % (name, tuple(out.shape), out.device))
    return out, step, _tokens(out, "out", H, D, (x.dtype,))


def rope(x, freqs, pos, first=0, amplitude=1.0, interleaved=False, inverse=False, out=None,
         stream=None):
    """Tensor-level spec_rope: x [B, N, H, D] (bf16 or fp32) at position indices
    pos [B, N] int32; the elements from `first` on that freqs (rope_freqs) covers
    are turned.  Returns out (out=x: in place)."""
    torch = _torch()
    B, N, H, D = x.shape
    out, step, out_step = _turned(x, out, "x", H, D, stream)
    device = x.get_device()
    rot, layout = _turn(freqs, interleaved, device)
    _lies(pos, "pos", torch.int32, (B, N), device)
    spec_rope(x.data_ptr(), step, out.data_ptr(), out_step, freqs.data_ptr(), rot, first, amplitude,
              layout, 1 if inverse else 0, pos.data_ptr(), B, N, H, D, _dtype_code(x),
              _launch(device, stream))
    return out


def kv_append_rope(cache, page_table, starts, k, v, freqs, q=None, rows=None, pos=None, amplitude=1.0,
                   interleaved=False, out_q=None, stream=None):
    """Tensor-level spec_kv_append_rope: kv_append with k turned to position
    indices pos [B, N] int32 (None: cache positions) on the way, and with q
    [B, N, Hq, D] the queries too.  Returns out_q, or None without q."""
    torch = _torch()
    c = cache.descriptor
    H, D = c.Hkv, c.D
    step = _tokens(k, "k", H, D, (torch.bfloat16, torch.float32))
    if v.shape != k.shape or _tokens(v, "v", H, D, (k.dtype,)) != step:
        raise ValueError("k and v must have one shape and token stride")
    B, N, _, _ = k.shape
    device = k.get_device()
    if v.get_device() != device or cache.k.get_device() != device:
        raise ValueError("k, v and the cache must be on one device")
    rot, layout = _turn(freqs, interleaved, device)
    M, width = N, page_table.shape[1]
    _lies(page_table, "page_table", torch.int32, (B, width), device)
    _lies(starts, "starts", torch.int32, (B,), device)
    if rows is not None:
        M = rows.shape[1]
        _lies(rows, "rows", torch.int32, (B, M), device)
    if pos is not None:
        _lies(pos, "pos", torch.int32, (B, N), device)
    q_step = out_step = Hq = 0
    if q is not None:
        if q.dtype != k.dtype or q.shape[:2] != (B, N) or q.get_device() != device:
            raise ValueError("q must be of k's type, tokens and device")
        Hq = q.shape[2]
        out_q, q_step, out_step = _turned(q, out_q, "q", Hq, D, stream)
    elif out_q is not None:
        raise ValueError("out_q without q")
    spec_kv_append_rope(c, page_table.data_ptr(), width, starts.data_ptr(), k.data_ptr(), v.data_ptr(),
                        step, _ptr(rows), _ptr(pos), freqs.data_ptr(), rot, amplitude, layout, _ptr(q),
                        q_step, _ptr(out_q), out_step, B, N, M, Hq, _dtype_code(k),
                        _launch(device, stream))
    return out_q


# ---------------------------------------------------------------- a latent cache

class LatentCache(collections.namedtuple("LatentCache", "data R")):
    """A paged latent cache: data [num_pages, page, C + R] bf16, the last R
    elements of a row the rotary part.  Checked once, here; the calls pass its C
    descriptor."""

    def __new__(cls, data, R=64):
        self = super().__new__(cls, data, R)
        n, page, width = data.shape
        _need(data, "data", _torch().bfloat16, (n, page, width))
        self.descriptor = LatentDescriptor(_ptr(data), n, page, width - R, R)
        return self

    @classmethod
    def _make(cls, fields):  # _replace comes here too
        return cls(*fields)

    def __reduce__(self):  # a copy's descriptor is of the copy's tensor
        return type(self), tuple(self)


def new_latent_cache(num_pages, page, C, device, R=64):
    """An empty (zeroed) latent cache of num_pages pages."""
    torch = _torch()
    return LatentCache(torch.zeros((num_pages, page, C + R), dtype=torch.bfloat16, device=device), R)


def latent_append(cache, page_table, starts, c, r, freqs=None, rows=None, pos=None, amplitude=1.0,
                  interleaved=False, stream=None):
    """Tensor-level spec_latent_append: tokens c [B, N, C] and r [B, N, R] (fp32 or
    bf16; parts of one projection, or tensors of their own) to positions
    starts[b] + t of a LatentCache, r turned to pos [B, N] (None: the cache
    positions) where freqs (rope_freqs(R)) are given; rows as in kv_append."""
    torch = _torch()
    d = cache.descriptor
    B, N = c.shape[:2]
    c_step = _parts(c, "c", d.C, (torch.bfloat16, torch.float32))
    r_step = _parts(r, "r", d.R, (c.dtype,))
    device = c.get_device()
    if r.shape[:2] != (B, N) or r.get_device() != device or cache.data.get_device() != device:
        raise ValueError("c and r must hold the same tokens, on the cache's device")
    rot, layout = (d.R, SPEC_ROPE_HALF) if freqs is None else _turn(freqs, interleaved, device)
    if rot != d.R:
        raise ValueError("freqs are of %d elements, the cache's rotary part has %d" % (rot, d.R))
    M, width = N, page_table.shape[1]
    _lies(page_table, "page_table", torch.int32, (B, width), device)
    _lies(starts, "starts", torch.int32, (B,), device)
    if rows is not None:
        M = rows.shape[1]
        _lies(rows, "rows", torch.int32, (B, M), device)
    if pos is not None:
        _lies(pos, "pos", torch.int32, (B, N), device)
    spec_latent_append(d, page_table.data_ptr(), width, starts.data_ptr(), c.data_ptr(), c_step,
                       r.data_ptr(), r_step, _ptr(rows), _ptr(pos), _ptr(freqs), amplitude, layout, B, N,
                       M, _dtype_code(c), _launch(device, stream))


def _parts(t, name, D, dtypes):
    """_tokens for [B, N, D], one vector a token."""
    if t.dim() == 3 and t.is_contiguous() and t.dtype in dtypes and t.is_cuda and t.shape[2] == D:
        return D
    return _tokens(t.unsqueeze(2), name, 1, D, dtypes)


def latent_attn(q, cache, page_table, lens, scale, mask=None, out=None, lse=None, workspace=None,
                stream=None):
    """Tensor-level spec_latent_attn: new tokens q [B, N, H, C + R] bf16 (each
    head's query with its key projection multiplied in, then the rotary part)
    over a LatentCache; mask as tree_mask returns it (None: a chain).  Returns out
    [B, N, H, C], or (out, lse) with lse=True or a tensor.  With ``stream``, what
    the call allocates belongs to that stream.  Data errors (last_error) are in
    the workspace: give one to read them."""
    torch = _torch()
    d = cache.descriptor
    B, N, H = q.shape[:3]
    C = d.C
    step = _tokens(q, "q", H, C + d.R, (torch.bfloat16,))
    device, width = q.get_device(), page_table.shape[1]
    if cache.data.get_device() != device:
        raise ValueError("q must be on the cache's device")
    _lies(page_table, "page_table", torch.int32, (B, width), device)
    _lies(lens, "lens", torch.int32, (B,), device)
    if mask is not None:
        _lies(mask, "mask", torch.uint8, (B, N, N), device)
    handle = _launch(device, stream)
    if out is None:
        out = _made(stream, torch.empty, (B, N, H, C), dtype=q.dtype, device=q.device)
    else:
        _lies(out, "out", q.dtype, (B, N, H, C), device)
    if lse is True:
        lse = _made(stream, torch.empty, (B, N, H), dtype=torch.float32, device=q.device)
    elif lse is False:
        lse = None
    elif lse is not None:
        _lies(lse, "lse", torch.float32, (B, N, H), device)
    if workspace is None:
        workspace = _made(stream, new_workspace, spec_latent_workspace_size(B, N, H, C), q.device)
    else:
        _room(workspace, device)
    spec_latent_attn(d, page_table.data_ptr(), width, lens.data_ptr(), q.data_ptr(), step, _ptr(mask), B,
                     N, H, scale, out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.numel(),
                     handle)
    return out if lse is None else (out, lse)
