"""Thin ctypes binding over libssm (include/ssm.h): argument marshalling only.

Every function takes CUDA torch tensors, checks their layouts, passes raw device
pointers, element strides and the current torch stream to the C ABI, and raises
``SSMError`` on a negative status.  All compute happens in libssm's kernels;
there is no CPU or PyTorch fallback, and a missing library or device is an error.
Output tensors are allocated with torch when the caller does not pass them.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from pathlib import Path

import torch

from .build import CALLS, LIB, STEP_CALLS

SSM_F32, SSM_BF16, SSM_I8 = 0, 1, 2
_STATUS = {0: "SSM_OK", -1: "SSM_ERR_INVALID_ARG", -2: "SSM_ERR_UNSUPPORTED", -3: "SSM_ERR_MISALIGNED",
           -4: "SSM_ERR_CUDA", -5: "SSM_ERR_DEVICE_TIMEOUT"}
DEV_WAIT_TIMEOUT, DEV_BAD_SLOT, DEV_BAD_INDEX = 1, 2, 8

EXPORTS = ("ssm_abi_version", "ssm_prefill", "ssm_prefill_workspace_bytes", "ssm_prefill_segmented",
           "ssm_prefill_segmented_noalloc", "ssm_decode_step", "ssm_decode_tokens", "ssm_out_proj_partial",
           "q8_reduce_partials", "q8_block_absmax", "q8_quantize_shared", "q8_sum_dequant",
           "ssd_prefill_workspace_bytes", "ssd_prefill", "ssd_decode_step",
           "attn_rope_table", "attn_append", "attn_cache_read", "attn_prefill", "attn_decode_workspace_bytes",
           "attn_decode_step", "norm_rms", "w4_quantize", "w4_linear_workspace_bytes", "w4_linear", "spec_probs",
           "spec_verify",
           "ssm_selftest_expire_wait", "ssm_selftest_expire_wait_of", "ssm_device_status", "ssm_last_error")
NOALLOC_SCRATCH_BYTES = 4 << 20     # SSM_NOALLOC_SCRATCH_BYTES


class SSMError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} -> {_STATUS.get(code, code)}: {msg}")
        self.code = code


_lib = None


def load(path: Path | str | None = None):
    """Load libssm.so (built by ``selective_state_space_prefill_gb300.build.build()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path else LIB
    if not p.exists():
        raise ImportError(f"libssm is not built ({p} missing): run "
                          "`python -c 'import __graft_entry__ as g; g.build()'` first")
    lib = ctypes.CDLL(str(p))
    P, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    lib.ssm_abi_version.argtypes = []
    lib.ssm_abi_version.restype = I
    lib.ssm_last_error.argtypes = []
    lib.ssm_last_error.restype = ctypes.c_char_p
    lib.ssm_prefill.argtypes = [I, I, I, I, I, I, I, P, P, P, L, L, P, P, P, P, P, P, P, P, P, L, L,
                                P, L, L, P, P, P]
    lib.ssm_prefill.restype = I
    lib.ssm_prefill_workspace_bytes.argtypes = [I, I, I, I]
    lib.ssm_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.ssm_prefill_segmented.argtypes = lib.ssm_prefill.argtypes[:-1] + [I, P, ctypes.c_size_t, P]
    lib.ssm_prefill_segmented.restype = I
    lib.ssm_prefill_segmented_noalloc.argtypes = lib.ssm_prefill.argtypes[:-1] + [I, P]
    lib.ssm_prefill_segmented_noalloc.restype = I
    lib.ssm_decode_step.argtypes = [I, I, I, I, I, I, P, P, P, L, P, P, P, P, P, P, P, P, P, L, L, I, P,
                                    P, L, P]
    lib.ssm_decode_step.restype = I
    lib.ssm_decode_tokens.argtypes = [I, I, I, I, I, I, I, P, P, P, L, L, P, P, P, P, P, P, P, P, P, L, L, I,
                                      P, P, L, L, P]
    lib.ssm_decode_tokens.restype = I
    lib.ssm_out_proj_partial.argtypes = [L, L, L, P, L, P, L, I, P, L, P, P]
    lib.ssm_out_proj_partial.restype = I
    lib.q8_reduce_partials.argtypes = [I, P, I, L, I, P, I, P, P, P]
    lib.q8_reduce_partials.restype = I
    lib.q8_block_absmax.argtypes = [P, I, L, I, P, P]
    lib.q8_block_absmax.restype = I
    lib.q8_quantize_shared.argtypes = [P, I, L, I, P, P, P, P]
    lib.q8_quantize_shared.restype = I
    lib.q8_sum_dequant.argtypes = [I, P, P, L, I, P, I, P, P]
    lib.q8_sum_dequant.restype = I
    lib.ssd_prefill_workspace_bytes.argtypes = [I, I, I, I]
    lib.ssd_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_prefill.argtypes = [I, I, I, I, I, I, I, I, I, P, L, L, P, L, L, P, L, L, P, P, P, P, P, P, P,
                                P, L, L, P, P, P, ctypes.c_size_t, P]
    lib.ssd_prefill.restype = I
    lib.ssd_decode_step.argtypes = [I, I, I, I, I, I, I, I, P, P, P, P, P, P, P, P, P, P, I, P, P, P]
    lib.ssd_decode_step.restype = I
    F, Z = ctypes.c_float, ctypes.c_size_t
    lib.attn_rope_table.argtypes = [L, I, P, ctypes.c_double, P, P, P]
    lib.attn_rope_table.restype = I
    lib.attn_append.argtypes = [L, I, I, I, I, I, P, L, L, P, L, L, P, L, L, P, P, P, L, P, I, P, P, P, P, I, I,
                                P, L, L, P, L, L, P]
    lib.attn_append.restype = I
    lib.attn_cache_read.argtypes = [I, L, I, I, I, P, P, P, P, I, I, P, L, I, P, P, I, P, P, P]
    lib.attn_cache_read.restype = I
    lib.attn_prefill.argtypes = [I, L, L, I, I, I, I, I, I, P, L, L, P, L, L, P, L, L, P, P, F, P, L, L, P, P]
    lib.attn_prefill.restype = I
    lib.attn_decode_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.attn_decode_workspace_bytes.restype = Z
    lib.attn_decode_step.argtypes = [I, I, I, I, I, I, P, L, L, I, P, P, P, P, I, I, P, L, I, P, I, F, P, L, L,
                                     P, P, Z, P]
    lib.attn_decode_step.restype = I
    lib.norm_rms.argtypes = [L, I, I, I, P, L, I, P, L, P, L, P, F, I, P, L, P, P]
    lib.norm_rms.restype = I
    lib.w4_quantize.argtypes = [L, L, I, I, P, L, P, L, I, P, L, P, L, P]
    lib.w4_quantize.restype = I
    lib.w4_linear.argtypes = [L, L, L, I, I, P, L, P, I, P, L, I, P, L, P, L, I, P, L, P, Z, P]
    lib.w4_linear.restype = I
    lib.w4_linear_workspace_bytes.argtypes = [L, L, L, I]
    lib.w4_linear_workspace_bytes.restype = Z
    lib.spec_probs.argtypes = [L, L, I, P, L, P, P, L, P]
    lib.spec_probs.restype = I
    lib.spec_verify.argtypes = [I, I, L, P, P, P, L, L, P, L, L, P, P, P, P]
    lib.spec_verify.restype = I
    lib.ssm_selftest_expire_wait.argtypes = [I, P]
    lib.ssm_selftest_expire_wait.restype = I
    lib.ssm_selftest_expire_wait_of.argtypes = [I, I, P]
    lib.ssm_selftest_expire_wait_of.restype = I
    lib.ssm_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), I]
    lib.ssm_device_status.restype = I
    if path is None:
        _lib = lib
    return lib


def _check(lib, fn: str, rc: int):
    if rc != 0:
        raise SSMError(fn, rc, lib.ssm_last_error().decode())


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return SSM_F32
    if t == torch.bfloat16:
        return SSM_BF16
    raise TypeError(f"unsupported dtype {t} (float32 or bfloat16)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on_stream(fn):
    """A call given ``stream`` runs with that stream current, so that outputs and workspaces made in it come
    from that stream's memory: a block of the current stream may be free there and still be used by work that
    has not run, and would be free again, on return, before the call has run.  New outputs are noted as used
    on the stream that was current, where the caller goes on with them."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        current = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
        given = {id(x) for x in (*args, *kw.values())}
        for t in out if isinstance(out, tuple) else (out,):
            if isinstance(t, torch.Tensor) and id(t) not in given:
                t.record_stream(current)
        return out
    return call


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libssm takes CUDA tensors only (no CPU path)")


def _chan_contig(t, name):
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must have channel stride 1")


def _param(t, shape, name):
    if t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be contiguous float32 {tuple(shape)}")


def _conv_state_layout(t, batch, d_inner, name):
    if t.dtype != torch.float32 or tuple(t.shape) != (batch, 3, d_inner) or t.stride(2) != 1 \
            or t.stride(0) != 3 * t.stride(1):
        raise ValueError(f"{name} must be float32 [batch, 3, d_inner] with rows of one stride")
    return t.stride(1)


def _ssm_state_layout(t, batch, d_inner, name):
    if t.dtype != torch.float32 or tuple(t.shape) != (batch, d_inner, 16) or t.stride(2) != 1 \
            or t.stride(1) != 16:
        raise ValueError(f"{name} must be float32 [batch, d_inner, 16] with channel stride 16")
    return t.stride(0)


def prefill_workspace_bytes(batch: int, seqlen: int, d_inner: int, seg_len: int) -> int:
    """ssm_prefill_workspace_bytes: device bytes the segmented prefill needs."""
    return int(load().ssm_prefill_workspace_bytes(batch, seqlen, d_inner, seg_len))


def suggest_seg_len(batch: int, seqlen: int, d_inner: int, n_sm: int, ctas_per_sm: int = 3) -> int | None:
    """A segment length that brings batch x ceil(d_inner/16) x segments close to the GPU's
    resident CTA slots, or None when the rows already fill it.  The choice depends on
    d_inner, so channel-slice runs that must match bit for bit pass one seg_len explicitly."""
    rows = batch * ((d_inner + 15) // 16)
    slots = n_sm * ctas_per_sm
    n_seg = min(slots // rows if rows else 1, (seqlen + 63) // 64)
    if n_seg < 2:
        return None
    return ((seqlen + n_seg - 1) // n_seg + 63) // 64 * 64


@_on_stream
def prefill(x, z, dt, B, C, A, D, dt_bias, conv_w, conv_b, conv_state_in=None, ssm_state_in=None,
            out=None, out_dtype=torch.float32, conv_state_out=None, ssm_state_out=None, stream=None,
            seg_len=None, workspace=None, noalloc=False):
    """ssm_prefill over [batch, L, d_inner] x/z/dt (channel-stride-1 views allowed).

    With ``seg_len`` (a multiple of 64) the rows are cut into segments that run in parallel
    (ssm_prefill_segmented); ``workspace`` is then a CUDA uint8 tensor of at least
    prefill_workspace_bytes(...) bytes, allocated here with torch when not given.  With
    ``noalloc=True`` (and ``seg_len``) the call is ssm_prefill_segmented_noalloc: the scratch
    is the library's fixed array of NOALLOC_SCRATCH_BYTES and no workspace is allocated.
    Returns (out, conv_state_out, ssm_state_out).
    """
    lib = load()
    _need_cuda(x, z, dt, B, C, A, D, dt_bias, conv_w, conv_b, conv_state_in, ssm_state_in)
    batch, L, d_inner = x.shape
    if z.shape != x.shape or dt.shape != x.shape or z.stride() != x.stride() or dt.stride() != x.stride():
        raise ValueError("x, z, dt must share shape and strides")
    if z.dtype != x.dtype or dt.dtype != x.dtype or B.dtype != x.dtype or C.dtype != x.dtype:
        raise ValueError("x, z, dt, B, C must share one dtype")
    for t, n in ((x, "x"),):
        _chan_contig(t, n)
    for t, n in ((B, "B"), (C, "C")):
        if tuple(t.shape) != (batch, L, 16) or not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous [batch, L, 16]")
    _param(A, (d_inner, 16), "A")
    for t, n in ((D, "D"), (dt_bias, "dt_bias"), (conv_b, "conv_b")):
        _param(t, (d_inner,), n)
    _param(conv_w, (d_inner, 4), "conv_w")
    dev = x.device
    if out is None:
        out = torch.empty(batch, L, d_inner, device=dev, dtype=out_dtype)
    _chan_contig(out, "out")
    if conv_state_out is None:
        conv_state_out = torch.empty(batch, 3, d_inner, device=dev, dtype=torch.float32)
    if ssm_state_out is None:
        ssm_state_out = torch.empty(batch, d_inner, 16, device=dev, dtype=torch.float32)
    ld = _conv_state_layout(conv_state_out, batch, d_inner, "conv_state_out")
    sb = _ssm_state_layout(ssm_state_out, batch, d_inner, "ssm_state_out")
    if conv_state_in is not None and _conv_state_layout(conv_state_in, batch, d_inner, "conv_state_in") != ld:
        raise ValueError("conv_state_in and conv_state_out must share the row stride")
    if ssm_state_in is not None and _ssm_state_layout(ssm_state_in, batch, d_inner, "ssm_state_in") != sb:
        raise ValueError("ssm_state_in and ssm_state_out must share the batch stride")
    args = (batch, L, d_inner, 16, 4, _dtype_code(x.dtype), _dtype_code(out.dtype),
            _ptr(x), _ptr(z), _ptr(dt), x.stride(0), x.stride(1), _ptr(B), _ptr(C),
            _ptr(A), _ptr(D), _ptr(dt_bias), _ptr(conv_w), _ptr(conv_b),
            _ptr(conv_state_in), _ptr(ssm_state_in), ld, sb,
            _ptr(out), out.stride(0), out.stride(1),
            _ptr(conv_state_out), _ptr(ssm_state_out))
    if seg_len is None:
        rc = lib.ssm_prefill(*args, _stream(stream))
        _check(lib, "ssm_prefill", rc)
        return out, conv_state_out, ssm_state_out
    if noalloc:
        if workspace is not None:
            raise ValueError("noalloc=True takes no workspace")
        rc = lib.ssm_prefill_segmented_noalloc(*args, int(seg_len), _stream(stream))
        _check(lib, "ssm_prefill_segmented_noalloc", rc)
        return out, conv_state_out, ssm_state_out
    need = int(lib.ssm_prefill_workspace_bytes(batch, L, d_inner, int(seg_len)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    if workspace is not None:
        _need_cuda(workspace)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.ssm_prefill_segmented(*args, int(seg_len), _ptr(workspace), ws_bytes, _stream(stream))
    _check(lib, "ssm_prefill_segmented", rc)
    return out, conv_state_out, ssm_state_out


@_on_stream
def decode_step(x, z, dt, B, C, A, D, dt_bias, conv_w, conv_b, conv_state, ssm_state, state_slot=None,
                out=None, out_dtype=torch.float32, stream=None):
    """ssm_decode_step: x/z/dt [batch, d_inner], B/C [batch, 16]; states updated in place.

    conv_state [n_slots, 3, d_inner], ssm_state [n_slots, d_inner, 16] (channel-slice views allowed).
    Returns out [batch, d_inner].
    """
    lib = load()
    _need_cuda(x, z, dt, B, C, A, D, dt_bias, conv_w, conv_b, conv_state, ssm_state, state_slot)
    batch, d_inner = x.shape
    if z.shape != x.shape or dt.shape != x.shape or z.stride() != x.stride() or dt.stride() != x.stride():
        raise ValueError("x, z, dt must share shape and strides")
    _chan_contig(x, "x")
    for t, n in ((B, "B"), (C, "C")):
        if tuple(t.shape) != (batch, 16) or not t.is_contiguous() or t.dtype != x.dtype:
            raise ValueError(f"{n} must be contiguous [batch, 16] of the input dtype")
    _param(A, (d_inner, 16), "A")
    for t, n in ((D, "D"), (dt_bias, "dt_bias"), (conv_b, "conv_b")):
        _param(t, (d_inner,), n)
    _param(conv_w, (d_inner, 4), "conv_w")
    n_slots = conv_state.shape[0]
    if ssm_state.shape[0] != n_slots:
        raise ValueError("conv_state and ssm_state must have the same number of slots")
    ld = _conv_state_layout(conv_state, n_slots, d_inner, "conv_state")
    sb = _ssm_state_layout(ssm_state, n_slots, d_inner, "ssm_state")
    if state_slot is not None and (state_slot.dtype != torch.int32 or tuple(state_slot.shape) != (batch,)
                                   or not state_slot.is_contiguous()):
        raise ValueError("state_slot must be contiguous int32 [batch]")
    if out is None:
        out = torch.empty(batch, d_inner, device=x.device, dtype=out_dtype)
    _chan_contig(out, "out")
    rc = lib.ssm_decode_step(batch, d_inner, 16, 4, _dtype_code(x.dtype), _dtype_code(out.dtype),
                             _ptr(x), _ptr(z), _ptr(dt), x.stride(0), _ptr(B), _ptr(C),
                             _ptr(A), _ptr(D), _ptr(dt_bias), _ptr(conv_w), _ptr(conv_b),
                             _ptr(conv_state), _ptr(ssm_state), ld, sb, n_slots, _ptr(state_slot),
                             _ptr(out), out.stride(0), _stream(stream))
    _check(lib, "ssm_decode_step", rc)
    return out


@_on_stream
def decode_tokens(x, z, dt, B, C, A, D, dt_bias, conv_w, conv_b, conv_state, ssm_state, state_slot=None,
                  out=None, out_dtype=torch.float32, stream=None):
    """ssm_decode_tokens: x/z/dt [batch, T, d_inner] (channel-stride-1 views), B/C [batch, T, 16];
    the cached states (as for decode_step) advance T tokens in place.  Returns out [batch, T, d_inner]."""
    lib = load()
    _need_cuda(x, z, dt, B, C, A, D, dt_bias, conv_w, conv_b, conv_state, ssm_state, state_slot)
    batch, T, d_inner = x.shape
    if z.shape != x.shape or dt.shape != x.shape or z.stride() != x.stride() or dt.stride() != x.stride():
        raise ValueError("x, z, dt must share shape and strides")
    _chan_contig(x, "x")
    for t, n in ((B, "B"), (C, "C")):
        if tuple(t.shape) != (batch, T, 16) or not t.is_contiguous() or t.dtype != x.dtype:
            raise ValueError(f"{n} must be contiguous [batch, T, 16] of the input dtype")
    _param(A, (d_inner, 16), "A")
    for t, n in ((D, "D"), (dt_bias, "dt_bias"), (conv_b, "conv_b")):
        _param(t, (d_inner,), n)
    _param(conv_w, (d_inner, 4), "conv_w")
    n_slots = conv_state.shape[0]
    if ssm_state.shape[0] != n_slots:
        raise ValueError("conv_state and ssm_state must have the same number of slots")
    ld = _conv_state_layout(conv_state, n_slots, d_inner, "conv_state")
    sb = _ssm_state_layout(ssm_state, n_slots, d_inner, "ssm_state")
    if state_slot is not None and (state_slot.dtype != torch.int32 or tuple(state_slot.shape) != (batch,)
                                   or not state_slot.is_contiguous()):
        raise ValueError("state_slot must be contiguous int32 [batch]")
    if out is None:
        out = torch.empty(batch, T, d_inner, device=x.device, dtype=out_dtype)
    _chan_contig(out, "out")
    rc = lib.ssm_decode_tokens(batch, T, d_inner, 16, 4, _dtype_code(x.dtype), _dtype_code(out.dtype),
                               _ptr(x), _ptr(z), _ptr(dt), x.stride(0), x.stride(1), _ptr(B), _ptr(C),
                               _ptr(A), _ptr(D), _ptr(dt_bias), _ptr(conv_w), _ptr(conv_b),
                               _ptr(conv_state), _ptr(ssm_state), ld, sb, n_slots, _ptr(state_slot),
                               _ptr(out), out.stride(0), out.stride(1), _stream(stream))
    _check(lib, "ssm_decode_tokens", rc)
    return out


@_on_stream
def q8_reduce(partials, block=128, out=None, out_dtype=None, sums=None, scales=None, stream=None):
    """q8_reduce_partials over P equal-shaped partial tensors (flattened).

    Returns (out, sums, scales); pass sums=False / scales=False to skip writing them.
    """
    lib = load()
    _need_cuda(*partials)
    P = len(partials)
    shape, dtype = partials[0].shape, partials[0].dtype
    for p in partials:
        if p.shape != shape or p.dtype != dtype or not p.is_contiguous():
            raise ValueError("partials must be contiguous tensors of one shape and dtype")
    n = partials[0].numel()
    dev = partials[0].device
    out_dtype = out_dtype or dtype
    if out is None:
        out = torch.empty(shape, device=dev, dtype=out_dtype)
    if sums is None:
        sums = torch.empty(n, device=dev, dtype=torch.int32)
    if scales is None:
        scales = torch.empty((n + block - 1) // block, device=dev, dtype=torch.float32)
    sums = sums if sums is not False else None
    scales = scales if scales is not False else None
    ptrs = (ctypes.c_void_p * P)(*[p.data_ptr() for p in partials])
    rc = lib.q8_reduce_partials(P, ctypes.cast(ptrs, ctypes.c_void_p), _dtype_code(dtype), n, block,
                                _ptr(out), _dtype_code(out.dtype), _ptr(sums), _ptr(scales), _stream(stream))
    _check(lib, "q8_reduce_partials", rc)
    return out, sums, scales


@_on_stream
def q8_block_absmax(x, block=128, out=None, stream=None):
    """q8_block_absmax: per-128-block maxima of |x| (x flattened, contiguous) -> float32 [nblk]."""
    lib = load()
    _need_cuda(x, out)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    n = x.numel()
    if out is None:
        out = torch.empty((n + block - 1) // block, device=x.device, dtype=torch.float32)
    rc = lib.q8_block_absmax(_ptr(x), _dtype_code(x.dtype), n, block, _ptr(out), _stream(stream))
    _check(lib, "q8_block_absmax", rc)
    return out


@_on_stream
def q8_quantize_shared(x, block_amax, block=128, codes=None, scales=None, stream=None):
    """q8_quantize_shared: int8 codes of x with the shared per-block maxima.

    Returns (codes int8 shaped like x, scales float32 [nblk]); pass scales=False to skip them.
    """
    lib = load()
    _need_cuda(x, block_amax, codes)
    if not x.is_contiguous() or not block_amax.is_contiguous() or block_amax.dtype != torch.float32:
        raise ValueError("x and block_amax (float32) must be contiguous")
    n = x.numel()
    nblk = (n + block - 1) // block
    if block_amax.numel() != nblk:
        raise ValueError(f"block_amax holds {block_amax.numel()} maxima, {nblk} needed")
    if codes is None:
        codes = torch.empty(x.shape, device=x.device, dtype=torch.int8)
    if scales is None:
        scales = torch.empty(nblk, device=x.device, dtype=torch.float32)
    scales = scales if scales is not False else None
    rc = lib.q8_quantize_shared(_ptr(x), _dtype_code(x.dtype), n, block, _ptr(block_amax), _ptr(codes),
                                _ptr(scales), _stream(stream))
    _check(lib, "q8_quantize_shared", rc)
    return codes, scales


@_on_stream
def q8_sum_dequant(codes, scales, block=128, out=None, out_dtype=torch.float32, sums=None, stream=None):
    """q8_sum_dequant over P equal-shaped int8 code tensors with their shared scales.

    Returns (out, sums int32 [n]); pass sums=False to skip them.
    """
    lib = load()
    _need_cuda(*codes, scales, out)
    P = len(codes)
    shape = codes[0].shape
    for c in codes:
        if c.shape != shape or c.dtype != torch.int8 or not c.is_contiguous():
            raise ValueError("codes must be contiguous int8 tensors of one shape")
    n = codes[0].numel()
    dev = codes[0].device
    if out is None:
        out = torch.empty(shape, device=dev, dtype=out_dtype)
    if sums is None:
        sums = torch.empty(n, device=dev, dtype=torch.int32)
    sums = sums if sums is not False else None
    ptrs = (ctypes.c_void_p * P)(*[c.data_ptr() for c in codes])
    rc = lib.q8_sum_dequant(P, ctypes.cast(ptrs, ctypes.c_void_p), _ptr(scales), n, block, _ptr(out),
                            _dtype_code(out.dtype), _ptr(sums), _stream(stream))
    _check(lib, "q8_sum_dequant", rc)
    return out, sums


def device_status(clear: bool = True) -> int:
    """The device status word (OR of DEV_* bits); synchronises the device."""
    lib = load()
    v = ctypes.c_uint32(0)
    _check(lib, "ssm_device_status", lib.ssm_device_status(ctypes.byref(v), 1 if clear else 0))
    return int(v.value)


@_on_stream
def out_proj_partial(y, W, out=None, out_dtype=torch.bfloat16, block_amax=True, stream=None):
    """ssm_out_proj_partial: y [M, K] bf16 and W [N, K] bf16 (row views with stride-1 K).

    Returns (out [M, N], block_amax [M*N/128] float32 or None).
    """
    lib = load()
    _need_cuda(y, W, out)
    if y.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError("y and W must be bfloat16")
    if y.dim() != 2 or W.dim() != 2 or y.stride(1) != 1 or W.stride(1) != 1 or y.shape[1] != W.shape[1]:
        raise ValueError("y [M, K] and W [N, K] must be 2-D with a stride-1 K dimension")
    M, K = y.shape
    N = W.shape[0]
    if out is None:
        out = torch.empty(M, N, device=y.device, dtype=out_dtype)
    if out.dim() != 2 or tuple(out.shape) != (M, N) or out.stride(1) != 1:
        raise ValueError("out must be [M, N] with a stride-1 N dimension")
    amax = None
    if block_amax is True:
        amax = torch.empty((M * N + 127) // 128, device=y.device, dtype=torch.float32)
    elif block_amax is not None and block_amax is not False:
        amax = block_amax
    rc = lib.ssm_out_proj_partial(M, N, K, _ptr(y), y.stride(0), _ptr(W), W.stride(0), _dtype_code(out.dtype),
                                  _ptr(out), out.stride(0), _ptr(amax), _stream(stream))
    _check(lib, "ssm_out_proj_partial", rc)
    return out, amax


def selftest_expire_wait(limit_us: int = 50000, stream=None, which: int = 0) -> None:
    """ssm_selftest_expire_wait: one kernel whose bounded wait expires after limit_us.  ``which``
    (ssm_selftest_expire_wait_of) 0: a copy's; 1: those of w4_linear; 2: spec_probs's and spec_verify's."""
    lib = load()
    _check(lib, "ssm_selftest_expire_wait_of", lib.ssm_selftest_expire_wait_of(int(which), int(limit_us), _stream(stream)))


# ------------------------------------------------------------------ SSD (Mamba-2-style) mixer
def _ssd_dims(n_heads, n_groups, head_dim=64, d_state=64):
    return n_heads * head_dim, n_heads * head_dim + 2 * n_groups * d_state


def ssd_prefill_workspace_bytes(batch: int, seqlen: int, n_heads: int, n_groups: int) -> int:
    """ssd_prefill_workspace_bytes: device bytes ssd_prefill needs."""
    return int(load().ssd_prefill_workspace_bytes(batch, seqlen, n_heads, n_groups))


def _ssd_params(conv_w, conv_b, A, D, dt_bias, H, Cx):
    _param(conv_w, (Cx, 4), "conv_w")
    _param(conv_b, (Cx,), "conv_b")
    for t, n in ((A, "A"), (D, "D"), (dt_bias, "dt_bias")):
        _param(t, (H,), n)


def _ssd_states(t, batch, H, Cx, name, conv):
    shape = (batch, 3, Cx) if conv else (batch, H, 64, 64)
    if t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 {shape}")


@_on_stream
def ssd_prefill(xBC, z, dt, conv_w, conv_b, A, D, dt_bias, n_heads, n_groups, conv_state_in=None,
                ssm_state_in=None, out=None, out_dtype=torch.float32, conv_state_out=None, ssm_state_out=None,
                workspace=None, stream=None):
    """ssd_prefill: xBC [batch, L, 64 H + 128 G], z [batch, L, 64 H], dt [batch, L, H] bf16
    (channel-stride-1 views), head_dim = d_state = 64.  ``workspace`` (a CUDA uint8 tensor of at
    least ssd_prefill_workspace_bytes(batch, L, n_heads, n_groups) bytes) is allocated here with torch when not given.
    Returns (out [batch, L, 64 H], conv_state_out [batch, 3, Cx], ssm_state_out [batch, H, 64, 64])."""
    lib = load()
    _need_cuda(xBC, z, dt, conv_w, conv_b, A, D, dt_bias, conv_state_in, ssm_state_in)
    H, G = int(n_heads), int(n_groups)
    HP, Cx = _ssd_dims(H, G)
    batch, L, cx = xBC.shape
    if cx != Cx or tuple(z.shape) != (batch, L, HP) or tuple(dt.shape) != (batch, L, H):
        raise ValueError("xBC, z, dt shapes disagree with n_heads / n_groups")
    if z.dtype != xBC.dtype or dt.dtype != xBC.dtype:
        raise ValueError("xBC, z, dt must share one dtype")
    for t, n in ((xBC, "xBC"), (z, "z"), (dt, "dt")):
        _chan_contig(t, n)
    _ssd_params(conv_w, conv_b, A, D, dt_bias, H, Cx)
    dev = xBC.device
    if out is None:
        out = torch.empty(batch, L, HP, device=dev, dtype=out_dtype)
    _chan_contig(out, "out")
    if conv_state_out is None:
        conv_state_out = torch.empty(batch, 3, Cx, device=dev, dtype=torch.float32)
    if ssm_state_out is None:
        ssm_state_out = torch.empty(batch, H, 64, 64, device=dev, dtype=torch.float32)
    for t, n, c in ((conv_state_out, "conv_state_out", True), (ssm_state_out, "ssm_state_out", False),
                    (conv_state_in, "conv_state_in", True), (ssm_state_in, "ssm_state_in", False)):
        if t is not None:
            _ssd_states(t, batch, H, Cx, n, c)
    need = int(lib.ssd_prefill_workspace_bytes(batch, L, H, G))
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=dev, dtype=torch.uint8)
    _need_cuda(workspace)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    rc = lib.ssd_prefill(batch, L, H, 64, G, 64, 4, _dtype_code(xBC.dtype), _dtype_code(out.dtype),
                         _ptr(xBC), xBC.stride(0), xBC.stride(1), _ptr(z), z.stride(0), z.stride(1),
                         _ptr(dt), dt.stride(0), dt.stride(1), _ptr(conv_w), _ptr(conv_b), _ptr(A), _ptr(D),
                         _ptr(dt_bias), _ptr(conv_state_in), _ptr(ssm_state_in), _ptr(out), out.stride(0),
                         out.stride(1), _ptr(conv_state_out), _ptr(ssm_state_out), _ptr(workspace),
                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check(lib, "ssd_prefill", rc)
    return out, conv_state_out, ssm_state_out


@_on_stream
def ssd_decode_step(xBC, z, dt, conv_w, conv_b, A, D, dt_bias, n_heads, n_groups, conv_state, ssm_state,
                    state_slot=None, out=None, out_dtype=torch.float32, stream=None):
    """ssd_decode_step: xBC [batch, Cx], z [batch, 64 H], dt [batch, H] (contiguous); the cached
    states conv_state [n_slots, 3, Cx] and ssm_state [n_slots, H, 64, 64] advance one token in
    place.  Returns out [batch, 64 H]."""
    lib = load()
    _need_cuda(xBC, z, dt, conv_w, conv_b, A, D, dt_bias, conv_state, ssm_state, state_slot)
    H, G = int(n_heads), int(n_groups)
    HP, Cx = _ssd_dims(H, G)
    batch = xBC.shape[0]
    if tuple(xBC.shape) != (batch, Cx) or tuple(z.shape) != (batch, HP) or tuple(dt.shape) != (batch, H):
        raise ValueError("xBC, z, dt shapes disagree with n_heads / n_groups")
    if z.dtype != xBC.dtype or dt.dtype != xBC.dtype:
        raise ValueError("xBC, z, dt must share one dtype")
    for t, n in ((xBC, "xBC"), (z, "z"), (dt, "dt")):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _ssd_params(conv_w, conv_b, A, D, dt_bias, H, Cx)
    n_slots = conv_state.shape[0]
    _ssd_states(conv_state, n_slots, H, Cx, "conv_state", True)
    _ssd_states(ssm_state, n_slots, H, Cx, "ssm_state", False)
    if state_slot is not None and (state_slot.dtype != torch.int32 or tuple(state_slot.shape) != (batch,)
                                   or not state_slot.is_contiguous()):
        raise ValueError("state_slot must be contiguous int32 [batch]")
    if out is None:
        out = torch.empty(batch, HP, device=xBC.device, dtype=out_dtype)
    if not out.is_contiguous() or tuple(out.shape) != (batch, HP):
        raise ValueError("out must be contiguous [batch, 64 H]")
    rc = lib.ssd_decode_step(batch, H, 64, G, 64, 4, _dtype_code(xBC.dtype), _dtype_code(out.dtype),
                             _ptr(xBC), _ptr(z), _ptr(dt), _ptr(conv_w), _ptr(conv_b), _ptr(A), _ptr(D),
                             _ptr(dt_bias), _ptr(conv_state), _ptr(ssm_state), n_slots, _ptr(state_slot),
                             _ptr(out), _stream(stream))
    _check(lib, "ssd_decode_step", rc)
    return out


# ------------------------------------------------------------------ attention (hybrid layers)
# The tensors of a call lie on one GPU, which need not be the current one.  With ``stream`` the call runs on
# that stream, which the caller makes wait for its inputs; outputs made here come from that stream's memory
# and may be used on the current stream once it waits for that one.
_calls = None


def _extension(path, entries):
    """An extension of the build that marshals calls, with libssm's entry points handed over."""
    import importlib.machinery
    import importlib.util

    if not path.exists():
        raise ImportError(f"{path.stem} is not built ({path} missing): run "
                          "`python -c 'import __graft_entry__ as g; g.build()'` first")
    loader = importlib.machinery.ExtensionFileLoader(path.stem, str(path))
    mod = importlib.util.module_from_spec(importlib.util.spec_from_loader(path.stem, loader))
    loader.exec_module(mod)
    lib = load()
    mod.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in entries))
    return mod


def attn_calls():
    """The extension that marshals the attention calls (csrc/attn_call.cpp): it checks the tensors,
    allocates missing outputs and calls libssm, in the microsecond that a short step allows."""
    global _calls
    if _calls is None:
        _calls = _extension(CALLS, ("attn_append", "attn_cache_read", "attn_prefill", "attn_decode_workspace_bytes",
                                    "attn_decode_step"))
    return _calls


def _outcome(r, fn):
    """What an extension's call returned: its outputs, or the status of its refusal."""
    if type(r) is int:
        raise SSMError(fn, r, load().ssm_last_error().decode())
    return r


def _raw(stream):
    return None if stream is None else stream.cuda_stream


@_on_stream
def attn_rope_table(inv_freq, n_pos, scale=1.0, device="cuda", stream=None):
    """attn_rope_table: (cos, sin) float32 [n_pos, half] for positions 0 .. n_pos-1; ``inv_freq`` is a
    sequence of half floats (see rope.rope_frequencies)."""
    lib = load()
    freqs = [float(f) for f in inv_freq]
    arr = (ctypes.c_double * max(1, len(freqs)))(*freqs)
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("libssm takes CUDA tensors only (no CPU path)")
    with torch.cuda.device(dev):                # the library works on the current device
        cos = torch.empty(n_pos, len(freqs), device=dev, dtype=torch.float32)
        sin = torch.empty_like(cos)
        rc = lib.attn_rope_table(n_pos, len(freqs), ctypes.cast(arr, ctypes.c_void_p), float(scale), _ptr(cos),
                                 _ptr(sin), _stream(stream))
        _check(lib, "attn_rope_table", rc)
    return cos, sin


def attn_append(q, k, v, positions, cos, sin, k_cache, v_cache, slots, k_scale=None, v_scale=None,
                interleaved=False, q_out=None, k_out=None, stream=None):
    """attn_append: rotate q [T, H, D] and k [T, Hk, D] (bf16 views) by positions [T] int32 and write k and
    v [T, Hk, D] into the paged cache at slots [T] int32 (page * page_size + row; -1: a padding token).

    k_cache, v_cache [n_pages, Hk, page_size, D] int8 (with k_scale, v_scale [n_pages, Hk, page_size]
    float32) or bfloat16, updated in place.  cos, sin [n_pos, rot_dim / 2] float32; None leaves the heads
    unrotated.  q may be None.  q_out may be q and k_out may be k; ``k_out=True`` allocates the rotated
    keys.  Returns (q_out, k_out), None for what was not asked."""
    return _outcome((_calls or attn_calls()).append(q, k, v, positions, cos, sin, k_cache, v_cache, slots, k_scale,
                                                    v_scale, interleaved, q_out, k_out, _raw(stream)), "attn_append")


def attn_cache_read(k_cache, v_cache, page_table, cu_len, n_tokens, k_scale=None, v_scale=None, first=None,
                    k_out=None, v_out=None, out_dtype=torch.bfloat16, stream=None):
    """attn_cache_read: the cached rows of every sequence back as packed (k, v) [n_tokens, Hk, D].

    page_table [batch, pages] int32; cu_len [batch + 1] int32, cu_len[batch] = n_tokens; first [batch]
    int32 names each sequence's first token read (None: 0).  k_out and v_out are contiguous, bfloat16 or
    float32 (``out_dtype`` when allocated here)."""
    return _outcome((_calls or attn_calls()).read(k_cache, v_cache, page_table, cu_len, n_tokens, k_scale, v_scale, first,
                                                  k_out, v_out, out_dtype, _raw(stream)), "attn_cache_read")


def attn_prefill(q, k, v, cu_q, cu_k, max_q, scale=None, out=None, out_dtype=torch.bfloat16, lse=None, stream=None):
    """attn_prefill: causal attention of packed sequences; q [Tq, H, D], k and v [Tk, Hk, D] bf16 views,
    cu_q and cu_k [batch + 1] int32, max_q an upper bound of the sequences' query rows.  A sequence's last
    query sees its last key.  ``scale`` defaults to head_dim ** -0.5; ``lse=True`` also returns the log of
    each row's softmax sum [Tq, H] float32.  Returns (out, lse)."""
    return _outcome((_calls or attn_calls()).prefill(q, k, v, cu_q, cu_k, max_q, scale, out, out_dtype, lse, _raw(stream)),
                    "attn_prefill")


def attn_decode_workspace_bytes(batch: int, n_heads: int, kv_heads: int, head_dim: int, max_len: int) -> int:
    """attn_decode_workspace_bytes: device bytes attn_decode_step needs."""
    return int(load().attn_decode_workspace_bytes(batch, n_heads, kv_heads, head_dim, max_len))


def attn_decode_step(q, k_cache, v_cache, page_table, lens, max_len, k_scale=None, v_scale=None, scale=None, out=None,
                     out_dtype=torch.bfloat16, lse=None, workspace=None, stream=None):
    """attn_decode_step: one query token per request, q [batch, H, D] bf16, over its lens[r] cached tokens
    (lens [batch] int32, at most max_len).  The cache and page_table are as for attn_cache_read.
    ``workspace`` (a CUDA uint8 tensor of at least attn_decode_workspace_bytes(...) bytes) is allocated
    here with torch when not given.  Returns (out, lse)."""
    return _outcome((_calls or attn_calls()).decode(q, k_cache, v_cache, page_table, lens, max_len, k_scale, v_scale, scale,
                                                    out, out_dtype, lse, workspace, _raw(stream)), "attn_decode_step")


# ------------------------------------------------------------------ around the mixers of a decode step
# The norm between blocks, projections with 4-bit weights, and the verification of drafted tokens.  Devices and
# streams are as for the attention calls.
_steps = None


def step_calls():
    """The extension that marshals these calls (csrc/step_call.cpp)."""
    global _steps
    if _steps is None:
        _steps = _extension(STEP_CALLS, ("norm_rms", "w4_quantize", "w4_linear_workspace_bytes", "w4_linear", "spec_probs", "spec_verify"))
    return _steps


def norm_rms(x, weight=None, residual=None, eps=1e-5, n_groups=1, out=None, out_dtype=torch.bfloat16, residual_out=None,
             out_scale=None, stream=None):
    """norm_rms: r = x + residual, and r / sqrt(mean(r^2) + eps) * weight over the row or over ``n_groups`` equal
    groups of its channels.

    x [rows, width] bfloat16 or float32; weight [width] float32; residual like x, bfloat16 or float32.
    ``residual_out`` takes r in residual's dtype: allocated when not given, residual itself for in place, False to
    skip it.  ``out_dtype`` bfloat16, float32, or int8 with a scale per row and group (out_scale [rows, n_groups]
    float32), which is what w4_linear takes as x and x_scale; with int8 a group that holds a NaN or an infinity
    reads as zeros.  Returns (out, residual_out, out_scale), None for what there is not."""
    return _outcome((_steps or step_calls()).norm(x, weight, residual, eps, n_groups, out, out_dtype, residual_out, out_scale,
                                                  _raw(stream)), "norm_rms")


def w4_quantize(W, group=128, zeros=False, scale_dtype=torch.bfloat16, stream=None):
    """w4_quantize: W [N, K] (bfloat16 or float32) to 4 bits, ``group`` (32, 64 or 128) elements of a row sharing a
    scale and, with ``zeros``, a zero.  Returns (codes [N, K / 2] uint8, even elements in the low half; scales
    [N, K / group] bfloat16 or float32; zeros [N, K / group] uint8 or None), rows padded to 16 bytes."""
    return _outcome((_steps or step_calls()).quantize(W, group, zeros, scale_dtype, _raw(stream)), "w4_quantize")


def w4_linear_workspace_bytes(M: int, N: int, K: int, group: int) -> int:
    """w4_linear_workspace_bytes: device bytes w4_linear needs."""
    return int(load().w4_linear_workspace_bytes(M, N, K, group))


def w4_linear(x, codes, scales, zeros=None, x_scale=None, out=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """w4_linear: x [M, K] times the transpose of a 4-bit weight (w4_quantize's layout), for the few rows (up to
    256) of a decode step.  x is bfloat16, or int8 with x_scale [M] or [M, blocks] float32 (norm_rms's).  ``zeros``
    None stands for 8.  ``workspace`` (a CUDA uint8 tensor of at least w4_linear_workspace_bytes(...) bytes) is
    allocated here with torch when not given.  Returns out [M, N] (bfloat16 or float32)."""
    return _outcome((_steps or step_calls()).linear(x, codes, scales, zeros, x_scale, out, out_dtype, workspace, _raw(stream)),
                    "w4_linear")[0]


def spec_probs(logits, temperature=None, out=None, stream=None):
    """spec_probs: probabilities [rows, vocab] float32 of logits [rows, vocab] (bfloat16 or float32) at the rows'
    temperatures [rows] float32 (None: 1; 0: greedy, the first largest logit)."""
    return _outcome((_steps or step_calls()).probs(logits, temperature, out, _raw(stream)), "spec_probs")[0]


def spec_verify(draft, target_probs, u, draft_probs=None, n_draft=None, tokens=None, n_kept=None, stream=None):
    """spec_verify: drafted tokens against the target's probabilities.

    draft [batch, n] int32; target_probs [batch, n + 1, vocab] float32, at the drafted places and after them; u
    [batch, n + 1] float32, uniform in [0, 1); draft_probs [batch, n, vocab] float32 that the drafts were drawn
    with (None: they were certain); n_draft [batch] int32, how many of the n a request has (None: all).  n may be
    0: a token is drawn from target_probs.  Returns (tokens [batch, n + 1] int32: the kept drafts, the next token,
    then -1; n_kept [batch] int32)."""
    return _outcome((_steps or step_calls()).verify(draft, target_probs, u, draft_probs, n_draft, tokens, n_kept, _raw(stream)),
                    "spec_verify")
