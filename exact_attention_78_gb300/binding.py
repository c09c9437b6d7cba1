"""ctypes binding of the C ABI (include/fa.h, include/fa_diag.h).

Argument marshalling only: torch tensors supply device memory and the current
CUDA stream; every step of the computation runs in the library's kernels.
There is no fallback: if the shared library is missing, every call raises.
"""

import ctypes
import functools
import os

import torch

from . import build as _build

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_WORKSPACE = range(6)
STATUS_NAMES = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_CUDA",
                4: "FA_ERR_TIMEOUT", 5: "FA_ERR_WORKSPACE"}


class FAError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s" % (where, STATUS_NAMES.get(status, status)))


class FwdTuning(ctypes.Structure):
    _fields_ = [("rescale_threshold", ctypes.c_float), ("emu_per_16", ctypes.c_int), ("split_p", ctypes.c_int),
                ("kv_stages", ctypes.c_int), ("head_group", ctypes.c_int)]


class BwdTuning(ctypes.Structure):
    _fields_ = [("paired", ctypes.c_int), ("schedule", ctypes.c_int), ("head_group", ctypes.c_int),
                ("reverse_blocks", ctypes.c_int), ("scores_first", ctypes.c_int), ("split_dq", ctypes.c_int)]


_LIB = None
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

_SIGNATURES = {
    "fa_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp]),
    "fa_fwd_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp,
                       ctypes.POINTER(FwdTuning), _vp]),
    "fa_fwd_default_tuning": (FwdTuning, []),
    "fa_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_int), _i, _i]),
    "fa_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i,
                    _vp, _sz, _vp]),
    "fa_bwd_default_tuning": (BwdTuning, []),
    "fa_bwd_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _i,
                       _vp, _sz, ctypes.POINTER(BwdTuning), _vp]),
    "fa_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp,
                            _i, _vp]),
    "fa_get_device_error": (_i, [_vp]),
    "fa_status_string": (ctypes.c_char_p, [_i]),
    "fa_rope": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, ctypes.POINTER(ctypes.c_int), ctypes.c_double, _i,
                     _i, _i, _vp]),
    "fa_cache_write": (_i, [_vp] * 6 + [_i] * 7 + [_vp] * 4),
    "fa_cache_read": (_i, [_vp] * 6 + [_i] * 7 + [_vp] * 3),
    "fa_fwd_paged_workspace_size": (_sz, [_i] * 7),
    "fa_fwd_paged": (_i, [_vp] * 7 + [_i] * 9 + [_f] + [_vp] * 3 + [_i, _vp, _sz, _vp]),
    "fa_diag_exp2": (_i, [_vp, _vp, _vp, ctypes.c_longlong, _vp]),
    "fa_diag_wait_timeout": (_i, [ctypes.c_ulonglong, _vp]),
    "fa_diag_fwd_paged": (_i, [_vp] * 7 + [_i] * 9 + [_f] + [_vp] * 3 + [_i, _vp, _sz, ctypes.c_ulonglong, _vp]),
}


def lib_path():
    return _build.LIB


def load_library(build_if_missing=False):
    """Loads the in-tree shared library; raises if absent.  With
    build_if_missing, (re)builds it first when it is absent or older than a
    source file."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        if not build_if_missing:
            raise RuntimeError("CUDA library %s is not built; run exact_attention_78_gb300.build.build()"
                               % _build.LIB)
        _build.build()
    lib = ctypes.CDLL(_build.LIB)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def _check(status, where):
    if status != FA_OK:
        raise FAError(status, where)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check_bf16(name, t):
    if not t.is_cuda or t.dtype is not torch.bfloat16 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA bfloat16 tensor" % name)


def _check_out(name, t, shape, dtype, device):
    """A caller-supplied output buffer: the library writes shape x dtype
    elements at its address, so anything else is refused here."""
    if (not t.is_cuda or t.device != device or t.dtype != dtype or not t.is_contiguous()
            or tuple(t.shape) != tuple(shape)):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (name, dtype, tuple(shape), device))


def _check_same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError("%s is on %s, q on %s" % (name, t.device, device))


def _dims(q, k, cu_seqlens):
    """(B, Hq, Hkv, Sq, Sk, D) as the C ABI wants them."""
    if cu_seqlens is None:
        if q.dim() != 4 or k.dim() != 4:
            raise ValueError("dense q/k/v are [B, S, H, D]")
        B, Sq, Hq, D = q.shape
        Sk, Hkv = k.shape[1], k.shape[2]
    else:
        if q.dim() != 3 or k.dim() != 3:
            raise ValueError("packed q/k/v are [total, H, D]")
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous CUDA int32 tensor")
        B = cu_seqlens.numel() - 1
        Sq, Hq, D = q.shape
        Sk, Hkv = k.shape[0], k.shape[1]
    return B, Hq, Hkv, Sq, Sk, D


def fwd(q, k, v, causal=False, scale=None, cu_seqlens=None, out=None, lse=None, rescale_threshold=None,
        emu_per_16=None, split_p=None, kv_stages=None, head_group=None, stream=None):
    """O, LSE = attention(q, k, v).  Dense [B,S,H,D] or packed [total,H,D].
    rescale_threshold, emu_per_16, split_p, kv_stages and head_group override
    the library's per-configuration choices (fa_fwd_tuning)."""
    lib = load_library()
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16(n, t)
    _check_same_device(q.device, k=k, v=v, cu_seqlens=cu_seqlens)
    B, Hq, Hkv, Sq, Sk, D = _dims(q, k, cu_seqlens)
    if scale is None:
        scale = D ** -0.5
    lse_shape = (Hq, Sq) if cu_seqlens is not None else (B, Hq, Sq)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out("out", out, q.shape, torch.bfloat16, q.device)
    if lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    else:
        _check_out("lse", lse, lse_shape, torch.float32, q.device)
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Sk, D, int(bool(causal)),
            float(scale), _ptr(cu_seqlens)]
    with torch.cuda.device(q.device):   # the library launches on the current device
        knobs = {"emu_per_16": emu_per_16, "split_p": split_p, "kv_stages": kv_stages, "head_group": head_group}
        if rescale_threshold is None and all(x is None for x in knobs.values()):
            st = lib.fa_fwd(*args, _stream(stream))
        else:
            t = lib.fa_fwd_default_tuning()
            if rescale_threshold is not None:
                t.rescale_threshold = float(rescale_threshold)
            for name, val in knobs.items():
                if val is not None:
                    setattr(t, name, int(val))
            st = lib.fa_fwd_ex(*args, ctypes.byref(t), _stream(stream))
    _check(st, "fa_fwd")
    return out, lse


def bwd_workspace_size(B, Hq, Hkv, Sq, Sk, D, deterministic=False, total_q=0, cu_seqlens_host=None):
    """Workspace bytes of fa_bwd.  Packed layout: total_q = packed row count
    (= Sq = Sk); cu_seqlens_host, if given, is a host sequence of B + 1 offsets."""
    offs = None
    if cu_seqlens_host is not None:
        vals = [int(x) for x in cu_seqlens_host]
        offs = (ctypes.c_int * len(vals))(*vals)
    return int(load_library().fa_bwd_workspace_size(B, Hq, Hkv, Sq, Sk, D, offs, int(total_q),
                                                    int(bool(deterministic))))


def bwd(q, k, v, o, lse, do, causal=False, scale=None, deterministic=False, workspace=None, dq=None, dk=None,
        dv=None, paired=None, cu_seqlens=None, stream=None, tuning=None):
    """dQ, dK, dV of attention(q, k, v) given O, LSE and dO.  Dense [B,S,H,D]
    or packed [total,H,D] with cu_seqlens (LSE [Hq, total]).  paired=True runs
    the main kernel on CTA pairs (paired tcgen05 MMAs; dense only).  tuning:
    a dict of fa_bwd_tuning fields (schedule, head_group, reverse_blocks,
    scores_first, split_dq) overriding the per-call defaults."""
    unknown = set(tuning or {}) - {f[0] for f in BwdTuning._fields_}
    if unknown:
        raise KeyError("unknown backward tuning field(s): %s" % ", ".join(sorted(unknown)))
    lib = load_library()
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _check_bf16(n, t)
    _check_same_device(q.device, k=k, v=v, o=o, lse=lse, do=do, cu_seqlens=cu_seqlens)
    B, Hq, Hkv, Sq, Sk, D = _dims(q, k, cu_seqlens)
    if tuple(o.shape) != tuple(q.shape) or tuple(do.shape) != tuple(q.shape):
        raise ValueError("o and do must have q's shape %s" % (tuple(q.shape),))
    if tuple(v.shape) != tuple(k.shape):
        raise ValueError("v must have k's shape %s" % (tuple(k.shape),))
    lse_shape = (Hq, Sq) if cu_seqlens is not None else (B, Hq, Sq)
    if not lse.is_cuda or lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != lse_shape:
        raise ValueError("lse must be a contiguous CUDA float32 tensor of shape %s" % (lse_shape,))
    if scale is None:
        scale = D ** -0.5
    need = bwd_workspace_size(B, Hq, Hkv, Sq, Sk, D, deterministic, total_q=Sq if cu_seqlens is not None else 0)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    elif not workspace.is_cuda or workspace.device != q.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % q.device)
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _check_out(name, t, like.shape, torch.bfloat16, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq,
            Sk, D, int(bool(causal)), float(scale), _ptr(cu_seqlens), int(bool(deterministic)), _ptr(workspace),
            workspace.numel() * workspace.element_size()]
    with torch.cuda.device(q.device):   # the library launches on the current device
        if paired is None and not tuning:
            st = lib.fa_bwd(*args, _stream(stream))
        else:
            t = lib.fa_bwd_default_tuning()
            if paired is not None:
                t.paired = int(bool(paired))
            for name, val in (tuning or {}).items():
                setattr(t, name, int(val))
            st = lib.fa_bwd_ex(*args, ctypes.byref(t), _stream(stream))
    _check(st, "fa_bwd")
    return dq, dk, dv


def _torch_forms(c):
    """(current stream of a device, allocation and release on the current device
    in a stream's order), as numbers: torch's own short forms where this release
    has them in `c`, which save a small call 3 us on the host (1.9 the stream, 1 the
    allocation), else the public ones."""
    return (getattr(c, "_cuda_getCurrentRawStream", None)
            or (lambda device: torch.cuda.current_stream(device).cuda_stream),
            getattr(c, "_cuda_cudaCachingAllocator_raw_alloc", None)
            or (lambda size, stream: torch.cuda.caching_allocator_alloc(size, stream=stream)),
            getattr(c, "_cuda_cudaCachingAllocator_raw_delete", None) or torch.cuda.caching_allocator_delete)


_current_stream, _alloc, _free = _torch_forms(torch._C)


class _Here:
    """The current stream of the current device, as a context like _OnStream."""

    def __init__(self, raw):
        self.raw = raw

    def __enter__(self):
        return self.raw

    def __exit__(self, *exc):
        return False


class _OnStream:
    """`stream` (or `device`'s current one) as the current stream for a call's
    launches and for what it allocates: outputs and workspace come from that
    stream's pool, so the allocator reuses them in its order."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
        self.ctx = torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device)

    def __enter__(self):
        self.ctx.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        return self.ctx.__exit__(*exc)


def _on(device, stream):
    # a small call takes a few microseconds on the GPU; entering a context
    # costs as much again on the host, and mostly changes nothing
    if stream is None and device.index == torch.cuda.current_device():
        return _Here(_current_stream(device.index))
    return _OnStream(device, stream)


def _adr(t):
    return None if t is None else t.data_ptr()


# A small call spends a few microseconds on the GPU, and as many on the host for
# every twenty or so attributes that are looked at.  So the checks below test
# everything in one expression and say what was wrong only when it is.

def _bad(name, what, device=None):
    raise ValueError("%s must be %s%s" % (name, what, "" if device is None else " on %s" % device))


def _check_int32(name, t, device, dims):
    if not (t.dtype is torch.int32 and t.is_cuda and t.device == device and t.is_contiguous() and t.dim() == dims):
        _bad(name, "a contiguous CUDA int32 tensor with %d dimension(s)" % dims, device)


def _cache_args(heads, D, device, k_pages, v_pages, k_scale, v_scale, block_table):
    """Checks the tensors of a cache; (num_pages, Hkv, page_size, max_pages)."""
    dtype = torch.bfloat16 if k_scale is None and v_scale is None else torch.float8_e4m3fn
    shape = k_pages.shape
    if not (k_pages.dtype is dtype and v_pages.dtype is dtype and k_pages.is_cuda and k_pages.device == device
            and v_pages.device == device and len(shape) == 4 and v_pages.shape == shape and k_pages.is_contiguous()
            and v_pages.is_contiguous()):
        _bad("k_pages and v_pages", "contiguous CUDA %s tensors of one shape [num_pages, Hkv, page_size, D]" % dtype,
             device)
    num_pages, Hkv, page_size, Dp = shape
    if Dp != D:
        raise ValueError("the pages' head dimension is %d, not %d" % (Dp, D))
    if heads is not None and heads != Hkv:
        raise ValueError("the pages have %d heads, k and v %d" % (Hkv, heads))
    if dtype is not torch.bfloat16:
        want = shape[:3]
        if not (k_scale is not None and v_scale is not None and k_scale.dtype is torch.uint8
                and v_scale.dtype is torch.uint8 and k_scale.device == device and v_scale.device == device
                and k_scale.shape == want and v_scale.shape == want and k_scale.is_contiguous()
                and v_scale.is_contiguous()):
            _bad("k_scale and v_scale", "contiguous CUDA uint8 tensors of shape %s" % (tuple(want),), device)
    _check_int32("block_table", block_table, device, 2)
    return num_pages, Hkv, page_size, block_table.shape[1]


def _new_tokens(name, x, B, cu_seqlens):
    """Sn of the C ABI for new tokens x, dense [B, Sn, H, D] or packed [Sn, H, D]."""
    _check_bf16(name, x)
    shape = x.shape
    if len(shape) != (4 if cu_seqlens is None else 3):
        raise ValueError("%s is [B, Sn, H, D], or [total, H, D] with cu_seqlens" % name)
    if cu_seqlens is None:
        if shape[0] != B:
            raise ValueError("%s has %d sequences, the block table %d" % (name, shape[0], B))
        return shape[1]
    _check_offsets(cu_seqlens, x.device, B)
    return shape[0]


def _check_offsets(cu_seqlens, device, B):
    _check_int32("cu_seqlens", cu_seqlens, device, 1)
    if cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens has %d offsets for %d sequences" % (cu_seqlens.numel(), B))


def _check_seq_lens(seq_lens, device, B):
    _check_int32("seq_lens", seq_lens, device, 1)
    if seq_lens.numel() != B:
        raise ValueError("seq_lens has %d lengths for %d sequences" % (seq_lens.numel(), B))


@functools.lru_cache(maxsize=256)
def _c_ints(values):
    """A C array of ints; the library reads it before its call returns."""
    return (ctypes.c_int * len(values))(*values)


def rope(q, k, positions, sections=None, base=10000.0, restart=False, interleaved=False, inverse=False, q_out=None,
         k_out=None, stream=None):
    """q and k ([..., H, D], the same leading shape; k may be None) turned by
    rotary positions.  positions: int32 [axes, ...] with that leading shape
    (or without the first dimension for one axis).  sections: rotary pairs of
    each axis (one axis: all D / 2 by default).  Frequencies base^(-i / pairs),
    starting anew on each axis with restart=True.  Pairs are elements i and
    i + pairs, or neighbours with interleaved=True.  inverse=True turns
    backwards: the gradients of a call without it.  q_out and k_out may be q
    and k.  Returns (q_out, k_out)."""
    lib = load_library()
    _check_bf16("q", q)
    shape, device = q.shape, q.device
    if len(shape) < 2:
        raise ValueError("q is [..., H, D]")
    lead, Hq, D = shape[:-2], shape[-2], shape[-1]
    Hkv = 0
    if k is not None:
        _check_bf16("k", k)
        if k.device != device or k.shape[:-2] != lead or k.shape[-1] != D:
            raise ValueError("k is [..., H, D] with q's leading shape, D and device")
        Hkv = k.shape[-2]
    elif k_out is not None:
        raise ValueError("k_out without k")
    if not (positions.dtype is torch.int32 and positions.device == device and positions.is_contiguous()):
        _bad("positions", "a contiguous CUDA int32 tensor", device)
    axes = 1
    if positions.shape != lead:
        if positions.shape[1:] != lead or positions.dim() == 0:
            raise ValueError("positions are %s, with a first dimension for the axes" % (tuple(lead),))
        axes = positions.shape[0]
    if sections is None:
        if axes != 1:
            raise ValueError("%d axes need sections" % axes)
        sections = (D // 2,)
    if len(sections) != axes:
        raise ValueError("%d sections for %d axes" % (len(sections), axes))
    if min(sections) < 1 or sum(sections) > D // 2:      # (the C interface's ints would wrap)
        raise ValueError("sections %s of at most %d pairs" % (tuple(sections), D // 2))
    tokens = lead.numel()
    if tokens >= 2 ** 31:
        raise ValueError("%d tokens in one call" % tokens)
    if q_out is not None:
        _check_out("q_out", q_out, shape, torch.bfloat16, device)
    if k_out is not None:
        _check_out("k_out", k_out, k.shape, torch.bfloat16, device)
    with _on(device, stream) as s:
        if q_out is None:
            q_out = torch.empty_like(q)
        if k is not None and k_out is None:
            k_out = torch.empty_like(k)
        st = lib.fa_rope(q.data_ptr(), _adr(k), q_out.data_ptr(), _adr(k_out), tokens, Hq, Hkv, D,
                         positions.data_ptr(), axes, _c_ints(tuple(sections)), base, bool(restart),
                         bool(interleaved), bool(inverse), s)
    if st:
        raise FAError(st, "fa_rope")
    return q_out, k_out


def cache_write(k, v, k_pages, v_pages, block_table, seq_lens, cu_seqlens=None, k_scale=None, v_scale=None,
                stream=None):
    """Writes new keys and values, dense [B, n, Hkv, D] or packed
    [total, Hkv, D] with cu_seqlens, into the pages [num_pages, Hkv, page_size,
    D]: the last tokens of sequences that are seq_lens long with them.  BF16
    pages; or float8_e4m3fn pages with uint8 scales [num_pages, Hkv,
    page_size], quantised on the way."""
    lib = load_library()
    B, device, shape = block_table.shape[0], k.device, k.shape
    Sn = _new_tokens("k", k, B, cu_seqlens)
    _check_bf16("v", v)
    if v.shape != shape or v.device != device:
        raise ValueError("v must have k's shape %s and device" % (tuple(shape),))
    num_pages, Hkv, page_size, max_pages = _cache_args(shape[-2], shape[-1], device, k_pages, v_pages, k_scale,
                                                       v_scale, block_table)
    _check_seq_lens(seq_lens, device, B)
    with _on(device, stream) as s:
        st = lib.fa_cache_write(k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _adr(k_scale),
                                _adr(v_scale), B, Hkv, Sn, shape[-1], num_pages, page_size, max_pages,
                                block_table.data_ptr(), seq_lens.data_ptr(), _adr(cu_seqlens), s)
    if st:
        raise FAError(st, "fa_cache_write")


def cache_read(k_pages, v_pages, block_table, cu_seqlens, total, k_scale=None, v_scale=None, k_out=None, v_out=None,
               stream=None):
    """The first cu_seqlens[b + 1] - cu_seqlens[b] tokens of every sequence as
    packed BF16 (k, v), each [total, Hkv, D]; rows from cu_seqlens[B] on are
    left as they were."""
    lib = load_library()
    if k_pages.dim() != 4:
        raise ValueError("k_pages is [num_pages, Hkv, page_size, D]")
    device, D, B = k_pages.device, k_pages.shape[3], block_table.shape[0]
    num_pages, Hkv, page_size, max_pages = _cache_args(None, D, device, k_pages, v_pages, k_scale, v_scale,
                                                       block_table)
    _check_offsets(cu_seqlens, device, B)
    shape = (total, Hkv, D)
    if k_out is not None:
        _check_out("k_out", k_out, shape, torch.bfloat16, device)
    if v_out is not None:
        _check_out("v_out", v_out, shape, torch.bfloat16, device)
    with _on(device, stream) as s:
        if k_out is None:
            k_out = torch.empty(shape, dtype=torch.bfloat16, device=device)
        if v_out is None:
            v_out = torch.empty(shape, dtype=torch.bfloat16, device=device)
        st = lib.fa_cache_read(k_pages.data_ptr(), v_pages.data_ptr(), _adr(k_scale), _adr(v_scale), k_out.data_ptr(),
                               v_out.data_ptr(), B, Hkv, total, D, num_pages, page_size, max_pages,
                               block_table.data_ptr(), cu_seqlens.data_ptr(), s)
    if st:
        raise FAError(st, "fa_cache_read")
    return k_out, v_out


@functools.lru_cache(maxsize=1024)
def fwd_paged_workspace_size(B, Hq, Hkv, Sn, D, packed=False, max_q=None):
    """Workspace bytes of fa_fwd_paged; max_q (packed) as in fwd_paged."""
    return int(load_library().fa_fwd_paged_workspace_size(B, Hq, Hkv, Sn, D, int(bool(packed)),
                                                          int(Sn if max_q is None else max_q)))


def fwd_paged(q, k_pages, v_pages, block_table, seq_lens, causal=True, scale=None, cu_seqlens=None, max_q=None,
              k_scale=None, v_scale=None, out=None, lse=None, workspace=None, stream=None):
    """O, LSE = attention of new tokens q, dense [B, n, Hq, D] or packed
    [total, Hq, D] with cu_seqlens, over the seq_lens[b] keys that each
    sequence has in the cache, the new tokens' own (written before by
    cache_write) as the last.  max_q: an upper bound of the new tokens of any
    one sequence (packed).  It chooses the kernel and the workspace, and the
    lengths themselves are on the device: a packed decoding step should give it
    (max_q=1).  Its default, `total`, is right for every call, but takes single
    tokens to the kernel of chunks, with 43 MB of workspace at D = 128 instead
    of 2.7 (64 tokens over 4096 keys each, 32/8 heads: BF16 192 us instead of
    163, E4M3 222 instead of 92)."""
    lib = load_library()
    B, device = block_table.shape[0], q.device
    Sn = _new_tokens("q", q, B, cu_seqlens)
    Hq, D = q.shape[-2:]
    num_pages, Hkv, page_size, max_pages = _cache_args(None, D, device, k_pages, v_pages, k_scale, v_scale,
                                                       block_table)
    _check_seq_lens(seq_lens, device, B)
    if cu_seqlens is None:
        max_q, lse_shape = Sn, (B, Hq, Sn)
    else:
        max_q, lse_shape = Sn if max_q is None else max_q, (Hq, Sn)
        if not 0 < max_q <= Sn:      # (the C interface's ints would wrap)
            raise ValueError("max_q is %d for %d rows" % (max_q, Sn))
    if out is not None:
        _check_out("out", out, q.shape, torch.bfloat16, device)
    if lse is not None:
        _check_out("lse", lse, lse_shape, torch.float32, device)
    if workspace is not None and (workspace.device != device or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    with _on(device, stream) as s:
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = torch.empty(lse_shape, dtype=torch.float32, device=device)
        if workspace is None:
            # from torch's allocator and back to it in the stream's order, as a
            # tensor would be, whose making takes 2 us more
            size = max(fwd_paged_workspace_size(B, Hq, Hkv, Sn, D, cu_seqlens is not None, max_q), 256)
            ws = _alloc(size, s)
        else:
            size, ws = workspace.numel() * workspace.element_size(), workspace.data_ptr()
        try:
            st = lib.fa_fwd_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _adr(k_scale), _adr(v_scale),
                                  out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Sn, D, num_pages, page_size, max_pages,
                                  bool(causal), D ** -0.5 if scale is None else scale, block_table.data_ptr(),
                                  seq_lens.data_ptr(), _adr(cu_seqlens), max_q, ws, size, s)
        finally:
            if workspace is None:
                _free(ws)
    if st:
        raise FAError(st, "fa_fwd_paged")
    return out, lse


def get_device_error(stream=None):
    """Synchronises and returns (and clears) the library's device error status."""
    return int(load_library().fa_get_device_error(_stream(stream)))


def status_string(status):
    return load_library().fa_status_string(int(status)).decode()


def exp2_probe(x, stream=None):
    """(2^x by the FMA polynomial, 2^x by the hardware unit) for a CUDA float32 tensor."""
    lib = load_library()
    if not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA float32 tensor")
    ye, yh = torch.empty_like(x), torch.empty_like(x)
    _check(lib.fa_diag_exp2(_ptr(x), _ptr(ye), _ptr(yh), x.numel(), _stream(stream)), "fa_diag_exp2")
    return ye, yh


def wait_timeout_probe(limit_ns, stream=None):
    _check(load_library().fa_diag_wait_timeout(int(limit_ns), _stream(stream)), "fa_diag_wait_timeout")
