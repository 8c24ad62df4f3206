"""Python binding of libflamia (block-scaled causal attention for training on GB300).

Argument marshalling only: every step runs in the library's CUDA kernels, called
through its C ABI (include/flamia.h) with the same names.  PyTorch provides the
device memory and streams.  There is no CPU path: without the compiled library
every call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libflamia.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE_TOO_SMALL, ERR_CUDA, ERR_TIMEOUT, ERR_BAD_SEQLENS = range(7)
ERR_NO_PAGES, ERR_BAD_PAGE = 7, 8
PATH_MXFP8, PATH_NVFP4_FP8 = 0, 1
F32, BF16, E4M3, E2M1 = 0, 1, 2, 3
ROLE_QKV, ROLE_DO = 0, 1

EXPORTED = ("flamia_workspace_size", "flamia_plan", "flamia_quantize", "flamia_fwd", "flamia_bwd",
            "flamia_get_device_status", "flamia_clear_device_status", "flamia_status_string",
            "flamia_debug_set_phat_dump", "flamia_debug_withhold_first_item", "flamia_debug_workspace_offset",
            "flamia_plan_noalloc", "flamia_debug_mma_idesc", "flamia_debug_smem_desc",
            "flamia_paged_workspace_size", "flamia_paged_plan", "flamia_paged_append", "flamia_paged_fwd",
            "flamia_paged_pages_workspace_size", "flamia_paged_plan_shared", "flamia_paged_copy", "flamia_paged_compact")
WS_FWD_ITEMS, WS_BWD_ITEMS, WS_DQ_PRESCALE = range(3)
MMA_F8F6F4, MMA_MXF8F6F4, MMA_MXF4NVF4 = range(3)
MMA_BF16, MMA_F16 = 4, 5
SWZ_NONE, SWZ_128B, SWZ_64B, SWZ_32B = 0, 2, 4, 6


class FlamiaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("n_seq", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p), ("causal", ctypes.c_int32),
                ("exact", ctypes.c_int32), ("causal_dq_scale", ctypes.c_int32), ("deterministic", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("path", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("dq_fp16", ctypes.c_int32), ("bitexp", ctypes.c_int32),
                ("hadamard", ctypes.c_int32), ("clc", ctypes.c_int32)]


class Operand(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("codes4", ctypes.c_void_p),
                ("scales4", ctypes.c_void_p), ("gscale4", ctypes.c_void_p)]


class Paged(ctypes.Structure):
    _fields_ = [("n_req", ctypes.c_int32), ("T", ctypes.c_int32), ("max_q", ctypes.c_int32), ("H", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("cache_dtype", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("kv_stride", ctypes.c_int64)]


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("k_blocks", ctypes.c_void_p),
                ("v_blocks", ctypes.c_void_p)]
    pool = None  # (Hkv, page_size, d, cache_dtype), n_pages of the tensors that paged_cache was given
    device = -1  # and where they are


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libflamia.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build()")
    L = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    P = ctypes.POINTER(Problem)
    O = ctypes.POINTER(Operand)
    L.flamia_workspace_size.restype, L.flamia_workspace_size.argtypes = sz, [P]
    L.flamia_plan.restype, L.flamia_plan.argtypes = i32, [P, vp, sz, vp]
    L.flamia_quantize.restype = i32
    L.flamia_quantize.argtypes = [P, i32, ctypes.POINTER(vp), vp, O, vp, vp, sz, vp]
    L.flamia_fwd.restype = i32
    L.flamia_fwd.argtypes = [P, O, O, O, vp, vp, vp, vp, sz, vp]
    L.flamia_bwd.restype = i32
    L.flamia_bwd.argtypes = [P, O, O, O, O, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flamia_get_device_status.restype, L.flamia_get_device_status.argtypes = i32, [vp, vp]
    L.flamia_clear_device_status.restype, L.flamia_clear_device_status.argtypes = i32, [vp, vp]
    L.flamia_status_string.restype, L.flamia_status_string.argtypes = ctypes.c_char_p, [i32]
    L.flamia_debug_set_phat_dump.restype = i32
    L.flamia_debug_set_phat_dump.argtypes = [vp, sz, vp, vp, vp]
    L.flamia_debug_workspace_offset.restype, L.flamia_debug_workspace_offset.argtypes = sz, [P, i32]
    L.flamia_debug_withhold_first_item.restype = i32
    L.flamia_debug_withhold_first_item.argtypes = [i32]
    L.flamia_debug_mma_idesc.restype = i32
    L.flamia_debug_mma_idesc.argtypes = [i32, ctypes.c_uint32, ctypes.c_uint32, i32, i32, i32, i32,
                                         ctypes.POINTER(ctypes.c_uint32)]
    L.flamia_debug_smem_desc.restype = i32
    L.flamia_debug_smem_desc.argtypes = [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32, i32,
                                         ctypes.POINTER(ctypes.c_uint64)]
    L.flamia_plan_noalloc.restype = i32
    L.flamia_plan_noalloc.argtypes = [P, vp, vp, vp, vp]
    G, K = ctypes.POINTER(Paged), ctypes.POINTER(Cache)
    L.flamia_paged_workspace_size.restype, L.flamia_paged_workspace_size.argtypes = sz, [G]
    L.flamia_paged_plan.restype, L.flamia_paged_plan.argtypes = i32, [G, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flamia_paged_append.restype, L.flamia_paged_append.argtypes = i32, [G, vp, vp, vp, K, vp, sz, vp]
    L.flamia_paged_fwd.restype, L.flamia_paged_fwd.argtypes = i32, [G, vp, K, vp, vp, vp, sz, vp]
    L.flamia_paged_pages_workspace_size.restype, L.flamia_paged_pages_workspace_size.argtypes = sz, [G]
    L.flamia_paged_plan_shared.restype = i32
    L.flamia_paged_plan_shared.argtypes = [G] + 9 * [vp] + [vp, sz, vp, sz, vp]
    L.flamia_paged_copy.restype, L.flamia_paged_copy.argtypes = i32, [G, i32, K, K, vp, i32, vp, vp, sz, vp]
    L.flamia_paged_compact.restype, L.flamia_paged_compact.argtypes = i32, [G] + 6 * [vp] + [vp, sz, vp]
    _lib = L
    return L


def status_string(s: int) -> str:
    return load_library().flamia_status_string(int(s)).decode()


def _check(s: int, what: str):
    if s != OK:
        raise FlamiaError(s, what)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def make_problem(T, H, Hkv, d, cu_seqlens, *, causal=True, exact=False, causal_dq_scale=False,
                 deterministic=False, softmax_scale=0.0, path=PATH_MXFP8, in_dtype=BF16, out_dtype=BF16,
                 dq_fp16=False, bitexp=False, hadamard=False, clc=False) -> Problem:
    """cu_seqlens: int32 device tensor [n_seq + 1] (kept referenced by the caller)."""
    return Problem(int(T), int(H), int(Hkv), int(d), int(cu_seqlens.numel() - 1), cu_seqlens.data_ptr(),
                   int(causal), int(exact), int(causal_dq_scale), int(deterministic), float(softmax_scale),
                   int(path), int(in_dtype), int(out_dtype), int(dq_fp16), int(bitexp),
                   int(hadamard), int(clc))


def operand(codes, scales, codes4=None, scales4=None, gscale4=None) -> Operand:
    return Operand(_ptr(codes), _ptr(scales), _ptr(codes4), _ptr(scales4), _ptr(gscale4))


def flamia_workspace_size(prob: Problem) -> int:
    return int(load_library().flamia_workspace_size(ctypes.byref(prob)))


def flamia_plan(prob: Problem, ws, stream=None):
    _check(load_library().flamia_plan(ctypes.byref(prob), _ptr(ws), ws.numel() * ws.element_size(),
                                      _stream(stream)), "flamia_plan")


def flamia_quantize(prob: Problem, role: int, inputs, O, outs, D, ws, stream=None):
    n = len(inputs)
    arr = (ctypes.c_void_p * n)(*[_ptr(t) for t in inputs])
    ops = (Operand * len(outs))(*outs)
    _check(load_library().flamia_quantize(ctypes.byref(prob), int(role), arr, _ptr(O), ops, _ptr(D), _ptr(ws),
                                          ws.numel() * ws.element_size(), _stream(stream)), "flamia_quantize")


def flamia_fwd(prob: Problem, q: Operand, k: Operand, v: Operand, O, m, l, ws, stream=None):
    _check(load_library().flamia_fwd(ctypes.byref(prob), ctypes.byref(q), ctypes.byref(k), ctypes.byref(v),
                                     _ptr(O), _ptr(m), _ptr(l), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream(stream)), "flamia_fwd")


def flamia_bwd(prob: Problem, q: Operand, k: Operand, v: Operand, dO: Operand, D, m, l, dQ, dK, dV, ws,
               stream=None):
    _check(load_library().flamia_bwd(ctypes.byref(prob), ctypes.byref(q), ctypes.byref(k), ctypes.byref(v),
                                     ctypes.byref(dO), _ptr(D), _ptr(m), _ptr(l), _ptr(dQ), _ptr(dK), _ptr(dV),
                                     _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "flamia_bwd")


def flamia_plan_noalloc(prob: Problem, fwd_items, bwd_items, n_items, stream=None):
    """Work lists without a workspace (library-held scratch; see include/flamia.h).
    fwd_items/bwd_items: int32 device tensors [ceil(T/128) + n_seq, 2]; n_items: int32 device [1]."""
    _check(load_library().flamia_plan_noalloc(ctypes.byref(prob), _ptr(fwd_items), _ptr(bwd_items), _ptr(n_items),
                                              _stream(stream)), "flamia_plan_noalloc")


def flamia_get_device_status(ws, stream=None) -> int:
    return int(load_library().flamia_get_device_status(_ptr(ws), _stream(stream)))


def flamia_debug_set_phat_dump(ws, codes, exps, stream=None):
    """Test hook: record P^ codes / block exponents of the next fwd/bwd calls (None, None: off)."""
    _check(load_library().flamia_debug_set_phat_dump(_ptr(ws), ws.numel() * ws.element_size(), _ptr(codes), _ptr(exps),
                                                     _stream(stream)), "flamia_debug_set_phat_dump")


def flamia_debug_workspace_offset(prob: Problem, region: int) -> int:
    """Byte offset of a workspace region (WS_FWD_ITEMS, WS_BWD_ITEMS, WS_DQ_PRESCALE)."""
    return int(load_library().flamia_debug_workspace_offset(ctypes.byref(prob), int(region)))


def flamia_debug_withhold_first_item(on: bool):
    """Test hook: the next attention launches withhold each CTA's first work
    item, and the page calls an arrival at their last barrier, so that their
    bounded waits run out (see include/flamia.h)."""
    _check(load_library().flamia_debug_withhold_first_item(int(bool(on))), "flamia_debug_withhold_first_item")


def flamia_debug_mma_idesc(kind: int, M: int, N: int, a_mn: int = 0, b_mn: int = 0, a_sf_id: int = 0,
                           b_sf_id: int = 0) -> int:
    """Test hook: the tcgen05.mma instruction descriptor the kernels encode
    for `kind` (MMA_F8F6F4, MMA_MXF8F6F4, MMA_MXF4NVF4) on an M x N tile."""
    out = ctypes.c_uint32()
    _check(load_library().flamia_debug_mma_idesc(int(kind), int(M), int(N), int(a_mn), int(b_mn), int(a_sf_id),
                                                 int(b_sf_id), ctypes.byref(out)), "flamia_debug_mma_idesc")
    return int(out.value)


def flamia_debug_smem_desc(saddr: int, lbo: int, sbo: int, swizzle: int) -> int:
    """Test hook: the shared-memory matrix descriptor the kernels encode."""
    out = ctypes.c_uint64()
    _check(load_library().flamia_debug_smem_desc(int(saddr), int(lbo), int(sbo), int(swizzle), ctypes.byref(out)),
           "flamia_debug_smem_desc")
    return int(out.value)


def flamia_clear_device_status(ws, stream=None):
    _check(load_library().flamia_clear_device_status(_ptr(ws), _stream(stream)), "flamia_clear_device_status")


def make_paged(T, H, Hkv, d, cu_q, kv_len, block_table, *, page_size, n_pages, max_q=0, cache_dtype=BF16,
               in_dtype=BF16, causal=True, softmax_scale=0.0, q_stride=0, kv_stride=0) -> Paged:
    """One serving step over a paged cache (see include/flamia.h).  cu_q [n_req + 1], kv_len [n_req] and
    block_table [n_req, max_pages]: contiguous int32 device tensors, kept referenced by the caller."""
    for t in (cu_q, kv_len, block_table):
        _int32(t)
    n_req = kv_len.numel()
    if cu_q.numel() != n_req + 1 or block_table.dim() != 2 or block_table.shape[0] != n_req:
        raise ValueError("cu_q must hold n_req + 1 offsets and block_table n_req rows")
    return Paged(n_req, int(T), int(max_q), int(H), int(Hkv), int(d), int(page_size), int(n_pages),
                 block_table.shape[1], int(cache_dtype), int(in_dtype), int(bool(causal)), float(softmax_scale),
                 cu_q.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(), int(q_stride), int(kv_stride))


def _int32(t, n=None):
    import torch
    if t.dtype != torch.int32 or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"expected a contiguous int32 tensor{'' if n is None else f' of {n}'}, got {tuple(t.shape)} "
                         f"{t.dtype}")


def paged_cache(k, v, k_scales=None, v_scales=None, k_blocks=None, v_blocks=None) -> Cache:
    """One layer's pool: k, v [n_pages, Hkv, page_size, d] (bf16, or uint8 E4M3 codes with uint8 scales
    [n_pages, Hkv, page_size]), or uint8 [n_pages, Hkv, page_size, d / 2] (two E2M1 codes a byte) with such scales and
    block scales [n_pages, Hkv, page_size, d / 16] (uint8 or float8_e4m3fn).  Pages may be strided (k = pool[:, 0],
    v = pool[:, 1]); a page is contiguous.  The calls refuse a pool of another type or page shape than the problem's, of
    fewer pages or on another device than the workspace's."""
    import torch
    if k.shape != v.shape or k.stride() != v.stride() or k.dim() != 4 or k.dtype != v.dtype:
        raise ValueError("k and v must be [n_pages, Hkv, page_size, d] of one type and layout")
    if k[0].is_contiguous() is False:
        raise ValueError("the pages of k and v must be contiguous")
    if k.shape[0] > 1 and k.stride(0) < k[0].numel():
        raise ValueError("the pages of k (and of v) must not share memory")
    for s in (k_scales, v_scales):
        if s is not None and (s.shape != k.shape[:3] or s.element_size() != 1 or not s.is_contiguous()):
            raise ValueError("scales must be contiguous bytes [n_pages, Hkv, page_size]")
    e2m1 = k_blocks is not None or v_blocks is not None
    if e2m1:
        for s in (k_blocks, v_blocks):
            if (s is None or s.shape[:3] != k.shape[:3] or s.dim() != 4 or 8 * s.shape[3] != k.shape[3] or
                    s.element_size() != 1 or not s.is_contiguous()):
                raise ValueError("block scales must be contiguous bytes [n_pages, Hkv, page_size, d / 16]")
        if k.dtype != torch.uint8 or k_scales is None or v_scales is None:
            raise ValueError("block scales go with uint8 codes and their scales")
    if any(t is not None and t.device != k.device for t in (v, k_scales, v_scales, k_blocks, v_blocks)):
        raise ValueError("a pool's tensors must be on one device")
    stride = k.stride(0) if k.shape[0] > 1 else 0
    cache = Cache(_ptr(k), _ptr(v), _ptr(k_scales), _ptr(v_scales), 2 * stride if e2m1 else stride, _ptr(k_blocks),
                  _ptr(v_blocks))
    dtype = E2M1 if e2m1 else {torch.bfloat16: BF16, torch.uint8: E4M3, torch.float8_e4m3fn: E4M3}.get(k.dtype)
    cache.device = k.get_device()
    cache.pool = (*k.shape[1:3], k.shape[3] * (2 if e2m1 else 1), dtype), k.shape[0]
    return cache


def flamia_paged_workspace_size(prob: Paged) -> int:
    return int(load_library().flamia_paged_workspace_size(ctypes.byref(prob)))


def _paged_call(name, ws, stream, *args):
    """One launch on the device of `ws`, on `stream` or that device's current stream.  These calls are short: their
    host time is what a small serving step costs."""
    import torch
    dev = ws.get_device()
    if dev < 0:
        raise FlamiaError(ERR_INVALID_ARG, name)
    s = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream.cuda_stream
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            st = getattr(_lib or load_library(), name)(*args, ws.data_ptr(), ws.nbytes, s)
    else:
        st = getattr(_lib or load_library(), name)(*args, ws.data_ptr(), ws.nbytes, s)
    if st:
        raise FlamiaError(st, name)


def flamia_paged_plan(prob: Paged, ws, slot_map=None, old_len=None, free_pages=None, n_free=None, n_free_out=None,
                      stream=None):
    """Once per step: block table, free stack, slot map and the attention's work split."""
    _paged_call("flamia_paged_plan", ws, stream, prob, _ptr(slot_map), _ptr(old_len), _ptr(free_pages), _ptr(n_free),
                _ptr(n_free_out))


def flamia_paged_pages_workspace_size(prob: Paged) -> int:
    """Bytes of the second workspace that the calls on shared pages take (see include/flamia.h)."""
    return int(load_library().flamia_paged_pages_workspace_size(ctypes.byref(prob)))


def _words(where, device, *pairs):
    """int32 tensors of at least so many words in a row on the device (None passes)."""
    import torch
    for t, n in pairs:
        if t is not None and (t.dtype is not torch.int32 or t.numel() < n or not t.is_contiguous() or t.get_device() != device):
            raise FlamiaError(ERR_INVALID_ARG, where)


def flamia_paged_plan_shared(prob: Paged, ws, pages_ws, slot_map, src, old_len, refs, free_pages, n_free, n_free_out, copies,
                             n_copies, stream=None):
    """Once per step of requests that share pages: forks (src), counts, copies on write, then as flamia_paged_plan.
    copies [n_req, 2] and n_copies list the pages that flamia_paged_copy must copy before anything is appended."""
    _words("flamia_paged_plan_shared", ws.get_device(), (slot_map, prob.T), (src, prob.n_req), (old_len, prob.n_req), (refs, prob.n_pages),
           (free_pages, prob.n_pages), (n_free, 1), (n_free_out, 1), (copies, 2 * prob.n_req), (n_copies, 1))
    if pages_ws.get_device() != ws.get_device():
        raise FlamiaError(ERR_INVALID_ARG, "flamia_paged_plan_shared")
    _paged_call("flamia_paged_plan_shared", ws, stream, prob, _ptr(slot_map), _ptr(src), _ptr(old_len), _ptr(refs),
                _ptr(free_pages), _ptr(n_free), _ptr(n_free_out), _ptr(copies), _ptr(n_copies), pages_ws.data_ptr(),
                pages_ws.nbytes)


def flamia_paged_copy(prob: Paged, src, dst, copies, n_copies, pages_ws, stream=None):
    """Pages copied in every layer: src and dst are lists of caches (paged_cache), which may be the same list."""
    n = len(src)
    if n == 0 or len(dst) != n:
        raise FlamiaError(ERR_INVALID_ARG, "flamia_paged_copy")
    page, n_pages, device = (prob.Hkv, prob.page_size, prob.d, prob.cache_dtype), prob.n_pages, pages_ws.get_device()
    for cache in src if dst is src else (*src, *dst):
        pool = cache.pool
        if pool is not None and (pool[0] != page or pool[1] < n_pages or cache.device != device):
            raise FlamiaError(ERR_INVALID_ARG, "flamia_paged_copy")
    _words("flamia_paged_copy", device, (copies, 0), (n_copies, 1))
    a = (Cache * n).from_buffer_copy(b"".join(src))  # (Cache * n)(*src) takes three times as long
    b = a if dst is src else (Cache * n).from_buffer_copy(b"".join(dst))
    _paged_call("flamia_paged_copy", pages_ws, stream, prob, n, a, b, copies.data_ptr(), copies.numel() // 2,
                n_copies.data_ptr())


def flamia_paged_compact(prob: Paged, pages_ws, length, refs, free_pages, n_free, copies, n_copies, stream=None):
    """The pages in use to the low end of the pool: tables, counts (refs may be None) and stack rewritten, the moves
    listed in copies [n_pages, 2] and n_copies for flamia_paged_copy."""
    _words("flamia_paged_compact", pages_ws.get_device(), (length, prob.n_req), (refs, prob.n_pages), (free_pages, prob.n_pages), (n_free, 1),
           (copies, 2 * prob.n_pages), (n_copies, 1))
    _paged_call("flamia_paged_compact", pages_ws, stream, prob, _ptr(length), _ptr(refs), _ptr(free_pages), _ptr(n_free),
                _ptr(copies), _ptr(n_copies))


def _check_pool(prob, cache, where, ws):
    if cache.pool is not None:
        page, n_pages = cache.pool
        if (page != (prob.Hkv, prob.page_size, prob.d, prob.cache_dtype) or n_pages < prob.n_pages or
                cache.device != ws.get_device()):
            raise FlamiaError(ERR_INVALID_ARG, where)


def flamia_paged_append(prob: Paged, k, v, slot_map, cache: Cache, ws, stream=None):
    """The step's K and V rows into their slots of one layer's cache."""
    _check_pool(prob, cache, "flamia_paged_append", ws)
    _paged_call("flamia_paged_append", ws, stream, prob, k.data_ptr(), v.data_ptr(), slot_map.data_ptr(), cache)


def flamia_paged_fwd(prob: Paged, q, cache: Cache, O, lse, ws, stream=None):
    """Attention of the step's queries over one layer's cache (lse may be None)."""
    _check_pool(prob, cache, "flamia_paged_fwd", ws)
    _paged_call("flamia_paged_fwd", ws, stream, prob, q.data_ptr(), cache, O.data_ptr(), _ptr(lse))


@dataclass
class TrainCall:
    """Device buffers for one training call of a fixed problem, and the call itself.

    Holds the quantized payloads, O, (m, l), D and the gradients.  ``run()``
    issues plan -> quantize(QKV) -> fwd -> quantize(dO) -> bwd on the current
    stream (no host synchronisation)."""

    T: int
    H: int
    Hkv: int
    d: int
    cu_seqlens: object  # int32 device tensor
    causal: bool = True
    exact: bool = False
    deterministic: bool = False
    causal_dq_scale: bool = False
    dq_fp16: bool = True  # FP16 dQ partials with the power-of-two prescale (the pages' default)
    bitexp: bool = False  # inference forward only: backward() raises
    hadamard: bool = False  # Q and K rotated before quantization; gradients rotated back
    clc: bool = False  # work items taken over by cluster launch control (a CTA per item)
    path: int = PATH_MXFP8
    in_dtype: int = BF16
    out_dtype: int = BF16
    softmax_scale: float = 0.0

    def __post_init__(self):
        import torch
        dev = self.cu_seqlens.device
        self.prob = make_problem(self.T, self.H, self.Hkv, self.d, self.cu_seqlens, causal=self.causal,
                                 exact=self.exact, deterministic=self.deterministic,
                                 causal_dq_scale=self.causal_dq_scale, dq_fp16=self.dq_fp16, bitexp=self.bitexp,
                                 hadamard=self.hadamard, clc=self.clc,
                                 softmax_scale=self.softmax_scale, path=self.path, in_dtype=self.in_dtype,
                                 out_dtype=self.out_dtype)
        nbytes = flamia_workspace_size(self.prob)
        if nbytes == 0:
            raise FlamiaError(ERR_INVALID_ARG, "flamia_workspace_size")
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        u8 = dict(dtype=torch.uint8, device=dev)
        T, H, Hkv, d = self.T, self.H, self.Hkv, self.d
        odt = torch.bfloat16 if self.out_dtype == BF16 else torch.float32
        self.q_codes, self.k_codes, self.v_codes = (torch.empty(T, h, d, **u8) for h in (H, Hkv, Hkv))
        self.q_scales, self.k_scales, self.v_scales = (torch.empty(h, T, **u8) for h in (H, Hkv, Hkv))
        self.do_codes, self.do_scales = torch.empty(T, H, d, **u8), torch.empty(H, T, **u8)
        self.q4 = self.k4 = None
        if self.path == PATH_NVFP4_FP8:
            self.q4 = (torch.empty(T, H, d // 2, **u8), torch.empty(T, H, d // 16, **u8),
                       torch.empty(H, T, dtype=torch.float32, device=dev))
            self.k4 = (torch.empty(T, Hkv, d // 2, **u8), torch.empty(T, Hkv, d // 16, **u8),
                       torch.empty(Hkv, T, dtype=torch.float32, device=dev))
        self.O = torch.empty(T, H, d, dtype=odt, device=dev)
        self.m = torch.empty(H, T, dtype=torch.int32, device=dev)
        self.l = torch.empty(H, T, dtype=torch.float32, device=dev)
        self.D = torch.empty(H, T, dtype=torch.float32, device=dev)
        self.dQ = torch.empty(T, H, d, dtype=odt, device=dev)
        self.dK = torch.empty(T, Hkv, d, dtype=odt, device=dev)
        self.dV = torch.empty(T, Hkv, d, dtype=odt, device=dev)
        q4, k4 = self.q4 or (None,) * 3, self.k4 or (None,) * 3
        self.opq = operand(self.q_codes, self.q_scales, *q4)
        self.opk = operand(self.k_codes, self.k_scales, *k4)
        self.opv = operand(self.v_codes, self.v_scales)
        self.opdo = operand(self.do_codes, self.do_scales)

    def plan(self, stream=None):
        flamia_plan(self.prob, self.ws, stream)

    def forward(self, q, k, v, stream=None):
        flamia_quantize(self.prob, ROLE_QKV, [q, k, v], None, [self.opq, self.opk, self.opv], None, self.ws, stream)
        flamia_fwd(self.prob, self.opq, self.opk, self.opv, self.O, self.m, self.l, self.ws, stream)

    def backward(self, do, stream=None):
        flamia_quantize(self.prob, ROLE_DO, [do], self.O, [self.opdo], self.D, self.ws, stream)
        flamia_bwd(self.prob, self.opq, self.opk, self.opv, self.opdo, self.D, self.m, self.l, self.dQ, self.dK,
                   self.dV, self.ws, stream)

    def run(self, q, k, v, do, stream=None):
        self.plan(stream)
        self.forward(q, k, v, stream)
        self.backward(do, stream)


@dataclass
class PagedCall:
    """Device buffers for serving up to ``n_req`` requests from paged caches of ``layers`` layers, and the calls.

    One step: ``plan(cu_q, kv_len)`` once, then per layer ``append(layer, k, v)`` and ``attend(layer, q)``; all on the
    current stream, no host synchronisation, so a step can be captured in a CUDA graph (cu_q and kv_len are then read
    from the tensors given at capture).  A request that ends passes kv_len 0; its pages serve others.  After a plan
    whose status is not OK (ERR_NO_PAGES, say) no page has moved: plan again with other lengths.

    With ``shared`` requests may hold the same pages: ``plan(cu_q, kv_len, src)`` says which request (as it was before
    the step) each one continues, -1 none; forks share pages, and one that is written to is copied first.  ``compact()``
    moves the pages in use to the low end of the pools.

    ``status`` (a word on the device) is the last plan's and its appends' and attentions', ``pages_status`` (``shared``
    only) that of the last plan's page management and copies or, after ``compact()``, of the compaction: read the latter
    before a pool is cut, a compaction that was refused has moved nothing."""

    n_req: int
    T: int           # new tokens of a step at most
    H: int
    Hkv: int
    d: int
    page_size: int
    n_pages: int
    max_pages: int   # pages of a request at most
    layers: int = 1
    max_q: int = 0   # new tokens of a request at most (0: T)
    cache_dtype: int = BF16
    in_dtype: int = BF16
    causal: bool = True
    softmax_scale: float = 0.0
    device: object = "cuda"
    shared: bool = False

    def __post_init__(self):
        import torch
        i32 = dict(dtype=torch.int32, device=self.device)
        self.cu_q = torch.zeros(self.n_req + 1, **i32)
        self.kv_len, self.held_len = torch.zeros(self.n_req, **i32), torch.zeros(self.n_req, **i32)
        self.block_table = torch.zeros(self.n_req, self.max_pages, **i32)
        self.free_pages = torch.arange(self.n_pages, **i32)
        self.n_free = torch.full((1,), self.n_pages, **i32)
        self.slot_map = torch.full((self.T,), -1, **i32)
        self.prob = make_paged(self.T, self.H, self.Hkv, self.d, self.cu_q, self.kv_len, self.block_table,
                               page_size=self.page_size, n_pages=self.n_pages, max_q=self.max_q,
                               cache_dtype=self.cache_dtype, in_dtype=self.in_dtype, causal=self.causal,
                               softmax_scale=self.softmax_scale)
        nbytes = flamia_paged_workspace_size(self.prob)
        if nbytes == 0:
            raise FlamiaError(ERR_INVALID_ARG, "flamia_paged_workspace_size")
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self.status = self.ws[:4].view(torch.int32)
        rows = (self.layers, self.n_pages, self.Hkv, self.page_size)
        codes, e2m1 = self.cache_dtype in (E4M3, E2M1), self.cache_dtype == E2M1

        def pair(shape, fill, dtype=torch.uint8):
            return [torch.full(shape, fill, dtype=dtype, device=self.device) for _ in range(2)]

        self.k, self.v = pair((*rows, self.d // 2 if e2m1 else self.d), 0, torch.uint8 if codes else torch.bfloat16)
        self.k_scales, self.v_scales = pair(rows, 127) if codes else (None, None)
        self.k_blocks, self.v_blocks = pair((*rows, self.d // 16), 0) if e2m1 else (None, None)
        pools = [x for x in (self.k, self.v, self.k_scales, self.v_scales, self.k_blocks, self.v_blocks) if x is not None]
        self.caches = [paged_cache(*layer) for layer in zip(*pools)]
        if self.shared:
            self.refs = torch.zeros(self.n_pages, **i32)
            self.same = torch.arange(self.n_req, **i32)
            self.src = self.same.clone()
            self.copies, self.n_copies = torch.zeros(max(self.n_req, self.n_pages), 2, **i32), torch.zeros(1, **i32)
            self.pages_ws = torch.zeros(flamia_paged_pages_workspace_size(self.prob), dtype=torch.uint8, device=self.device)
            self.pages_status = self.pages_ws[:4].view(torch.int32)
        self.O = torch.zeros(self.T, self.H, self.d, dtype=torch.bfloat16, device=self.device)
        self.lse = torch.zeros(self.H, self.T, dtype=torch.float32, device=self.device)
        self.kv_dtype = torch.bfloat16 if self.in_dtype == BF16 else torch.float32

    @staticmethod
    def _check(where, device, *tensors):
        for x, shape, dtype in tensors:
            if (tuple(x.shape) != tuple(shape) or x.dtype != dtype or not x.is_contiguous() or
                    device not in (None, x.device)):
                raise FlamiaError(ERR_INVALID_ARG, "PagedCall." + where)

    def plan(self, cu_q, kv_len, src=None):
        """cu_q [n_req + 1], kv_len [n_req]: int32 tensors; kv_len counts the step's new tokens too.  They are copied
        on the stream: pinned host tensors must keep their values until that has run.  src [n_req] int32 (``shared``
        only; None: each continues itself): see the class."""
        import torch
        self._check("plan", None, (cu_q, self.cu_q.shape, torch.int32), (kv_len, self.kv_len.shape, torch.int32),
                    *(() if src is None else ((src, self.kv_len.shape, torch.int32),)))
        if src is not None and not self.shared:
            raise FlamiaError(ERR_INVALID_ARG, "PagedCall.plan")
        self.cu_q.copy_(cu_q, non_blocking=True)
        self.kv_len.copy_(kv_len, non_blocking=True)
        if self.shared:
            self.src.copy_(self.same if src is None else src, non_blocking=True)
            flamia_paged_plan_shared(self.prob, self.ws, self.pages_ws, self.slot_map, self.src, self.held_len, self.refs,
                                     self.free_pages, self.n_free, self.n_free, self.copies, self.n_copies)
            flamia_paged_copy(self.prob, self.caches, self.caches, self.copies, self.n_copies, self.pages_ws)
        else:
            flamia_paged_plan(self.prob, self.ws, self.slot_map, self.held_len, self.free_pages, self.n_free, self.n_free)
        torch.where(self.status == OK, self.kv_len, self.held_len, out=self.held_len)

    def compact(self):
        """The pages in use to ids 0 .. n_pages - n_free - 1 of every layer's pools, tables and data (``shared`` only).
        Between steps: the next plan must follow before append and attend.  ``pages_status`` says whether it was done."""
        if not self.shared:
            raise FlamiaError(ERR_INVALID_ARG, "PagedCall.compact")
        flamia_paged_compact(self.prob, self.pages_ws, self.held_len, self.refs, self.free_pages, self.n_free, self.copies,
                             self.n_copies)
        flamia_paged_copy(self.prob, self.caches, self.caches, self.copies, self.n_copies, self.pages_ws)

    def append(self, layer, k, v):
        """k, v [T, Hkv, d] (in_dtype, contiguous); rows behind cu_q[n_req] may hold anything."""
        rows, dtype = (self.T, self.Hkv, self.d), self.kv_dtype
        self._check("append", self.ws.device, (k, rows, dtype), (v, rows, dtype))
        flamia_paged_append(self.prob, k, v, self.slot_map, self.caches[layer], self.ws)

    def attend(self, layer, q):
        """q [T, H, d] bf16, contiguous; returns (O, lse), overwritten by the next call."""
        self._check("attend", self.ws.device, (q, self.O.shape, self.O.dtype))
        flamia_paged_fwd(self.prob, q, self.caches[layer], self.O, self.lse, self.ws)
        return self.O, self.lse
