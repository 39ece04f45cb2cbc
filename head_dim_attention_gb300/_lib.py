"""ctypes binding of libffpa.so: argument marshalling only.

Each Python function here has the name of the C entry point it calls and does
nothing but fill ``ffpa_tensor_t`` descriptors from torch tensors (pointer,
dtype, sizes, strides) and pass the current CUDA stream.  Every step of the
computation runs in the library's kernels.  If the library cannot be built or
loaded, loading raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build as _build

FFPA_F16, FFPA_BF16, FFPA_F32 = 0, 1, 2
STATUS = {0: "FFPA_OK", 1: "FFPA_ERR_INVALID_ARG", 2: "FFPA_ERR_UNSUPPORTED", 3: "FFPA_ERR_ALIGNMENT",
          4: "FFPA_ERR_CUDA", 5: "FFPA_ERR_TIMEOUT", 6: "FFPA_ERR_SCRATCH_LIMIT"}
EXPORTS = ("ffpa_fwd", "ffpa_bwd", "ffpa_fwd_dropout", "ffpa_bwd_dropout", "ffpa_fwd_decode_noalloc",
           "ffpa_fwd_varlen", "ffpa_bwd_varlen", "ffpa_fwd_tree", "ffpa_cache_plan", "ffpa_cache_append",
           "ffpa_status_string", "ffpa_check_status",
           "ffpa_set_timing_events", "ffpa_selftest_wait_timeout", "ffpa_version")


class FfpaTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class FfpaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


_LIB = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libffpa.so (building it first if it is missing or stale)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    lib_path = path or _build.build()
    if not os.path.exists(lib_path):
        raise FileNotFoundError(lib_path)
    lib = ctypes.CDLL(lib_path)
    P = ctypes.POINTER(FfpaTensor)
    lib.ffpa_fwd.argtypes = [P, P, P, P, ctypes.c_int, ctypes.c_float, P, P, ctypes.c_void_p]
    lib.ffpa_fwd.restype = ctypes.c_int
    lib.ffpa_bwd.argtypes = [P, P, P, P, ctypes.c_int, ctypes.c_float, P, P, P, P, P, P, ctypes.c_void_p]
    lib.ffpa_bwd.restype = ctypes.c_int
    D, U64, U32 = ctypes.c_double, ctypes.c_uint64, ctypes.c_uint32
    lib.ffpa_fwd_dropout.argtypes = [P, P, P, P, ctypes.c_int, ctypes.c_float, D, U64, U32, P, P, ctypes.c_void_p]
    lib.ffpa_fwd_dropout.restype = ctypes.c_int
    lib.ffpa_bwd_dropout.argtypes = [P, P, P, P, ctypes.c_int, ctypes.c_float, D, U64, U32, P, P, P, P, P, P,
                                     ctypes.c_void_p]
    lib.ffpa_bwd_dropout.restype = ctypes.c_int
    lib.ffpa_fwd_decode_noalloc.argtypes = [P, P, P, P, ctypes.c_int, ctypes.c_float, P, P, ctypes.c_void_p]
    lib.ffpa_fwd_decode_noalloc.restype = ctypes.c_int
    # the packed and paged calls: descriptors as addresses (a ctypes structure by reference, or packed bytes)
    I, F, L, V = ctypes.c_int, ctypes.c_float, ctypes.c_int64, ctypes.c_void_p
    for name, args in (("ffpa_fwd_varlen", [V, V, V, V, I, I, F, V, V, V]),
                       ("ffpa_bwd_varlen", [V, V, V, V, I, I, F, V, V, V, V, V, V, V]),
                       ("ffpa_fwd_tree", [V, V, V, V, I, V, V, V, I, F, V, V, V]),
                       ("ffpa_cache_plan", [V, V, I, I, V, I, V, I, V, V, V, L, V, V, V]),
                       ("ffpa_cache_append", [V, V, V, V, V, V])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = I
    lib.ffpa_status_string.argtypes = [ctypes.c_int]
    lib.ffpa_status_string.restype = ctypes.c_char_p
    lib.ffpa_check_status.argtypes = [ctypes.c_void_p]
    lib.ffpa_check_status.restype = ctypes.c_int
    lib.ffpa_set_timing_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
    lib.ffpa_set_timing_events.restype = ctypes.c_int
    lib.ffpa_selftest_wait_timeout.argtypes = [ctypes.c_void_p]
    lib.ffpa_selftest_wait_timeout.restype = ctypes.c_int
    lib.ffpa_version.argtypes = []
    lib.ffpa_version.restype = ctypes.c_int
    if path is None:
        _LIB = lib
    return lib


def _dtype_code(t) -> int:
    import torch
    return {torch.float16: FFPA_F16, torch.bfloat16: FFPA_BF16, torch.float32: FFPA_F32}.get(t.dtype, -1)


def describe(t, as_lse: bool = False):
    """ffpa_tensor_t for a torch tensor (4-D; an lse [B,H,N] gets a trailing size-1 dim)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("ffpa tensors must be CUDA tensors (the library takes device pointers)")
    d = FfpaTensor()
    d.data = t.data_ptr()
    d.dtype = _dtype_code(t)
    d.reserved = 0
    shape, stride = list(t.shape), list(t.stride())
    if as_lse and len(shape) == 3:
        shape, stride = shape + [1], stride + [1]
    if len(shape) != 4:
        raise ValueError("ffpa tensors are 4-D")
    for i in range(4):
        d.shape[i] = shape[i]
        d.stride[i] = stride[i]
    return d


def check_devices(tensors, current: int) -> None:
    """All tensors of one call on one CUDA device, and that device the current
    one: the library encodes its TMA maps, reads its status word and launches
    on the current device, so a tensor elsewhere would be addressed from the
    wrong GPU."""
    devs = {(t.device.type, t.device.index) for t in tensors if t is not None}
    if len(devs) != 1:
        raise ValueError(f"ffpa tensors must all be on one CUDA device, got {sorted(map(str, devs))}")
    kind, index = devs.pop()
    if kind != "cuda":
        raise ValueError("ffpa tensors must be CUDA tensors (the library takes device pointers)")
    if index != current:
        raise ValueError(f"ffpa tensors are on cuda:{index} but the current device is cuda:{current}; "
                         f"call torch.cuda.set_device({index}) or use torch.cuda.device({index}) first")


def _current_device() -> int:
    import torch
    return torch.cuda.current_device()


def _ref(d):
    return None if d is None else ctypes.byref(d)


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _raise(code: int):
    if code != 0:
        raise FfpaError(code, load().ffpa_status_string(code).decode())


def ffpa_fwd(q, k, v, bias, causal, scale, out, lse, stream=None) -> None:
    """Call ffpa_fwd on torch tensors (device memory); raises FfpaError on a non-zero status."""
    lib = load()
    check_devices((q, k, v, bias, out, lse), _current_device())
    ds = [describe(q), describe(k), describe(v), describe(bias), describe(out), describe(lse, as_lse=True)]
    rc = lib.ffpa_fwd(_ref(ds[0]), _ref(ds[1]), _ref(ds[2]), _ref(ds[3]), int(causal), float(scale),
                      _ref(ds[4]), _ref(ds[5]), _stream(stream))
    _raise(rc)


def ffpa_fwd_dropout(q, k, v, bias, causal, scale, dropout_p, seed, offset, out, lse, stream=None) -> None:
    """Call ffpa_fwd_dropout (the forward with dropout on P); raises FfpaError on a non-zero status."""
    lib = load()
    check_devices((q, k, v, bias, out, lse), _current_device())
    ds = [describe(q), describe(k), describe(v), describe(bias), describe(out), describe(lse, as_lse=True)]
    rc = lib.ffpa_fwd_dropout(_ref(ds[0]), _ref(ds[1]), _ref(ds[2]), _ref(ds[3]), int(causal), float(scale),
                              float(dropout_p), int(seed), int(offset), _ref(ds[4]), _ref(ds[5]), _stream(stream))
    _raise(rc)


def ffpa_bwd_dropout(q, k, v, bias, causal, scale, dropout_p, seed, offset, out, lse, dout, dq, dk, dv,
                     stream=None) -> None:
    """Call ffpa_bwd_dropout (the backward of ffpa_fwd_dropout with the same p, seed and offset)."""
    lib = load()
    check_devices((q, k, v, bias, out, lse, dout, dq, dk, dv), _current_device())
    ds = [describe(x) for x in (q, k, v, bias, out)] + [describe(lse, as_lse=True)] + \
        [describe(x) for x in (dout, dq, dk, dv)]
    rc = lib.ffpa_bwd_dropout(*[_ref(x) for x in ds[:4]], int(causal), float(scale), float(dropout_p), int(seed),
                              int(offset), *[_ref(x) for x in ds[4:]], _stream(stream))
    _raise(rc)


def ffpa_fwd_decode_noalloc(q, k, v, bias, causal, scale, out, lse, stream=None) -> None:
    """Call ffpa_fwd_decode_noalloc (decode forward, Nq <= 16, no device allocation)."""
    lib = load()
    check_devices((q, k, v, bias, out, lse), _current_device())
    ds = [describe(q), describe(k), describe(v), describe(bias), describe(out), describe(lse, as_lse=True)]
    rc = lib.ffpa_fwd_decode_noalloc(_ref(ds[0]), _ref(ds[1]), _ref(ds[2]), _ref(ds[3]), int(causal),
                                     float(scale), _ref(ds[4]), _ref(ds[5]), _stream(stream))
    _raise(rc)


def ffpa_bwd(q, k, v, bias, causal, scale, out, lse, dout, dq, dk, dv, stream=None) -> None:
    """Call ffpa_bwd on torch tensors (device memory); raises FfpaError on a non-zero status."""
    lib = load()
    check_devices((q, k, v, bias, out, lse, dout, dq, dk, dv), _current_device())
    ds = [describe(x) for x in (q, k, v, bias, out)] + [describe(lse, as_lse=True)] + \
        [describe(x) for x in (dout, dq, dk, dv)]
    rc = lib.ffpa_bwd(*[_ref(x) for x in ds[:4]], int(causal), float(scale), *[_ref(x) for x in ds[4:]],
                      _stream(stream))
    _raise(rc)


# The packed and paged calls are often shorter on the GPU than a descriptor built
# field by field is on the host, so theirs are packed in one go: a tensor costs
# about 1 us instead of 3, a call 5 to 12 us instead of 20 to 30.
_DESCRIPTOR = struct.Struct("Pii8q")  # ffpa_tensor_t
_CODES = {torch.float16: FFPA_F16, torch.bfloat16: FFPA_BF16, torch.float32: FFPA_F32}


def _pack(t):
    """ffpa_tensor_t of a 4-D tensor, as bytes."""
    shape = t.shape
    if len(shape) != 4:
        raise ValueError("ffpa tensors are 4-D")
    return _DESCRIPTOR.pack(t.data_ptr(), _CODES.get(t.dtype, -1), 0, *shape, *t.stride())


def _pack_lse(t):
    """ffpa_tensor_t of an lse [B, H, N] or [B, H, N, 1] (None: no lse), as bytes."""
    if t is None or t.dim() != 3:
        return None if t is None else _pack(t)
    return _DESCRIPTOR.pack(t.data_ptr(), _CODES.get(t.dtype, -1), 0, *t.shape, 1, *t.stride(), 1)


def _ints(t, name, shape, dtype=torch.int32):
    """Address of a contiguous integer (or bool) tensor of the given shape."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
                     f"{tuple(t.shape)}{'' if t.is_contiguous() else ', not contiguous'}")


def _row(t, name, dtype=torch.int32):
    """Address and size of a contiguous 1-D integer tensor."""
    n = t.shape[0] if t.dim() == 1 else -1
    return _ints(t, name, (n,), dtype), n


def _device(*tensors) -> int:
    """The current device, once every tensor has been found on it (check_devices says what is wrong otherwise)."""
    current = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != current:
            check_devices(tensors, current)
    return current


def _raw_stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else int(stream)


def ffpa_fwd_varlen(q, k, v, cu_seqlens, causal, scale, out, lse, stream=None) -> None:
    """Call ffpa_fwd_varlen (the forward over packed sequences); raises FfpaError on a non-zero status."""
    lib = load()
    cu, n = _row(cu_seqlens, "cu_seqlens")
    dev = _device(q, k, v, cu_seqlens, out, lse)
    rc = lib.ffpa_fwd_varlen(_pack(q), _pack(k), _pack(v), cu, n - 1, int(causal), scale, _pack(out),
                             _pack_lse(lse), _raw_stream(stream, dev))
    _raise(rc)


def ffpa_bwd_varlen(q, k, v, cu_seqlens, causal, scale, out, lse, dout, dq, dk, dv, stream=None) -> None:
    """Call ffpa_bwd_varlen (the backward of ffpa_fwd_varlen); raises FfpaError on a non-zero status."""
    lib = load()
    cu, n = _row(cu_seqlens, "cu_seqlens")
    dev = _device(q, k, v, cu_seqlens, out, lse, dout, dq, dk, dv)
    rc = lib.ffpa_bwd_varlen(_pack(q), _pack(k), _pack(v), cu, n - 1, int(causal), scale, _pack(out),
                             _pack_lse(lse), _pack(dout), _pack(dq), _pack(dk), _pack(dv), _raw_stream(stream, dev))
    _raise(rc)


def ffpa_fwd_tree(q, k_cache, v_cache, block_table, seq_lens, draft_lens, tree_mask, scale, out, lse,
                  stream=None) -> None:
    """Call ffpa_fwd_tree (drafted tokens over a paged cache); raises FfpaError on a non-zero status."""
    lib = load()
    B, _, T, _ = q.shape
    pages = block_table.shape[-1]
    table, lens = _ints(block_table, "block_table", (B, pages)), _ints(seq_lens, "seq_lens", (B,))
    drafts = None if draft_lens is None else _ints(draft_lens, "draft_lens", (B,))
    masks = 0 if tree_mask is None else tree_mask.shape[0]
    mask = None if tree_mask is None else _ints(tree_mask, "tree_mask", (masks, T, T), torch.bool)
    dev = _device(q, k_cache, v_cache, block_table, seq_lens, draft_lens, tree_mask, out, lse)
    rc = lib.ffpa_fwd_tree(_pack(q), _pack(k_cache), _pack(v_cache), table, pages, lens, drafts, mask, masks, scale,
                           _pack(out), _pack_lse(lse), _raw_stream(stream, dev))
    _raise(rc)


def ffpa_cache_plan(lens, new_lens, page_size, block_table, free_pages, free_head, cu_new, slots, lens_out,
                    free_head_out, stream=None) -> None:
    """Call ffpa_cache_plan (block tables and slots from request lengths); raises FfpaError on a non-zero status."""
    lib = load()
    (at_lens, n), (at_free, n_free), (at_slots, most) = _row(lens, "lens"), _row(free_pages, "free_pages"), \
        _row(slots, "slots", torch.int64)
    each, one, pages = (n,), (1,), block_table.shape[-1]
    dev = _device(lens, new_lens, block_table, free_pages, free_head, cu_new, slots, lens_out, free_head_out)
    rc = lib.ffpa_cache_plan(
        at_lens, _ints(new_lens, "new_lens", each), n, page_size, _ints(block_table, "block_table", (n, pages)), pages,
        at_free, n_free, _ints(free_head, "free_head", one), _ints(cu_new, "cu_new", (n + 1,)), at_slots, most,
        _ints(lens_out, "lens_out", each), _ints(free_head_out, "free_head_out", one), _raw_stream(stream, dev))
    _raise(rc)


def ffpa_cache_append(k, v, k_cache, v_cache, slots, stream=None) -> None:
    """Call ffpa_cache_append (rows of k and v into their slots); raises FfpaError on a non-zero status."""
    lib = load()
    where = _ints(slots, "slots", (k.shape[2],), torch.int64)
    dev = _device(k, v, k_cache, v_cache, slots)
    _raise(lib.ffpa_cache_append(_pack(k), _pack(v), _pack(k_cache), _pack(v_cache), where, _raw_stream(stream, dev)))


def ffpa_check_status(stream=None) -> int:
    return load().ffpa_check_status(_stream(stream))


def ffpa_status_string(code: int) -> str:
    return load().ffpa_status_string(code).decode()


def ffpa_set_timing_events(events) -> None:
    """Register torch.cuda.Event objects (enable_timing=True) the library records between its launches."""
    handles = [int(e.cuda_event) for e in (events or [])]
    if any(h == 0 for h in handles):
        raise ValueError("record each torch.cuda.Event once before registering it (torch creates events lazily)")
    arr = (ctypes.c_void_p * max(1, len(handles)))(*handles)
    _raise(load().ffpa_set_timing_events(arr if handles else None, len(handles)))


def ffpa_selftest_wait_timeout(stream=None) -> None:
    """Launch the timeout self-check (a wait that nothing completes); see include/ffpa.h."""
    _raise(load().ffpa_selftest_wait_timeout(_stream(stream)))


def ffpa_version() -> int:
    return load().ffpa_version()
