"""Python binding of libpagedfp8 (paged FP8 KV cache + GQA decode, sm_103a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libpagedfp8.so``.  torch supplies device memory and the current
stream.  The entry points mirror the C ABI in ``include/pagedfp8.h``:

* ``pkv_kv_append_fp8``       -- quantise new K/V rows into their pages
* ``pkv_paged_gqa_decode``    -- grouped-query decode attention over the pages
* ``pkv_append_decode_fp8``    -- both in one launch (one whole decode step)
* ``pkv_kv_calibrate``         -- running |K|, |V| maxima per kv head and the scales
* ``pkv_decode_calibrate_split``, ``pkv_decode_set_split_weights``,
  ``pkv_decode_get_split_weights`` -- per-CTA weights of the decode split
* ``pkv_decode_workspace_size``, ``pkv_status_string``, ``pkv_version``
* ``pkv_kv_append_fp4``, ``pkv_kv_read_fp4``, ``pkv_paged_gqa_decode_fp4``,
  ``pkv_paged_prefill_fp4`` -- the 4-bit cache: writing it, reading it back,
  and decode and prefill attention over it with an optional sliding window
* ``pkv_kv_append_fp8b``, ``pkv_kv_read_fp8b``, ``pkv_paged_gqa_decode_fp8b``,
  ``pkv_paged_prefill_fp8b`` -- the same calls for the block-scaled FP8 cache
* ``pkv_plan_pages``, ``pkv_release_pages`` -- a step's pages, block tables,
  slots and positions from its requests' lengths, on the GPU

``kv_append_fp8`` / ``paged_gqa_decode`` are the same calls with the output
and workspace allocated by torch when not given.  There is no CPU fallback:
if the library is not built, loading raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import math
import os
import threading
import warnings

import torch

from . import build as _build

PKV_F32, PKV_BF16 = 0, 1
DEVERR_SLOT, DEVERR_PAGE, DEVERR_SEQLEN, DEVERR_TIMEOUT, DEVERR_PAGESIZE, DEVERR_INTERNAL = 1, 2, 4, 8, 16, 32
DEVERR_POOL = 64
HEAD_DIM = 128
MAX_GROUP = 8
MAX_BATCH = 8192
FP4_ROW_BYTES = 72
FP8B_BLOCK = 16
PAGE_POOL_HEADER = 4
_INT32_MAX = 2 ** 31 - 1

_lib = None
_fast = None                         # the fast path of the block-scaled cache's and the plan's calls
_lock = threading.Lock()


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = f"{what}: status {status} ({pkv_status_string(status)})"
        if status == 6:
            code, name = pkv_last_cuda_error()
            msg += f" [{name} ({code})]"
        super().__init__(msg)
        self.status = status


def lib_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libpagedfp8.so (built in-tree by build()); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build the CUDA library first "
                               "(python -m paged_fp8_kv_03_gb300.build)")
        lib = ctypes.CDLL(path)
        vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        lib.pkv_kv_append_fp8.restype = i32
        lib.pkv_kv_append_fp8.argtypes = [vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, i64, i32, vp, vp]
        lib.pkv_decode_workspace_size.restype = sz
        lib.pkv_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        lib.pkv_paged_gqa_decode.restype = i32
        lib.pkv_paged_gqa_decode.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32,
                                             i64, f32, vp, i32, vp, sz, vp, i32, vp]
        lib.pkv_append_decode_fp8.restype = i32
        lib.pkv_append_decode_fp8.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32,
                                              i32, i32, i32, i64, f32, vp, i32, vp, sz, vp, i32, vp]
        lib.pkv_kv_calibrate.restype = i32
        lib.pkv_kv_calibrate.argtypes = [vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, vp]
        lib.pkv_paged_gqa_decode_noalloc.restype = i32
        lib.pkv_paged_gqa_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32,
                                                     i32, i64, f32, vp, i32, vp, i32, vp]
        lib.pkv_decode_noalloc_scratch_bytes.restype = sz
        lib.pkv_decode_noalloc_scratch_bytes.argtypes = []
        lib.pkv_prefill_workspace_size.restype = sz
        lib.pkv_prefill_workspace_size.argtypes = [i32, i32, i32, i64]
        lib.pkv_paged_prefill.restype = i32
        lib.pkv_paged_prefill.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i64, i32, i32,
                                          i32, i32, i64, ctypes.c_float, vp, i32, vp, sz, vp, vp]
        lib.pkv_kv_append_fp4.restype = i32
        lib.pkv_kv_append_fp4.argtypes = lib.pkv_kv_append_fp8.argtypes
        lib.pkv_kv_read_fp4.restype = i32
        lib.pkv_kv_read_fp4.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, i64, i32, vp, vp, i32, vp, vp]
        lib.pkv_decode_fp4_workspace_size.restype = sz
        lib.pkv_decode_fp4_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        lib.pkv_paged_gqa_decode_fp4.restype = i32
        lib.pkv_paged_gqa_decode_fp4.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32,
                                                 i64, f32, i32, i32, vp, i32, vp, sz, vp, i32, vp]
        lib.pkv_prefill_fp4_workspace_size.restype = sz
        lib.pkv_prefill_fp4_workspace_size.argtypes = [i32, i32, i32, i32, i64, i32, i32]
        lib.pkv_paged_prefill_fp4.restype = i32
        lib.pkv_paged_prefill_fp4.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i64, i32,
                                              i32, i32, i32, i64, f32, i32, i32, vp, i32, vp, sz, vp, vp]
        lib.pkv_kv_append_fp8b.restype = i32
        lib.pkv_kv_append_fp8b.argtypes = [vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, i64, i32, vp, vp]
        lib.pkv_kv_read_fp8b.restype = i32
        lib.pkv_kv_read_fp8b.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, i64, i32, vp, vp, i32, vp, vp]
        lib.pkv_decode_fp8b_workspace_size.restype = sz
        lib.pkv_decode_fp8b_workspace_size.argtypes = lib.pkv_decode_fp4_workspace_size.argtypes
        lib.pkv_paged_gqa_decode_fp8b.restype = i32
        lib.pkv_paged_gqa_decode_fp8b.argtypes = lib.pkv_paged_gqa_decode_fp4.argtypes
        lib.pkv_prefill_fp8b_workspace_size.restype = sz
        lib.pkv_prefill_fp8b_workspace_size.argtypes = lib.pkv_prefill_fp4_workspace_size.argtypes
        lib.pkv_paged_prefill_fp8b.restype = i32
        lib.pkv_paged_prefill_fp8b.argtypes = lib.pkv_paged_prefill_fp4.argtypes
        lib.pkv_plan_pages.restype = i32
        lib.pkv_plan_pages.argtypes = [vp, vp, i32, vp, i32, i32, vp, i64, vp, vp, vp, vp, i32, vp, vp]
        lib.pkv_release_pages.restype = i32
        lib.pkv_release_pages.argtypes = [vp, vp, i32, vp, i32, i32, vp, i64, vp, vp]
        lib.pkv_read_device_error.restype = i32
        lib.pkv_read_device_error.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_int32), vp]
        lib.pkv_decode_set_split_weights.restype = i32
        lib.pkv_decode_set_split_weights.argtypes = [vp, i32]
        lib.pkv_decode_get_split_weights.restype = i32
        lib.pkv_decode_get_split_weights.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_int)]
        lib.pkv_decode_calibrate_split.restype = i32
        lib.pkv_decode_calibrate_split.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32,
                                                   i64, f32, vp, i32, vp, sz, i32, i32, vp, i32,
                                                   ctypes.POINTER(ctypes.c_int), vp]
        lib.pkv_last_cuda_error.restype = i32
        lib.pkv_last_cuda_error.argtypes = [ctypes.POINTER(ctypes.c_char_p)]
        lib.pkv_test_withhold_load.restype = None
        lib.pkv_test_withhold_load.argtypes = [i32]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_status_string.argtypes = [i32]
        lib.pkv_version.restype = i32
        lib.pkv_version.argtypes = []
        _load_fast()
        _lib = lib
        return lib


class _NoFast:
    """In the place of the fast path where there is none: every call goes on to the checks in Python."""
    append = read = decode = prefill = plan = release = staticmethod(lambda *args: None)


def _load_fast() -> None:
    global _fast
    path, name = _build.BINDING, __name__ + "._binding"
    loader = importlib.machinery.ExtensionFileLoader(name, path)
    try:
        module = importlib.util.module_from_spec(importlib.util.spec_from_file_location(name, path, loader=loader))
        loader.exec_module(module)
    except ImportError as error:
        warnings.warn(f"the binding's fast path does not load ({error}): calls of the block-scaled cache and of the page plan "
                      "are checked in Python, which takes 4 to 7 us longer a call (python -m paged_fp8_kv_03_gb300.build)",
                      RuntimeWarning, stacklevel=3)
        module = _NoFast
    _fast = module


def _load_and_fast():
    load()
    return _fast


def _done(st, what) -> None:
    if st != 0:
        raise PkvError(st, what)


def pkv_read_device_error(device_error, clear: bool = False, stream=None) -> int:
    """The bits of a device error word (waits for the work enqueued on the
    stream); with clear=True the word is reset to 0 afterwards."""
    _need(device_error, "device_error", torch.int32)
    code = ctypes.c_int32(0)
    with _device_of(device_error):
        st = load().pkv_read_device_error(_ptr(device_error), 1 if clear else 0, ctypes.byref(code), _stream(stream))
    if st != 0:
        raise PkvError(st, "pkv_read_device_error")
    return int(code.value)


def pkv_decode_set_split_weights(weights, device=None) -> None:
    """Install per-CTA split weights (ints in [768, 1280]) for decode calls on
    `device` (default: the current one) whose grid has len(weights) CTAs;
    None or an empty sequence removes them (even split)."""
    w = [int(x) for x in (weights if weights is not None else [])]
    if any(x < 0 or x > 0xFFFF for x in w):
        raise PkvError(2, "pkv_decode_set_split_weights")
    buf = (ctypes.c_uint16 * max(1, len(w)))(*w)
    with _device_of_index(device):
        st = load().pkv_decode_set_split_weights(ctypes.addressof(buf), len(w))
    if st != 0:
        raise PkvError(st, "pkv_decode_set_split_weights")


def pkv_decode_get_split_weights(device=None) -> list:
    """The split weights installed for `device` (empty: even split)."""
    cap = 1024
    buf = (ctypes.c_uint16 * cap)()
    n = ctypes.c_int(0)
    with _device_of_index(device):
        st = load().pkv_decode_get_split_weights(ctypes.addressof(buf), cap, ctypes.byref(n))
    if st != 0:
        raise PkvError(st, "pkv_decode_get_split_weights")
    return list(buf[:n.value])


def pkv_decode_calibrate_split(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace,
                               sm_scale=None, max_ctas=0, rounds=6, stream=None, max_seq_len=0,
                               seq_page_sizes=None) -> list:
    """Measure and install split weights for decode calls shaped like this
    one (runs 4 * rounds decode calls on these inputs, writing out and
    workspace, and synchronises the stream).  Returns the weights."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(k_scale, "k_scale", torch.float32, 1)
    _need(v_scale, "v_scale", torch.float32, 1)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(out, "out", dim=3)
    _need(workspace, "workspace", torch.uint8)
    B, Hq, D = q.shape
    NP, Hkv, P, D2 = k_cache.shape
    if v_cache.shape != k_cache.shape or D2 != D or out.shape != q.shape:
        raise ValueError("q / cache / out shapes disagree")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens shapes disagree with q")
    _check_page_sizes(seq_page_sizes, B)
    _same_device(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace, seq_page_sizes)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    cap = 1024
    buf = (ctypes.c_uint16 * cap)()
    n = ctypes.c_int(0)
    with _device_of(q):
        st = load().pkv_decode_calibrate_split(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                               _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
                                               int(max_seq_len), _ptr(seq_page_sizes), B, Hq, Hkv, D, P, NP,
                                               float(sm_scale), _ptr(out), _act_code(out), _ptr(workspace),
                                               workspace.numel(), int(max_ctas), int(rounds),
                                               ctypes.addressof(buf), cap, ctypes.byref(n), _stream(stream))
    if st != 0:
        raise PkvError(st, "pkv_decode_calibrate_split")
    return list(buf[:n.value])


def pkv_test_withhold_load(index: int) -> None:
    """Test facility (failure-detection tests only): decode worker warp /
    prefill CTA `index` skips its first load so its bounded wait runs out;
    a negative index turns it off."""
    load().pkv_test_withhold_load(int(index))


def pkv_last_cuda_error():
    """(code, name) of the CUDA error behind this thread's last PKV_ERR_CUDA."""
    name = ctypes.c_char_p()
    code = load().pkv_last_cuda_error(ctypes.byref(name))
    return int(code), (name.value or b"").decode()


def pkv_status_string(status: int) -> str:
    return load().pkv_status_string(int(status)).decode()


def pkv_version() -> int:
    return int(load().pkv_version())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _device_of(t):
    """Runs a call with the tensors' device current: the library launches on
    the current device and takes the current stream of that device."""
    if t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _device_of_index(device):
    if device is None:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _same_device(ref, *ts):
    for t in ts:
        if t is not None and t.device != ref.device:
            raise ValueError(f"all tensors must be on {ref.device}, got one on {t.device}")


def _check_page_sizes(seq_page_sizes, batch):
    if seq_page_sizes is not None:
        _need(seq_page_sizes, "seq_page_sizes", torch.int32, 1)
        if seq_page_sizes.shape[0] != batch:
            raise ValueError("seq_page_sizes must have one entry per sequence")


def _need(t, name, dtype=None, dim=None, cuda=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _act_code(t) -> int:
    if t.dtype == torch.float32:
        return PKV_F32
    if t.dtype == torch.bfloat16:
        return PKV_BF16
    raise TypeError(f"activations must be float32 or bfloat16, got {t.dtype}")


def pkv_kv_append_fp8(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache,
                      device_error=None, stream=None) -> None:
    """k_new/v_new [T, Hkv, 128] fp32|bf16; slot_mapping int64 [T]; scales fp32
    [Hkv]; caches uint8 [num_pages, Hkv, P, 128] (written in place)."""
    _need(k_new, "k_new", dim=3)
    _need(v_new, "v_new", dtype=k_new.dtype, dim=3)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need(k_scale, "k_scale", torch.float32, 1)
    _need(v_scale, "v_scale", torch.float32, 1)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    if device_error is not None:
        _need(device_error, "device_error", torch.int32)
    T, H, D = k_new.shape
    NP, H2, P, D2 = k_cache.shape
    if v_new.shape != k_new.shape or v_cache.shape != k_cache.shape or H2 != H or D2 != D:
        raise ValueError("k/v shapes disagree")
    if slot_mapping.shape[0] != T or k_scale.shape[0] != H or v_scale.shape[0] != H:
        raise ValueError("slot_mapping / scale shapes disagree")
    _same_device(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache, device_error)
    with _device_of(k_new):
        st = load().pkv_kv_append_fp8(_ptr(k_new), _ptr(v_new), _act_code(k_new), T, H, D, _ptr(slot_mapping),
                                      _ptr(k_scale), _ptr(v_scale), _ptr(k_cache), _ptr(v_cache), NP, P,
                                      _ptr(device_error), _stream(stream))
    if st != 0:
        raise PkvError(st, "pkv_kv_append_fp8")


def pkv_kv_calibrate(k_new, v_new, k_running_max, v_running_max, k_scale=None, v_scale=None,
                     stream=None) -> None:
    """Fold prefill rows k_new/v_new [T, Hkv, 128] (fp32|bf16) into the running
    per-head maxima (fp32 [Hkv], in place) and, if given, write the scales
    max(running_max / 448, 1e-12)."""
    _need(k_new, "k_new", dim=3)
    _need(v_new, "v_new", dtype=k_new.dtype, dim=3)
    for t, n in ((k_running_max, "k_running_max"), (v_running_max, "v_running_max")):
        _need(t, n, torch.float32, 1)
    if (k_scale is None) != (v_scale is None):
        raise ValueError("give both scales or neither")
    if k_scale is not None:
        _need(k_scale, "k_scale", torch.float32, 1)
        _need(v_scale, "v_scale", torch.float32, 1)
    T, H, D = k_new.shape
    if v_new.shape != k_new.shape or k_running_max.shape[0] != H or v_running_max.shape[0] != H:
        raise ValueError("shapes disagree")
    _same_device(k_new, v_new, k_running_max, v_running_max, k_scale, v_scale)
    with _device_of(k_new):
        st = load().pkv_kv_calibrate(_ptr(k_new), _ptr(v_new), _act_code(k_new), T, H, D, _ptr(k_running_max),
                                     _ptr(v_running_max), _ptr(k_scale), _ptr(v_scale), _stream(stream))
    if st != 0:
        raise PkvError(st, "pkv_kv_calibrate")


def pkv_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim=HEAD_DIM, max_seq_len=0, page_size=16,
                              max_ctas=0) -> int:
    """Workspace bytes of a decode call whose seq_lens are all <= max_seq_len."""
    return int(load().pkv_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, int(max_seq_len),
                                                page_size, max_ctas))


def pkv_paged_gqa_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace,
                         sm_scale=None, device_error=None, max_ctas=0, stream=None, max_seq_len=0,
                         seq_page_sizes=None) -> None:
    """q bf16 [B, Hq, 128]; caches uint8 [num_pages, Hkv, P, 128]; scales fp32
    [Hkv]; block_table int32 [B, max_pages]; seq_lens int32 [B]; out
    [B, Hq, 128] bf16 or fp32; workspace uint8 (pkv_decode_workspace_size
    bytes for max_seq_len); seq_page_sizes int32 [B] or None (tokens per page
    of each sequence, a power-of-two multiple of P: runs of pool pages)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(k_scale, "k_scale", torch.float32, 1)
    _need(v_scale, "v_scale", torch.float32, 1)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(out, "out", dim=3)
    _need(workspace, "workspace", torch.uint8)
    if device_error is not None:
        _need(device_error, "device_error", torch.int32)
    B, Hq, D = q.shape
    NP, Hkv, P, D2 = k_cache.shape
    if v_cache.shape != k_cache.shape or D2 != D or out.shape != q.shape:
        raise ValueError("q / cache / out shapes disagree")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens shapes disagree with q")
    _check_page_sizes(seq_page_sizes, B)
    _same_device(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace, device_error,
                 seq_page_sizes)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    with _device_of(q):
        st = load().pkv_paged_gqa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                         _ptr(block_table), block_table.shape[1], _ptr(seq_lens), int(max_seq_len),
                                         _ptr(seq_page_sizes), B, Hq, Hkv, D, P, NP, float(sm_scale), _ptr(out),
                                         _act_code(out), _ptr(workspace), workspace.numel(), _ptr(device_error),
                                         int(max_ctas), _stream(stream))
    if st != 0:
        raise PkvError(st, "pkv_paged_gqa_decode")


def pkv_append_decode_fp8(k_new, v_new, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out,
                          workspace, sm_scale=None, device_error=None, max_ctas=0, stream=None, max_seq_len=0,
                          seq_page_sizes=None) -> None:
    """One fused decode step: k_new/v_new [B, n_new, Hkv, 128] (fp32|bf16) are
    quantised into the cache at positions seq_lens[b] - n_new .. seq_lens[b] - 1
    (seq_lens counts them), then attention as pkv_paged_gqa_decode."""
    _need(k_new, "k_new", dim=4)
    _need(v_new, "v_new", dtype=k_new.dtype, dim=4)
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(k_scale, "k_scale", torch.float32, 1)
    _need(v_scale, "v_scale", torch.float32, 1)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(out, "out", dim=3)
    _need(workspace, "workspace", torch.uint8)
    if device_error is not None:
        _need(device_error, "device_error", torch.int32)
    B, Hq, D = q.shape
    NP, Hkv, P, D2 = k_cache.shape
    Bn, n_new, Hn, Dn = k_new.shape
    if v_cache.shape != k_cache.shape or D2 != D or out.shape != q.shape:
        raise ValueError("q / cache / out shapes disagree")
    if v_new.shape != k_new.shape or Bn != B or Hn != Hkv or Dn != D:
        raise ValueError("k_new / v_new must be [B, n_new, Hkv, head_dim]")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens shapes disagree with q")
    _check_page_sizes(seq_page_sizes, B)
    _same_device(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace, k_new, v_new,
                 device_error, seq_page_sizes)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    with _device_of(k_new):
        st = load().pkv_append_decode_fp8(_ptr(k_new), _ptr(v_new), _act_code(k_new), n_new, _ptr(q), _ptr(k_cache),
                                          _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_table),
                                          block_table.shape[1], _ptr(seq_lens), int(max_seq_len),
                                          _ptr(seq_page_sizes), B, Hq, Hkv, D, P, NP, float(sm_scale), _ptr(out),
                                          _act_code(out), _ptr(workspace), workspace.numel(), _ptr(device_error),
                                          int(max_ctas), _stream(stream))
    if st != 0:
        raise PkvError(st, "pkv_append_decode_fp8")


def append_decode_fp8(k_new, v_new, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out=None,
                      out_dtype=torch.bfloat16, workspace=None, sm_scale=None, device_error=None, max_ctas=0,
                      stream=None, max_seq_len=0, seq_page_sizes=None) -> torch.Tensor:
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    max_seq_len = _default_max_len(block_table, k_cache, max_seq_len, seq_page_sizes)
    if workspace is None:
        workspace = decode_workspace(q.shape[0], q.shape[1], k_cache.shape[1], k_cache.shape[2], q.device,
                                     max_ctas, max_seq_len)
    pkv_append_decode_fp8(k_new, v_new, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out,
                          workspace, sm_scale, device_error, max_ctas, stream, max_seq_len, seq_page_sizes)
    return out


def _default_max_len(block_table, k_cache, max_seq_len, seq_page_sizes):
    """The allocating forms bound seq_lens by the table's capacity at the pool
    page size unless told otherwise; with per-sequence page sizes the bound
    must be given."""
    if max_seq_len:
        return int(max_seq_len)
    if seq_page_sizes is not None:
        raise ValueError("give max_seq_len when seq_page_sizes is given")
    return int(block_table.shape[1] * k_cache.shape[2])


def pkv_paged_gqa_decode_noalloc(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out,
                                 sm_scale=None, device_error=None, max_ctas=0, stream=None, max_seq_len=0,
                                 seq_page_sizes=None) -> None:
    """pkv_paged_gqa_decode without a workspace, for callers that cannot
    allocate device memory: the split-K scratch is a fixed array inside the
    library (see pkv_decode_noalloc_scratch_bytes).  Calls that overlap on the
    GPU share that array and race; calls on one stream are safe."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(k_scale, "k_scale", torch.float32, 1)
    _need(v_scale, "v_scale", torch.float32, 1)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(out, "out", dim=3)
    if device_error is not None:
        _need(device_error, "device_error", torch.int32)
    B, Hq, D = q.shape
    NP, Hkv, P, D2 = k_cache.shape
    if v_cache.shape != k_cache.shape or D2 != D or out.shape != q.shape:
        raise ValueError("q / cache / out shapes disagree")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens shapes disagree with q")
    _check_page_sizes(seq_page_sizes, B)
    _same_device(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, device_error, seq_page_sizes)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    with _device_of(q):
        st = load().pkv_paged_gqa_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                                 _ptr(v_scale), _ptr(block_table), block_table.shape[1],
                                                 _ptr(seq_lens), int(max_seq_len), _ptr(seq_page_sizes), B, Hq, Hkv,
                                                 D, P, NP, float(sm_scale), _ptr(out), _act_code(out),
                                                 _ptr(device_error), int(max_ctas), _stream(stream))
    if st != 0:
        raise PkvError(st, "pkv_paged_gqa_decode_noalloc")


def pkv_decode_noalloc_scratch_bytes() -> int:
    return int(load().pkv_decode_noalloc_scratch_bytes())


_ws_cache: dict = {}


def decode_workspace(batch, num_q_heads, num_kv_heads, page_size, device=None, max_ctas=0,
                     max_seq_len=0) -> torch.Tensor:
    """A workspace tensor for these sizes, cached per (device, stream, sizes).
    Calls that use it must not overlap on the GPU (same stream is fine)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    stream = torch.cuda.current_stream(device).cuda_stream
    key = (device.index, stream, batch, num_q_heads, num_kv_heads, page_size, max_ctas, max_seq_len)
    ws = _ws_cache.get(key)
    if ws is None:
        with torch.cuda.device(device):
            n = pkv_decode_workspace_size(batch, num_q_heads, num_kv_heads, HEAD_DIM, max_seq_len, page_size,
                                          max_ctas)
        if n == 0:
            raise PkvError(4, "pkv_decode_workspace_size")
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def kv_append_fp8(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache, device_error=None,
                  stream=None) -> None:
    pkv_kv_append_fp8(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache, device_error, stream)


def paged_gqa_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out=None,
                     out_dtype=torch.bfloat16, workspace=None, sm_scale=None, device_error=None, max_ctas=0,
                     stream=None, max_seq_len=0, seq_page_sizes=None) -> torch.Tensor:
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    max_seq_len = _default_max_len(block_table, k_cache, max_seq_len, seq_page_sizes)
    if workspace is None:
        workspace = decode_workspace(q.shape[0], q.shape[1], k_cache.shape[1], k_cache.shape[2], q.device,
                                     max_ctas, max_seq_len)
    pkv_paged_gqa_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace,
                         sm_scale, device_error, max_ctas, stream, max_seq_len, seq_page_sizes)
    return out


def pkv_prefill_workspace_size(batch, num_kv_heads, max_kv_len, max_total_kv=0) -> int:
    return int(load().pkv_prefill_workspace_size(int(batch), int(num_kv_heads), int(max_kv_len),
                                                 int(max_total_kv)))


def pkv_paged_prefill(q, cu_q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, max_q_len,
                      max_kv_len, workspace, sm_scale=None, device_error=None, stream=None, max_total_kv=0,
                      seq_page_sizes=None) -> None:
    """q bf16 [total_q, Hq, 128] (the chunks of all sequences back to back);
    cu_q int32 [B + 1] row offsets; seq_lens int32 [B] (lengths including the
    chunk); caches, scales, block_table and seq_page_sizes as for decode; out
    [total_q, Hq, 128] bf16 or fp32; max_q_len / max_kv_len bounds of the
    chunk lengths and of seq_lens, max_total_kv (0 or) a bound of their sum;
    workspace uint8 (pkv_prefill_workspace_size bytes)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(cu_q, "cu_q", torch.int32, 1)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(k_scale, "k_scale", torch.float32, 1)
    _need(v_scale, "v_scale", torch.float32, 1)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(out, "out", dim=3)
    _need(workspace, "workspace", torch.uint8)
    if device_error is not None:
        _need(device_error, "device_error", torch.int32)
    T, Hq, D = q.shape
    NP, Hkv, P, D2 = k_cache.shape
    B = seq_lens.shape[0]
    if v_cache.shape != k_cache.shape or D2 != D or out.shape != q.shape:
        raise ValueError("q / cache / out shapes disagree")
    if block_table.shape[0] != B or cu_q.shape[0] != B + 1:
        raise ValueError("block_table / cu_q shapes disagree with seq_lens")
    _check_page_sizes(seq_page_sizes, B)
    _same_device(q, cu_q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace, device_error,
                 seq_page_sizes)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    with _device_of(q):
        st = load().pkv_paged_prefill(_ptr(q), _ptr(cu_q), T, int(max_q_len), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(k_scale), _ptr(v_scale), _ptr(block_table), block_table.shape[1],
                                      _ptr(seq_lens), _ptr(seq_page_sizes), B, int(max_kv_len), int(max_total_kv),
                                      Hq, Hkv, D, P, NP, float(sm_scale), _ptr(out), _act_code(out),
                                      _ptr(workspace), workspace.numel(), _ptr(device_error), _stream(stream))
    if st != 0:
        raise PkvError(st, "pkv_paged_prefill")


def paged_prefill(q, cu_q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, max_q_len, out=None,
                  out_dtype=torch.bfloat16, max_kv_len=None, workspace=None, sm_scale=None, device_error=None,
                  stream=None, max_total_kv=0, seq_page_sizes=None) -> torch.Tensor:
    """Allocating convenience form: max_kv_len defaults to the block table's
    capacity (max_pages x page size; give it with seq_page_sizes), the
    workspace to a fresh buffer."""
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if max_kv_len is None:
        if seq_page_sizes is not None:
            raise ValueError("give max_kv_len when seq_page_sizes is given")
        max_kv_len = block_table.shape[1] * k_cache.shape[2]
    if workspace is None:
        workspace = torch.empty(pkv_prefill_workspace_size(seq_lens.shape[0], k_cache.shape[1], max_kv_len,
                                                           max_total_kv), dtype=torch.uint8, device=q.device)
    pkv_paged_prefill(q, cu_q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, max_q_len,
                      max_kv_len, workspace, sm_scale, device_error, stream, max_total_kv, seq_page_sizes)
    return out


# ---------------------------------------------------------------------------
# the 4-bit cache
# ---------------------------------------------------------------------------
# A decode step makes these calls once a layer and the smallest of them run for
# a few microseconds, so the checks are made in one pass over each tensor.
def _addr(t, name, dtype, dim, dev):
    """The address of a contiguous tensor of this type and number of
    dimensions on CUDA device index dev."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a CUDA device")
        raise ValueError(f"all tensors must be on cuda:{dev}, got {name} on {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _cuda_index(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return dev


def _act(t, name):
    if t.dtype is torch.bfloat16:
        return PKV_BF16
    if t.dtype is torch.float32:
        return PKV_F32
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _call(name, dev, stream, fn, *args):
    """fn(*args, stream) with device dev current; stream None: its current one."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _call(name, dev, stream, fn, *args)
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream
    else:
        raw = int(stream)
    st = fn(*args, raw)
    if st != 0:
        raise PkvError(st, name)


def _fp4_pools(k_cache, v_cache, dev):
    """Addresses, pages, kv heads and page size of a K and a V pool."""
    k, v = _addr(k_cache, "k_cache", torch.uint8, 4, dev), _addr(v_cache, "v_cache", torch.uint8, 4, dev)
    shape = k_cache.shape
    if v_cache.shape != shape or shape[3] != FP4_ROW_BYTES:
        raise ValueError(f"4-bit caches must be uint8 [num_pages, Hkv, P, {FP4_ROW_BYTES}], both alike")
    return k, v, shape[0], shape[1], shape[2]


def _fp4_rows(slot_mapping, k_scale, v_scale, k, v, H, dev):
    """What append and read back share: addresses of slots, scales and rows."""
    shape = k.shape
    slots = _addr(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    ks, vs = _addr(k_scale, "k_scale", torch.float32, 1, dev), _addr(v_scale, "v_scale", torch.float32, 1, dev)
    if v.shape != shape or shape[1] != H:
        raise ValueError("k/v shapes disagree")
    if slot_mapping.shape[0] != shape[0] or k_scale.shape[0] != H or v_scale.shape[0] != H:
        raise ValueError("slot_mapping / scale shapes disagree")
    return slots, ks, vs, shape[0], shape[2]


def _error_word(device_error, dev):
    return None if device_error is None else _addr(device_error, "device_error", torch.int32, None, dev)


def _fp4_attention(q, out, k_scale, v_scale, block_table, seq_lens, seq_page_sizes, workspace, Hkv, dev):
    """What decode and prefill share: the tensors' addresses."""
    try:
        if out.shape != q.shape:
            raise ValueError("q / out shapes disagree")
        B = seq_lens.shape[0]
        if k_scale.shape[0] != Hkv or v_scale.shape[0] != Hkv:
            raise ValueError("scales must have one entry per kv head")
        if block_table.shape[0] != B or (seq_page_sizes is not None and seq_page_sizes.shape[0] != B):
            raise ValueError("block_table, seq_lens and seq_page_sizes must have one entry per sequence")
    except (AttributeError, IndexError):                       # no tensor, or of no dimensions: refused below
        pass
    return (_addr(q, "q", torch.bfloat16, 3, dev), _addr(out, "out", getattr(out, "dtype", None), 3, dev),
            _act(out, "out"), _addr(k_scale, "k_scale", torch.float32, 1, dev),
            _addr(v_scale, "v_scale", torch.float32, 1, dev), _addr(block_table, "block_table", torch.int32, 2, dev),
            _addr(seq_lens, "seq_lens", torch.int32, 1, dev),
            None if seq_page_sizes is None else _addr(seq_page_sizes, "seq_page_sizes", torch.int32, 1, dev),
            _addr(workspace, "workspace", torch.uint8, None, dev))


def _on(stream, device):
    """Where a call allocates: memory belongs to the stream that uses it (else
    work still ahead on the current stream may write to it, or get it next)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device) if int(stream) else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _check_window(window, sinks):
    """Both as the library's 32-bit arguments; no sequence is longer than the
    largest of them."""
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    return min(int(window), _INT32_MAX), min(int(sinks), _INT32_MAX)


def _int32(value, name):
    """value as a 32-bit argument (ctypes would keep its low bits)."""
    value = int(value)
    if not -_INT32_MAX <= value <= _INT32_MAX:
        raise ValueError(f"{name} must fit 32 bits, got {value}")
    return value


def fp4_cache(num_pages, num_kv_heads, page_size, device=None) -> torch.Tensor:
    """One zeroed 4-bit pool (K or V): uint8 [num_pages, Hkv, P, 72]."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return torch.zeros((num_pages, num_kv_heads, page_size, FP4_ROW_BYTES), dtype=torch.uint8, device=device)


def pkv_kv_append_fp4(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache,
                      device_error=None, stream=None) -> None:
    """k_new/v_new [T, Hkv, 128] fp32|bf16; slot_mapping int64 [T] (negative:
    not written); scales fp32 [Hkv]; caches uint8 [num_pages, Hkv, P, 72]
    (written in place)."""
    dev = _cuda_index(k_new, "k_new")
    k, v = _addr(k_new, "k_new", k_new.dtype, 3, dev), _addr(v_new, "v_new", k_new.dtype, 3, dev)
    kc, vc, NP, H, P = _fp4_pools(k_cache, v_cache, dev)
    slots, ks, vs, T, D = _fp4_rows(slot_mapping, k_scale, v_scale, k_new, v_new, H, dev)
    _call("pkv_kv_append_fp4", dev, stream, (_lib or load()).pkv_kv_append_fp4, k, v, _act(k_new, "k_new"), T, H, D,
          slots, ks, vs, kc, vc, NP, P, _error_word(device_error, dev))


def pkv_kv_read_fp4(slot_mapping, k_scale, v_scale, k_cache, v_cache, k_out, v_out, device_error=None,
                    stream=None) -> None:
    """The rows at slot_mapping (int64 [T]) as values, into k_out/v_out
    [T, Hkv, 128] fp32|bf16; rows of negative slots are left as they were."""
    dev = _cuda_index(k_out, "k_out")
    k, v = _addr(k_out, "k_out", k_out.dtype, 3, dev), _addr(v_out, "v_out", k_out.dtype, 3, dev)
    kc, vc, NP, H, P = _fp4_pools(k_cache, v_cache, dev)
    slots, ks, vs, T, D = _fp4_rows(slot_mapping, k_scale, v_scale, k_out, v_out, H, dev)
    _call("pkv_kv_read_fp4", dev, stream, (_lib or load()).pkv_kv_read_fp4, slots, T, H, D, ks, vs, kc, vc, NP, P, k,
          v, _act(k_out, "k_out"), _error_word(device_error, dev))


def kv_append_fp4(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache, device_error=None,
                  stream=None) -> None:
    pkv_kv_append_fp4(k_new, v_new, slot_mapping, k_scale, v_scale, k_cache, v_cache, device_error, stream)


def kv_read_fp4(slot_mapping, k_scale, v_scale, k_cache, v_cache, k_out=None, v_out=None,
                out_dtype=torch.bfloat16, device_error=None, stream=None) -> tuple:
    """Allocating form of pkv_kv_read_fp4: (K, V) [T, Hkv, 128]; without
    outputs given, rows of negative slots are zeros."""
    if (k_out is None) != (v_out is None):
        raise ValueError("give both outputs or neither")
    if k_out is None:
        shape = (slot_mapping.shape[0], k_cache.shape[1], HEAD_DIM)
        with _on(stream, slot_mapping.device):
            k_out = torch.zeros(shape, dtype=out_dtype, device=slot_mapping.device)
            v_out = torch.zeros_like(k_out)
    pkv_kv_read_fp4(slot_mapping, k_scale, v_scale, k_cache, v_cache, k_out, v_out, device_error, stream)
    return k_out, v_out


def pkv_decode_fp4_workspace_size(batch, num_q_heads, num_kv_heads, head_dim=HEAD_DIM, max_seq_len=0, page_size=16,
                                  max_ctas=0) -> int:
    """Workspace bytes of a 4-bit decode call of these sizes."""
    return int(load().pkv_decode_fp4_workspace_size(int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim),
                                                    _int32(max_seq_len, "max_seq_len"), int(page_size),
                                                    _int32(max_ctas, "max_ctas")))


def pkv_paged_gqa_decode_fp4(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace,
                             sm_scale=None, device_error=None, max_ctas=0, stream=None, max_seq_len=0,
                             seq_page_sizes=None, window=0, sinks=0) -> None:
    """pkv_paged_gqa_decode over 4-bit caches uint8 [num_pages, Hkv, P, 72];
    window > 0: only the last `window` tokens and the first `sinks` are
    attended.  workspace uint8 (pkv_decode_fp4_workspace_size bytes)."""
    dev = _cuda_index(q, "q")
    kc, vc, NP, Hkv, P = _fp4_pools(k_cache, v_cache, dev)
    qa, oa, odt, ks, vs, bt, lens, psz, ws = _fp4_attention(q, out, k_scale, v_scale, block_table, seq_lens,
                                                           seq_page_sizes, workspace, Hkv, dev)
    B, Hq, D = q.shape
    if seq_lens.shape[0] != B:
        raise ValueError("seq_lens must have one entry per row of q")
    window, sinks = _check_window(window, sinks)
    _call("pkv_paged_gqa_decode_fp4", dev, stream, (_lib or load()).pkv_paged_gqa_decode_fp4, qa, kc, vc, ks, vs, bt,
          block_table.shape[1], lens, _int32(max_seq_len, "max_seq_len"), psz, B, Hq, Hkv, D, P, NP,
          1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale), window, sinks, oa, odt, ws, workspace.numel(),
          _error_word(device_error, dev), _int32(max_ctas, "max_ctas"))


def paged_gqa_decode_fp4(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out=None,
                         out_dtype=torch.bfloat16, workspace=None, sm_scale=None, device_error=None, max_ctas=0,
                         stream=None, max_seq_len=0, seq_page_sizes=None, window=0, sinks=0) -> torch.Tensor:
    """Allocating form of pkv_paged_gqa_decode_fp4 (on the stream it runs on)."""
    if out is None:
        with _on(stream, q.device):
            out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    max_seq_len = _default_max_len(block_table, k_cache, max_seq_len, seq_page_sizes)
    if workspace is None:
        _cuda_index(q, "q")
        with _device_of(q):
            n = pkv_decode_fp4_workspace_size(q.shape[0], q.shape[1], k_cache.shape[1], q.shape[2], max_seq_len,
                                              k_cache.shape[2], max_ctas)
        if n == 0:
            raise PkvError(4, "pkv_decode_fp4_workspace_size")
        with _on(stream, q.device):
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    pkv_paged_gqa_decode_fp4(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace, sm_scale,
                             device_error, max_ctas, stream, max_seq_len, seq_page_sizes, window, sinks)
    return out


def pkv_prefill_fp4_workspace_size(batch, num_kv_heads, max_q_len, max_kv_len, max_total_kv=0, window=0,
                                   sinks=0) -> int:
    window, sinks = (max(-1, min(int(x), _INT32_MAX)) for x in (window, sinks))
    return int(load().pkv_prefill_fp4_workspace_size(int(batch), int(num_kv_heads), _int32(max_q_len, "max_q_len"),
                                                     _int32(max_kv_len, "max_kv_len"), int(max_total_kv), window,
                                                     sinks))


def pkv_paged_prefill_fp4(q, cu_q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, max_q_len,
                          max_kv_len, workspace, sm_scale=None, device_error=None, stream=None, max_total_kv=0,
                          seq_page_sizes=None, window=0, sinks=0) -> None:
    """pkv_paged_prefill over 4-bit caches uint8 [num_pages, Hkv, P, 72];
    window > 0: a query sees itself, the window - 1 tokens before it and the
    first `sinks` tokens.  workspace uint8 (pkv_prefill_fp4_workspace_size
    bytes for the same bounds)."""
    dev = _cuda_index(q, "q")
    kc, vc, NP, Hkv, P = _fp4_pools(k_cache, v_cache, dev)
    qa, oa, odt, ks, vs, bt, lens, psz, ws = _fp4_attention(q, out, k_scale, v_scale, block_table, seq_lens,
                                                           seq_page_sizes, workspace, Hkv, dev)
    cu = _addr(cu_q, "cu_q", torch.int32, 1, dev)
    T, Hq, D = q.shape
    B = seq_lens.shape[0]
    if cu_q.shape[0] != B + 1:
        raise ValueError("cu_q must have one entry more than seq_lens")
    window, sinks = _check_window(window, sinks)
    _call("pkv_paged_prefill_fp4", dev, stream, (_lib or load()).pkv_paged_prefill_fp4, qa, cu, T,
          _int32(max_q_len, "max_q_len"), kc, vc, ks, vs, bt, block_table.shape[1], lens, psz, B,
          _int32(max_kv_len, "max_kv_len"), int(max_total_kv), Hq, Hkv, D, P, NP,
          1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale), window, sinks, oa, odt, ws, workspace.numel(),
          _error_word(device_error, dev))


def paged_prefill_fp4(q, cu_q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, max_q_len, out=None,
                      out_dtype=torch.bfloat16, max_kv_len=None, workspace=None, sm_scale=None, device_error=None,
                      stream=None, max_total_kv=0, seq_page_sizes=None, window=0, sinks=0) -> torch.Tensor:
    """Allocating form of pkv_paged_prefill_fp4 (on the stream it runs on):
    max_kv_len defaults to the block table's capacity, as in paged_prefill."""
    if out is None:
        with _on(stream, q.device):
            out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if max_kv_len is None:
        if seq_page_sizes is not None:
            raise ValueError("give max_kv_len when seq_page_sizes is given")
        max_kv_len = block_table.shape[1] * k_cache.shape[2]
    if workspace is None:
        _check_window(window, sinks)
        n = pkv_prefill_fp4_workspace_size(seq_lens.shape[0], k_cache.shape[1], max_q_len, max_kv_len, max_total_kv,
                                           window, sinks)
        with _on(stream, q.device):
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    pkv_paged_prefill_fp4(q, cu_q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, max_q_len,
                          max_kv_len, workspace, sm_scale, device_error, stream, max_total_kv, seq_page_sizes,
                          window, sinks)
    return out


# ---------------------------------------------------------------------------
# the block-scaled FP8 cache
# ---------------------------------------------------------------------------
# These calls, and the page plan's, go through the compiled binding where their
# tensors are plain, on the current device, and the stream is the current one.  It
# returns None for anything else, and for whatever is wrong, and the checks below say
# what, or make the call.
def fp8b_cache(num_pages, num_kv_heads, page_size, device=None) -> tuple:
    """One zeroed block-scaled pool (K or V): codes uint8 [num_pages, Hkv, P, 128]
    and exponent bytes uint8 [num_pages, Hkv, P / 16]."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return (torch.zeros((num_pages, num_kv_heads, page_size, HEAD_DIM), dtype=torch.uint8, device=device),
            torch.zeros((num_pages, num_kv_heads, page_size // FP8B_BLOCK), dtype=torch.uint8, device=device))


def _fp8b_pools(k_cache, v_cache, k_exp, v_exp, dev):
    """Addresses, pages, kv heads and page size of the pools."""
    k, v = _addr(k_cache, "k_cache", torch.uint8, 4, dev), _addr(v_cache, "v_cache", torch.uint8, 4, dev)
    ke, ve = _addr(k_exp, "k_exp", torch.uint8, 3, dev), _addr(v_exp, "v_exp", torch.uint8, 3, dev)
    shape = k_cache.shape
    if v_cache.shape != shape or shape[3] != HEAD_DIM:
        raise ValueError(f"caches must be uint8 [num_pages, Hkv, P, {HEAD_DIM}], both alike")
    if k_exp.shape != v_exp.shape or tuple(k_exp.shape) != (shape[0], shape[1], shape[2] // FP8B_BLOCK):
        raise ValueError(f"k_exp and v_exp must be uint8 [num_pages, Hkv, P / {FP8B_BLOCK}]")
    return k, v, ke, ve, shape[0], shape[1], shape[2]


def _fp8b_rows(slot_mapping, k, v, H, dev):
    """What append and read back share: the slots' address, tokens and head_dim."""
    slots = _addr(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    if v.shape != k.shape or k.shape[1] != H:
        raise ValueError("k/v shapes disagree")
    if slot_mapping.shape[0] != k.shape[0]:
        raise ValueError("slot_mapping must have one entry per token")
    return slots, k.shape[0], k.shape[2]


def pkv_kv_append_fp8b(k_new, v_new, slot_mapping, k_cache, v_cache, k_exp, v_exp, device_error=None,
                       stream=None) -> None:
    """k_new/v_new [T, Hkv, 128] fp32|bf16; slot_mapping int64 [T] (negative: not
    written; a block's tokens within 32 consecutive ones, as sequence by sequence
    they are); caches uint8
    [num_pages, Hkv, P, 128] and k_exp/v_exp uint8 [num_pages, Hkv, P / 16]
    (written in place)."""
    st = (_fast or _load_and_fast()).append(k_new, v_new, slot_mapping, k_cache, v_cache, k_exp, v_exp, device_error, stream)
    if st is not None:
        return _done(st, "pkv_kv_append_fp8b")
    dev = _cuda_index(k_new, "k_new")
    k, v = _addr(k_new, "k_new", k_new.dtype, 3, dev), _addr(v_new, "v_new", k_new.dtype, 3, dev)
    kc, vc, ke, ve, NP, H, P = _fp8b_pools(k_cache, v_cache, k_exp, v_exp, dev)
    slots, T, D = _fp8b_rows(slot_mapping, k_new, v_new, H, dev)
    _call("pkv_kv_append_fp8b", dev, stream, (_lib or load()).pkv_kv_append_fp8b, k, v, _act(k_new, "k_new"), T, H, D,
          slots, kc, vc, ke, ve, NP, P, _error_word(device_error, dev))


def kv_append_fp8b(k_new, v_new, slot_mapping, k_cache, v_cache, k_exp, v_exp, device_error=None,
                   stream=None) -> None:
    pkv_kv_append_fp8b(k_new, v_new, slot_mapping, k_cache, v_cache, k_exp, v_exp, device_error, stream)


def pkv_kv_read_fp8b(slot_mapping, k_cache, v_cache, k_exp, v_exp, k_out, v_out, device_error=None,
                     stream=None) -> None:
    """The rows at slot_mapping (int64 [T]) as values, into k_out/v_out
    [T, Hkv, 128] fp32|bf16; rows of negative slots are left as they were."""
    st = (_fast or _load_and_fast()).read(slot_mapping, k_cache, v_cache, k_exp, v_exp, k_out, v_out, device_error, stream)
    if st is not None:
        return _done(st, "pkv_kv_read_fp8b")
    dev = _cuda_index(k_out, "k_out")
    k, v = _addr(k_out, "k_out", k_out.dtype, 3, dev), _addr(v_out, "v_out", k_out.dtype, 3, dev)
    kc, vc, ke, ve, NP, H, P = _fp8b_pools(k_cache, v_cache, k_exp, v_exp, dev)
    slots, T, D = _fp8b_rows(slot_mapping, k_out, v_out, H, dev)
    _call("pkv_kv_read_fp8b", dev, stream, (_lib or load()).pkv_kv_read_fp8b, slots, T, H, D, kc, vc, ke, ve, NP, P, k,
          v, _act(k_out, "k_out"), _error_word(device_error, dev))


def kv_read_fp8b(slot_mapping, k_cache, v_cache, k_exp, v_exp, k_out=None, v_out=None, out_dtype=torch.bfloat16,
                 device_error=None, stream=None) -> tuple:
    """Allocating form of pkv_kv_read_fp8b: (K, V) [T, Hkv, 128]; without
    outputs given, rows of negative slots are zeros."""
    if (k_out is None) != (v_out is None):
        raise ValueError("give both outputs or neither")
    if k_out is None:
        shape = (slot_mapping.shape[0], k_cache.shape[1], HEAD_DIM)
        with _on(stream, slot_mapping.device):
            k_out = torch.zeros(shape, dtype=out_dtype, device=slot_mapping.device)
            v_out = torch.zeros_like(k_out)
    pkv_kv_read_fp8b(slot_mapping, k_cache, v_cache, k_exp, v_exp, k_out, v_out, device_error, stream)
    return k_out, v_out


def _fp8b_attention(q, out, block_table, seq_lens, seq_page_sizes, workspace, dev):
    """What decode and prefill share: the tensors' addresses."""
    addrs = (_addr(q, "q", torch.bfloat16, 3, dev), _addr(out, "out", getattr(out, "dtype", None), 3, dev),
             _act(out, "out"), _addr(block_table, "block_table", torch.int32, 2, dev),
             _addr(seq_lens, "seq_lens", torch.int32, 1, dev),
             None if seq_page_sizes is None else _addr(seq_page_sizes, "seq_page_sizes", torch.int32, 1, dev),
             _addr(workspace, "workspace", torch.uint8, None, dev))
    if out.shape != q.shape:
        raise ValueError("q / out shapes disagree")
    B = seq_lens.shape[0]
    if block_table.shape[0] != B or (seq_page_sizes is not None and seq_page_sizes.shape[0] != B):
        raise ValueError("block_table, seq_lens and seq_page_sizes must have one entry per sequence")
    return addrs


def pkv_decode_fp8b_workspace_size(batch, num_q_heads, num_kv_heads, head_dim=HEAD_DIM, max_seq_len=0, page_size=16,
                                   max_ctas=0) -> int:
    """Workspace bytes of a block-scaled decode call of these sizes."""
    return int(load().pkv_decode_fp8b_workspace_size(int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim),
                                                     _int32(max_seq_len, "max_seq_len"), int(page_size),
                                                     _int32(max_ctas, "max_ctas")))


def pkv_paged_gqa_decode_fp8b(q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, out, workspace,
                              sm_scale=None, device_error=None, max_ctas=0, stream=None, max_seq_len=0,
                              seq_page_sizes=None, window=0, sinks=0) -> None:
    """pkv_paged_gqa_decode over block-scaled caches (see pkv_kv_append_fp8b);
    window > 0: only the last `window` tokens and the first `sinks` are
    attended.  workspace uint8 (pkv_decode_fp8b_workspace_size bytes)."""
    st = (_fast or _load_and_fast()).decode(q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, out, workspace, sm_scale,
                                            device_error, max_ctas, stream, max_seq_len, seq_page_sizes, window, sinks)
    if st is not None:
        return _done(st, "pkv_paged_gqa_decode_fp8b")
    dev = _cuda_index(q, "q")
    kc, vc, ke, ve, NP, Hkv, P = _fp8b_pools(k_cache, v_cache, k_exp, v_exp, dev)
    qa, oa, odt, bt, lens, psz, ws = _fp8b_attention(q, out, block_table, seq_lens, seq_page_sizes, workspace, dev)
    B, Hq, D = q.shape
    if seq_lens.shape[0] != B:
        raise ValueError("seq_lens must have one entry per row of q")
    window, sinks = _check_window(window, sinks)
    _call("pkv_paged_gqa_decode_fp8b", dev, stream, (_lib or load()).pkv_paged_gqa_decode_fp8b, qa, kc, vc, ke, ve, bt,
          block_table.shape[1], lens, _int32(max_seq_len, "max_seq_len"), psz, B, Hq, Hkv, D, P, NP,
          1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale), window, sinks, oa, odt, ws, workspace.numel(),
          _error_word(device_error, dev), _int32(max_ctas, "max_ctas"))


def paged_gqa_decode_fp8b(q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, out=None,
                          out_dtype=torch.bfloat16, workspace=None, sm_scale=None, device_error=None, max_ctas=0,
                          stream=None, max_seq_len=0, seq_page_sizes=None, window=0, sinks=0) -> torch.Tensor:
    """Allocating form of pkv_paged_gqa_decode_fp8b (on the stream it runs on)."""
    if out is None:
        with _on(stream, q.device):
            out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    max_seq_len = _default_max_len(block_table, k_cache, max_seq_len, seq_page_sizes)
    if workspace is None:
        _cuda_index(q, "q")
        with _device_of(q):
            n = pkv_decode_fp8b_workspace_size(q.shape[0], q.shape[1], k_cache.shape[1], q.shape[2], max_seq_len,
                                               k_cache.shape[2], max_ctas)
        if n == 0:
            raise PkvError(4, "pkv_decode_fp8b_workspace_size")
        with _on(stream, q.device):
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    pkv_paged_gqa_decode_fp8b(q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, out, workspace, sm_scale,
                              device_error, max_ctas, stream, max_seq_len, seq_page_sizes, window, sinks)
    return out


def pkv_prefill_fp8b_workspace_size(batch, num_kv_heads, max_q_len, max_kv_len, max_total_kv=0, window=0,
                                    sinks=0) -> int:
    window, sinks = (max(-1, min(int(x), _INT32_MAX)) for x in (window, sinks))
    return int(load().pkv_prefill_fp8b_workspace_size(int(batch), int(num_kv_heads), _int32(max_q_len, "max_q_len"),
                                                      _int32(max_kv_len, "max_kv_len"), int(max_total_kv), window,
                                                      sinks))


def pkv_paged_prefill_fp8b(q, cu_q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, out, max_q_len,
                           max_kv_len, workspace, sm_scale=None, device_error=None, stream=None, max_total_kv=0,
                           seq_page_sizes=None, window=0, sinks=0) -> None:
    """pkv_paged_prefill over block-scaled caches (see pkv_kv_append_fp8b);
    window > 0: a query sees itself, the window - 1 tokens before it and the
    first `sinks` tokens.  workspace uint8 (pkv_prefill_fp8b_workspace_size
    bytes for the same bounds)."""
    st = (_fast or _load_and_fast()).prefill(q, cu_q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, out, max_q_len,
                                             max_kv_len, workspace, sm_scale, device_error, stream, max_total_kv,
                                             seq_page_sizes, window, sinks)
    if st is not None:
        return _done(st, "pkv_paged_prefill_fp8b")
    dev = _cuda_index(q, "q")
    kc, vc, ke, ve, NP, Hkv, P = _fp8b_pools(k_cache, v_cache, k_exp, v_exp, dev)
    qa, oa, odt, bt, lens, psz, ws = _fp8b_attention(q, out, block_table, seq_lens, seq_page_sizes, workspace, dev)
    cu = _addr(cu_q, "cu_q", torch.int32, 1, dev)
    T, Hq, D = q.shape
    B = seq_lens.shape[0]
    if cu_q.shape[0] != B + 1:
        raise ValueError("cu_q must have one entry more than seq_lens")
    window, sinks = _check_window(window, sinks)
    _call("pkv_paged_prefill_fp8b", dev, stream, (_lib or load()).pkv_paged_prefill_fp8b, qa, cu, T,
          _int32(max_q_len, "max_q_len"), kc, vc, ke, ve, bt, block_table.shape[1], lens, psz, B,
          _int32(max_kv_len, "max_kv_len"), int(max_total_kv), Hq, Hkv, D, P, NP,
          1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale), window, sinks, oa, odt, ws, workspace.numel(),
          _error_word(device_error, dev))


def paged_prefill_fp8b(q, cu_q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, max_q_len, out=None,
                       out_dtype=torch.bfloat16, max_kv_len=None, workspace=None, sm_scale=None, device_error=None,
                       stream=None, max_total_kv=0, seq_page_sizes=None, window=0, sinks=0) -> torch.Tensor:
    """Allocating form of pkv_paged_prefill_fp8b (on the stream it runs on):
    max_kv_len defaults to the block table's capacity, as in paged_prefill."""
    if out is None:
        with _on(stream, q.device):
            out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if max_kv_len is None:
        if seq_page_sizes is not None:
            raise ValueError("give max_kv_len when seq_page_sizes is given")
        max_kv_len = block_table.shape[1] * k_cache.shape[2]
    if workspace is None:
        _check_window(window, sinks)
        n = pkv_prefill_fp8b_workspace_size(seq_lens.shape[0], k_cache.shape[1], max_q_len, max_kv_len, max_total_kv,
                                            window, sinks)
        with _on(stream, q.device):
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    pkv_paged_prefill_fp8b(q, cu_q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, out, max_q_len, max_kv_len,
                           workspace, sm_scale, device_error, stream, max_total_kv, seq_page_sizes, window, sinks)
    return out


# ---------------------------------------------------------------------------
# the page pool and the page plan
# ---------------------------------------------------------------------------
def page_pool(num_pages, device=None, pages=None) -> torch.Tensor:
    """A pool for plan_pages: int32 [4 + num_pages], its free pages all of
    0 .. num_pages - 1, or the ones given (handed out from the last one on)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    free = torch.arange(num_pages, dtype=torch.int32) if pages is None else torch.as_tensor(pages).to("cpu", torch.int32)
    if free.dim() != 1 or free.numel() > num_pages:
        raise ValueError("pages must be a list of at most num_pages pages")
    pool = torch.zeros(PAGE_POOL_HEADER + num_pages, dtype=torch.int32)
    pool[0] = free.numel()
    pool[PAGE_POOL_HEADER:PAGE_POOL_HEADER + free.numel()] = free
    return pool.to(device)


def _plan_table(block_table, pool, batch, dev):
    """Addresses of table and pool, entries a row, and pages of the pool."""
    bt, pa = _addr(block_table, "block_table", torch.int32, 2, dev), _addr(pool, "pool", torch.int32, 1, dev)
    if block_table.shape[0] != batch:
        raise ValueError("block_table must have one row per sequence")
    if pool.shape[0] <= PAGE_POOL_HEADER:
        raise ValueError(f"pool must be int32 [{PAGE_POOL_HEADER} + num_pages]")
    return bt, pa, block_table.shape[1], pool.shape[0] - PAGE_POOL_HEADER


def pkv_plan_pages(past_lens, new_lens, block_table, pool, page_size, seq_lens, cu_q, slot_mapping, positions=None,
                   device_error=None, stream=None) -> None:
    """Sequence b holds past_lens[b] tokens and brings new_lens[b] (int32 [B]):
    takes the pages it lacks from the pool into block_table [B, max_pages], and
    writes seq_lens [B] (may be past_lens), cu_q [B + 1], slot_mapping int64 [T]
    and positions int32 [T] of the new tokens, back to back; rows behind them get
    slot -1.  All or nothing (see device_error)."""
    st = (_fast or _load_and_fast()).plan(past_lens, new_lens, block_table, pool, page_size, seq_lens, cu_q, slot_mapping, positions,
                                          device_error, stream)
    if st is not None:
        return _done(st, "pkv_plan_pages")
    dev = _cuda_index(past_lens, "past_lens")
    past, new = _addr(past_lens, "past_lens", torch.int32, 1, dev), _addr(new_lens, "new_lens", torch.int32, 1, dev)
    B = past_lens.shape[0]
    bt, pa, mp, NP = _plan_table(block_table, pool, B, dev)
    lens, cu = _addr(seq_lens, "seq_lens", torch.int32, 1, dev), _addr(cu_q, "cu_q", torch.int32, 1, dev)
    slots = _addr(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    pos = None if positions is None else _addr(positions, "positions", torch.int32, 1, dev)
    if new_lens.shape[0] != B or seq_lens.shape[0] != B or cu_q.shape[0] != B + 1:
        raise ValueError("new_lens and seq_lens must have one entry per sequence, cu_q one more")
    if positions is not None and positions.shape != slot_mapping.shape:
        raise ValueError("positions must have one entry per slot")
    _call("pkv_plan_pages", dev, stream, (_lib or load()).pkv_plan_pages, past, new, B, bt, mp, int(page_size), pa, NP,
          lens, cu, slots, pos, _int32(slot_mapping.shape[0], "max_tokens"), _error_word(device_error, dev))


def plan_pages(past_lens, new_lens, block_table, pool, page_size, max_tokens=None, seq_lens=None, cu_q=None,
               slot_mapping=None, positions=None, device_error=None, stream=None) -> tuple:
    """Allocating form of pkv_plan_pages (on the stream it runs on): give
    slot_mapping or max_tokens.  Returns (seq_lens, cu_q, slot_mapping, positions)."""
    if slot_mapping is None and max_tokens is None:
        raise ValueError("give slot_mapping or max_tokens")
    if slot_mapping is not None and max_tokens is not None and max_tokens != slot_mapping.shape[0]:
        raise ValueError("max_tokens must be slot_mapping's length")
    if seq_lens is None or cu_q is None or slot_mapping is None or positions is None:
        _cuda_index(past_lens, "past_lens")
        with _on(stream, past_lens.device):
            B, device = past_lens.shape[0], past_lens.device
            n = slot_mapping.shape[0] if max_tokens is None else max_tokens
            if seq_lens is None:
                seq_lens = torch.empty(B, dtype=torch.int32, device=device)
            if cu_q is None:
                cu_q = torch.empty(B + 1, dtype=torch.int32, device=device)
            if slot_mapping is None:
                slot_mapping = torch.empty(n, dtype=torch.int64, device=device)
            if positions is None:
                positions = torch.empty(n, dtype=torch.int32, device=device)
    pkv_plan_pages(past_lens, new_lens, block_table, pool, page_size, seq_lens, cu_q, slot_mapping, positions,
                   device_error, stream)
    return seq_lens, cu_q, slot_mapping, positions


def pkv_release_pages(seq_lens, block_table, pool, page_size, keep_lens=None, device_error=None, stream=None) -> None:
    """The pages behind keep_lens[b] tokens (None: all) of sequences of
    seq_lens[b] tokens (int32 [B]) go back to the pool.  All or nothing."""
    st = (_fast or _load_and_fast()).release(seq_lens, block_table, pool, page_size, keep_lens, device_error, stream)
    if st is not None:
        return _done(st, "pkv_release_pages")
    dev = _cuda_index(seq_lens, "seq_lens")
    lens = _addr(seq_lens, "seq_lens", torch.int32, 1, dev)
    keep = None if keep_lens is None else _addr(keep_lens, "keep_lens", torch.int32, 1, dev)
    B = seq_lens.shape[0]
    bt, pa, mp, NP = _plan_table(block_table, pool, B, dev)
    if keep_lens is not None and keep_lens.shape[0] != B:
        raise ValueError("keep_lens must have one entry per sequence")
    _call("pkv_release_pages", dev, stream, (_lib or load()).pkv_release_pages, lens, keep, B, bt, mp, int(page_size),
          pa, NP, _error_word(device_error, dev))


def release_pages(seq_lens, block_table, pool, page_size, keep_lens=None, device_error=None, stream=None) -> None:
    pkv_release_pages(seq_lens, block_table, pool, page_size, keep_lens, device_error, stream)



__all__ = ["load", "lib_path", "pkv_kv_append_fp8", "pkv_paged_gqa_decode", "pkv_decode_workspace_size",
           "pkv_paged_gqa_decode_noalloc", "pkv_decode_noalloc_scratch_bytes", "pkv_append_decode_fp8",
           "append_decode_fp8", "pkv_kv_calibrate", "pkv_paged_prefill", "paged_prefill", "pkv_prefill_workspace_size",
           "pkv_status_string", "pkv_version", "pkv_read_device_error", "pkv_test_withhold_load", "kv_append_fp8",
           "paged_gqa_decode", "decode_workspace", "pkv_decode_set_split_weights", "pkv_decode_get_split_weights",
           "pkv_decode_calibrate_split",
           "PkvError", "PKV_F32", "PKV_BF16", "DEVERR_SLOT", "DEVERR_PAGE", "DEVERR_SEQLEN",
           "DEVERR_TIMEOUT", "DEVERR_PAGESIZE", "DEVERR_INTERNAL", "pkv_last_cuda_error",
           "FP4_ROW_BYTES", "fp4_cache", "pkv_kv_append_fp4", "pkv_kv_read_fp4", "kv_append_fp4", "kv_read_fp4",
           "pkv_decode_fp4_workspace_size", "pkv_paged_gqa_decode_fp4", "paged_gqa_decode_fp4",
           "pkv_prefill_fp4_workspace_size", "pkv_paged_prefill_fp4", "paged_prefill_fp4",
           "FP8B_BLOCK", "fp8b_cache", "pkv_kv_append_fp8b", "pkv_kv_read_fp8b", "kv_append_fp8b", "kv_read_fp8b",
           "pkv_decode_fp8b_workspace_size", "pkv_paged_gqa_decode_fp8b", "paged_gqa_decode_fp8b",
           "pkv_prefill_fp8b_workspace_size", "pkv_paged_prefill_fp8b", "paged_prefill_fp8b",
           "DEVERR_POOL", "PAGE_POOL_HEADER", "page_pool", "pkv_plan_pages", "plan_pages", "pkv_release_pages",
           "release_pages"]
