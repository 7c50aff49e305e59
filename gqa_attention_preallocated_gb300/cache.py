"""Python binding: argument marshalling over the libkvc C ABI.

Every step of the path runs in libkvc's kernels; this module only allocates
device memory through PyTorch, checks tensor shapes, and passes raw pointers,
host length arrays and the current CUDA stream.

The API mirrors the pages' ``KVCache.append`` / ``gqa_attention``
("Implement grouped-query attention over a preallocated KV cache...",
"A strong answer") and ``truncate`` / ``reset`` / ``length`` ("16. Prefill,
decode and the KV cache", "Layout and validity").
"""

from __future__ import annotations

import array
import ctypes

import numpy as np
import torch

from ._lib import KVC_BF16, KVC_F32, KVC_FP8_E4M3, KVC_Q4, KVCError, check, lib

_I64P = ctypes.POINTER(ctypes.c_int64)

# storage dtype -> library dtype; FP8 E4M3 and 4-bit ("q4") caches take bf16 q / k_new / v_new / out
_DTYPES = {torch.float32: KVC_F32, torch.bfloat16: KVC_BF16, torch.float8_e4m3fn: KVC_FP8_E4M3, "q4": KVC_Q4}


def _io_dtype(dtype) -> torch.dtype:
    return torch.float32 if dtype == torch.float32 else torch.bfloat16


def _buffers(given, layers: int, shape, dtype: torch.dtype, device: torch.device, name: str) -> list:
    """One buffer a layer: the caller's, checked, or new ones."""
    if given is None:
        return [torch.empty(shape, dtype=dtype, device=device) for _ in range(layers)]
    bufs = list(given)
    for t in bufs:
        if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
            raise KVCError(1, f"{name} must be contiguous {tuple(shape)} {dtype}")
    return bufs


def _layer_buffers(dtype, layers: int, head, d: int, device, k_bufs, v_bufs, k_scales, v_scales):
    """(k, v, k_scale, v_scale) buffer lists: rows [*head, d] of ``dtype``, or for 4-bit caches codes
    [*head, d / 2] uint8 and scale words int32 [*head[:-1], head[-1] rounded up to a multiple of 4]."""
    if dtype != "q4":
        if k_scales is not None or v_scales is not None:
            raise KVCError(1, "scale buffers belong to 4-bit caches")
        shape = (*head, d)
        return (_buffers(k_bufs, layers, shape, dtype, device, "cache buffers"),
                _buffers(v_bufs, layers, shape, dtype, device, "cache buffers"), None, None)
    codes, words = (*head, d // 2), (*head[:-1], -(-head[-1] // 4) * 4)
    return (_buffers(k_bufs, layers, codes, torch.uint8, device, "code buffers"),
            _buffers(v_bufs, layers, codes, torch.uint8, device, "code buffers"),
            _buffers(k_scales, layers, words, torch.int32, device, "scale buffers"),
            _buffers(v_scales, layers, words, torch.int32, device, "scale buffers"))


def _pointers(bufs) -> ctypes.Array:
    return (ctypes.c_void_p * len(bufs))(*[t.data_ptr() for t in bufs])


def _stream_ptr(device: torch.device, stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # (torch.cuda.current_stream builds a Stream object: 2 us of a step's host time)
    return torch._C._cuda_getCurrentRawStream(device.index)


# Host arrays go to the library by address.  Short integer arrays are copied
# through array.array, whose conversion checks the range (0.2 us against 5 us
# for the numpy route on the Grace host); the caller keeps the returned object
# alive across the call.
_SHORT = 128


def _short(a, n: int, code: str):
    if type(a) is np.ndarray:
        if a.ndim != 1 or a.shape[0] != n or n > _SHORT or a.dtype.kind != "i":
            return None
        a = a.tolist()
    elif type(a) is not list or len(a) != n or n > _SHORT:
        return None
    try:
        arr = array.array(code, a)
    except OverflowError:
        raise KVCError(1, f"per-row entry out of int{8 * array.array(code).itemsize} range") from None
    except TypeError:  # not all integers: numpy's conversion decides
        return None
    return arr, arr.buffer_info()[0]


def _i32(a, n: int):
    """(object to keep, address) of n int32 entries."""
    short = _short(a, n, "i")
    if short is not None:
        return short
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    arr = np.ascontiguousarray(np.asarray(a, dtype=np.int64).reshape(-1))
    if arr.shape[0] != n:
        raise KVCError(1, f"expected {n} per-row entries, got {arr.shape[0]}")
    if np.any(arr > np.iinfo(np.int32).max) or np.any(arr < np.iinfo(np.int32).min):
        raise KVCError(1, "per-row entry out of int32 range")
    arr = arr.astype(np.int32)
    return arr, arr.ctypes.data


def _i64(a, n: int, what: str):
    """(object to keep, address) of n int64 entries."""
    short = _short(a, n, "q")
    if short is not None:
        return short
    arr = np.ascontiguousarray(np.asarray(a, dtype=np.int64).reshape(-1))
    if arr.shape[0] != n:
        raise KVCError(1, f"expected {n} {what}")
    return arr, arr.ctypes.data


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


class KVCache:
    """Preallocated K/V buffers [B, Hkv, max_len, d] per layer plus the C handle.

    ``k_bufs`` / ``v_bufs`` may be given (lists of contiguous CUDA tensors of
    that shape); otherwise they are allocated here with ``torch.empty``.  The
    handle borrows them; this object keeps them alive.

    ``dtype="q4"`` holds K and V in 4 bits, with a step and a zero point for
    every row (token and KV head) that appends choose: ``k`` / ``v`` are then
    uint8 codes [B, Hkv, max_len, d / 2] and ``k_scale`` / ``v_scale`` int32
    words [B, Hkv, max_len rounded up to a multiple of 4]; inputs and outputs
    are bf16 (the format is in ``include/kvc.h``, kvc_create_quantized).
    """

    def __init__(self, layers: int, batch: int, kv_heads: int, max_len: int, head_dim: int,
                 dtype=torch.bfloat16, device="cuda", k_bufs=None, v_bufs=None, k_scales=None, v_scales=None):
        if dtype not in _DTYPES:
            raise KVCError(1, f"unsupported dtype {dtype}")
        self.layers, self.B, self.Hkv, self.max_len, self.d = layers, batch, kv_heads, max_len, head_dim
        self.dtype = dtype
        self.io_dtype = _io_dtype(dtype)
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.k, self.v, self.k_scale, self.v_scale = _layer_buffers(
            dtype, layers, (batch, kv_heads, max_len), head_dim, self.device, k_bufs, v_bufs, k_scales, v_scales)
        h = ctypes.c_void_p()
        if dtype == "q4":
            check(lib().kvc_create_quantized(ctypes.byref(h), layers, batch, kv_heads, max_len, head_dim,
                                             _pointers(self.k), _pointers(self.v), _pointers(self.k_scale),
                                             _pointers(self.v_scale)))
        else:
            check(lib().kvc_create(ctypes.byref(h), layers, batch, kv_heads, max_len, head_dim, _DTYPES[dtype],
                                   _pointers(self.k), _pointers(self.v)))
        self._h = h
        self._ws = None
        self._dev_lens = None

    # ------------------------------------------------------------------ state
    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().kvc_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def lens(self, layer: int = 0) -> np.ndarray:
        out = np.zeros(self.B, dtype=np.int64)
        check(lib().kvc_get_lens(self._h, layer, out.ctypes.data_as(_I64P)))
        return out

    def set_lens(self, layer: int, lens) -> None:
        """Adopt lengths for a layer whose buffers were filled by other means."""
        keep, addr = _i64(lens, self.B, "lengths")
        check(lib().kvc_set_lens(self._h, layer, addr))

    def length(self) -> np.ndarray:
        """Per-row length shared by every layer; raises if a forward pass stopped part-way."""
        out = np.zeros(self.B, dtype=np.int64)
        check(lib().kvc_length(self._h, out.ctypes.data_as(_I64P)))
        return out

    def truncate(self, new_lens) -> None:
        keep, addr = _i64(new_lens, self.B, "lengths")
        check(lib().kvc_truncate(self._h, addr))

    def reset(self) -> None:
        check(lib().kvc_reset(self._h))

    def set_kv_scales(self, layer: int, k_scale, v_scale) -> None:
        """One K and one V scale per KV head of an FP8 E4M3 cache's layer (only while it is empty)."""
        ks = np.ascontiguousarray(np.asarray(k_scale, dtype=np.float32).reshape(-1))
        vs = np.ascontiguousarray(np.asarray(v_scale, dtype=np.float32).reshape(-1))
        if ks.shape[0] != self.Hkv or vs.shape[0] != self.Hkv:
            raise KVCError(1, f"k_scale and v_scale need {self.Hkv} entries")
        fp = ctypes.POINTER(ctypes.c_float)
        check(lib().kvc_set_kv_scales(self._h, layer, ks.ctypes.data_as(fp), vs.ctypes.data_as(fp)))

    def set_window(self, window: int, ring: bool = False) -> None:
        """Sliding window (0 = none) and ring storage (slot = position mod max_len), for every layer."""
        check(lib().kvc_set_window(self._h, int(window), 1 if ring else 0))

    def kernel_launches(self) -> int:
        """Kernels this cache's handle has enqueued so far."""
        return int(lib().kvc_kernel_launches(self._h))

    # ------------------------------------------------------------------ compute
    def workspace_bytes(self, q_heads: int, T: int) -> int:
        return int(lib().kvc_workspace_bytes(self._h, q_heads, T))

    def workspace(self, q_heads: int, T: int) -> torch.Tensor | None:
        """A workspace buffer owned by this cache, grown as needed (reused across calls).

        Allocated zeroed, so its error word reads clean (device_status) even
        before a call has used it.
        """
        need = self.workspace_bytes(q_heads, T)
        if need == 0:
            return None
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.zeros(need, dtype=torch.uint8, device=self.device)
        return self._ws

    def _check_tensor(self, t: torch.Tensor, shape, name: str) -> None:
        if tuple(t.shape) != tuple(shape) or t.dtype != self.io_dtype or not t.is_contiguous() or t.device != self.device:
            raise KVCError(1, f"{name} must be a contiguous {self.io_dtype} tensor of shape {tuple(shape)} on {self.device}")

    def append(self, layer: int, k_new: torch.Tensor, v_new: torch.Tensor, n_new, stream=None) -> None:
        """Write k_new[b, :, :n_new[b]] at each row's current length (in place)."""
        T = k_new.shape[2] if k_new.dim() == 4 else -1
        self._check_tensor(k_new, (self.B, self.Hkv, T, self.d), "k_new")
        self._check_tensor(v_new, (self.B, self.Hkv, T, self.d), "v_new")
        keep, nn = _i32(n_new, self.B)
        check(lib().kvc_append(self._h, layer, _ptr(k_new), _ptr(v_new), T, nn,
                               _stream_ptr(self.device, stream)))

    def read(self, layer: int, first, count, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
             stream=None):
        """Rows read back: positions first[b] .. first[b] + count[b] - 1 of row b, as (k, v) [B, Hkv, T, d].

        ``k_out`` / ``v_out`` (both or neither) fix T and keep what they hold
        at t >= count[b]; without them T is the largest count and those entries
        are zeros.  A 4-bit or FP8 cache's values come rounded to bf16.
        """
        keep_first, first_at = _i64(first, self.B, "first positions")
        counts, count_at = _i32(count, self.B)
        if (k_out is None) != (v_out is None):
            raise KVCError(1, "k_out and v_out come together")
        if k_out is None:
            T = max(0, int(max(counts))) if self.B else 0
            with torch.cuda.stream(stream):  # (None: the current one) so that the zeros are there first
                k_out = torch.zeros((self.B, self.Hkv, T, self.d), dtype=self.io_dtype, device=self.device)
                v_out = torch.zeros_like(k_out)
        T = k_out.shape[2] if k_out.dim() == 4 else -1
        self._check_tensor(k_out, (self.B, self.Hkv, T, self.d), "k_out")
        self._check_tensor(v_out, (self.B, self.Hkv, T, self.d), "v_out")
        check(lib().kvc_read(self._h, layer, first_at, count_at, T, _ptr(k_out),
                             _ptr(v_out), _stream_ptr(self.device, stream)))
        return k_out, v_out

    def gqa_attention(self, layer: int, q: torch.Tensor, n_new, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of the chunk just appended: q [B, Hq, T, d] -> out [B, Hq, T, d]."""
        if q.dim() != 4:
            raise KVCError(1, "q must be [B, Hq, T, d]")
        B, Hq, T, d = q.shape
        self._check_tensor(q, (self.B, Hq, T, self.d), "q")
        if out is None:
            out = torch.empty_like(q)
        self._check_tensor(out, q.shape, "out")
        ws = workspace if workspace is not None else self.workspace(Hq, T)
        keep, nn = _i32(n_new, self.B)
        check(lib().kvc_gqa_attention(self._h, layer, _ptr(q), Hq, T, nn, _ptr(out),
                                      _ptr(ws), 0 if ws is None else ws.numel(), _stream_ptr(self.device, stream)))
        return out

    def gqa_attention_noalloc(self, layer: int, q: torch.Tensor, n_new, out: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
        """``gqa_attention`` through the allocation-free entry point (library-owned static scratch).

        For callers that cannot allocate device memory, so ``out`` must be
        passed in: this wrapper allocates nothing either (``out=None`` raises).
        Shapes whose scratch exceeds the static array are rejected.  Errors of
        the kernels stay recorded in the scratch until ``noalloc_status``.
        """
        if q.dim() != 4:
            raise KVCError(1, "q must be [B, Hq, T, d]")
        B, Hq, T, d = q.shape
        self._check_tensor(q, (self.B, Hq, T, self.d), "q")
        if out is None:
            raise KVCError(1, "the allocation-free call takes a caller-owned out tensor (out is None)")
        self._check_tensor(out, q.shape, "out")
        keep, nn = _i32(n_new, self.B)
        check(lib().kvc_gqa_attention_noalloc(self._h, layer, _ptr(q), Hq, T, nn, _ptr(out),
                                              _stream_ptr(self.device, stream)))
        return out

    def append_attention(self, layer: int, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, n_new,
                         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
        """Append then attend, validated together (an error runs neither step)."""
        if q.dim() != 4:
            raise KVCError(1, "q must be [B, Hq, T, d]")
        B, Hq, T, d = q.shape
        self._check_tensor(q, (self.B, Hq, T, self.d), "q")
        self._check_tensor(k_new, (self.B, self.Hkv, T, self.d), "k_new")
        self._check_tensor(v_new, (self.B, self.Hkv, T, self.d), "v_new")
        if out is None:
            out = torch.empty_like(q)
        self._check_tensor(out, q.shape, "out")
        ws = workspace if workspace is not None else self.workspace(Hq, T)
        keep, nn = _i32(n_new, self.B)
        check(lib().kvc_append_attention(self._h, layer, _ptr(q), _ptr(k_new), _ptr(v_new), Hq, T,
                                         nn, _ptr(out), _ptr(ws),
                                         0 if ws is None else ws.numel(), _stream_ptr(self.device, stream)))
        return out

    def append_attention_host(self, layer: int, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, n_new,
                              out: torch.Tensor, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """``append_attention`` on CPU tensors (page-locked for the copies to overlap).

        The library copies positions t < n_new[b] of q, k_new and v_new to its
        own device staging, runs the step on ``stream`` and copies those
        positions of out back; out's other positions are left as they were.
        Returns once enqueued: after ``host_copies_done`` and a synchronize of
        that stream, ``out`` holds the result and the inputs may change.
        """
        if q.dim() != 4:
            raise KVCError(1, "q must be [B, Hq, T, d]")
        B, Hq, T, d = q.shape
        for t, shape, name in ((q, (self.B, Hq, T, self.d), "q"), (k_new, (self.B, self.Hkv, T, self.d), "k_new"),
                               (v_new, (self.B, self.Hkv, T, self.d), "v_new"), (out, (self.B, Hq, T, self.d), "out")):
            if tuple(t.shape) != shape or t.dtype != self.io_dtype or not t.is_contiguous() or t.device.type != "cpu":
                raise KVCError(1, f"{name} must be a contiguous {self.io_dtype} CPU tensor of shape {shape}")
        ws = workspace if workspace is not None else self.workspace(Hq, T)
        keep, nn = _i32(n_new, self.B)
        check(lib().kvc_append_attention_host(self._h, layer, _ptr(q), _ptr(k_new), _ptr(v_new), Hq, T,
                                              nn, _ptr(out), _ptr(ws),
                                              0 if ws is None else ws.numel(), _stream_ptr(self.device, stream)))
        return out

    def host_copies_done(self, stream=None) -> None:
        """Make ``stream`` wait for every output copy of the host-buffer calls enqueued so far."""
        check(lib().kvc_host_copies_done(self._h, _stream_ptr(self.device, stream)))

    # ------------------------------------------------ device-resident lengths
    def lens_to_device(self, stream=None) -> torch.Tensor:
        """Hand the lengths over to a device array (int32 [layers, B]) owned by this object.

        Until ``lens_from_device``, only ``decode_step`` may run: it reads and
        advances the device lengths, so a step can be captured in a CUDA graph.
        """
        n = int(lib().kvc_device_lens_bytes(self._h)) // 4
        self._dev_lens = torch.zeros(max(n, 1), dtype=torch.int32, device=self.device)
        check(lib().kvc_lens_to_device(self._h, self._dev_lens.data_ptr(), _stream_ptr(self.device, stream)))
        return self._dev_lens[:n].view(self.layers, self.B)

    def lens_from_device(self, stream=None) -> None:
        """Make the host lengths authoritative again (copies the device lengths back)."""
        check(lib().kvc_lens_from_device(self._h, _stream_ptr(self.device, stream)))

    def decode_step(self, layer: int, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                    n_new: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, stream=None) -> torch.Tensor:
        """``append_attention`` with the lengths on the device and ``n_new`` a device int32 [B].

        Nothing per-step comes from the host, so the call can be captured in a
        CUDA graph; ``out`` and ``workspace`` must be passed in.
        """
        if q.dim() != 4:
            raise KVCError(1, "q must be [B, Hq, T, d]")
        B, Hq, T, d = q.shape
        self._check_tensor(q, (self.B, Hq, T, self.d), "q")
        self._check_tensor(k_new, (self.B, self.Hkv, T, self.d), "k_new")
        self._check_tensor(v_new, (self.B, self.Hkv, T, self.d), "v_new")
        self._check_tensor(out, q.shape, "out")
        if n_new.dtype != torch.int32 or n_new.device != self.device or n_new.numel() != self.B or not n_new.is_contiguous():
            raise KVCError(1, f"n_new must be a contiguous int32 tensor of {self.B} entries on {self.device}")
        check(lib().kvc_decode_step(self._h, layer, _ptr(q), _ptr(k_new), _ptr(v_new), Hq, T, n_new.data_ptr(),
                                    _ptr(out), _ptr(workspace), workspace.numel(), _stream_ptr(self.device, stream)))
        return out

    def append_attention_tree(self, layer: int, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, n_new,
                              parents, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
        """``append_attention`` for a draft tree: parents [B, T] (-1 = off the cached prefix)."""
        if q.dim() != 4:
            raise KVCError(1, "q must be [B, Hq, T, d]")
        B, Hq, T, d = q.shape
        self._check_tensor(q, (self.B, Hq, T, self.d), "q")
        self._check_tensor(k_new, (self.B, self.Hkv, T, self.d), "k_new")
        self._check_tensor(v_new, (self.B, self.Hkv, T, self.d), "v_new")
        if out is None:
            out = torch.empty_like(q)
        self._check_tensor(out, q.shape, "out")
        ws = workspace if workspace is not None else self.workspace(Hq, T)
        keep, nn = _i32(n_new, self.B)
        keep_par, par = _i32(parents, self.B * T)
        check(lib().kvc_append_attention_tree(self._h, layer, _ptr(q), _ptr(k_new), _ptr(v_new), Hq, T,
                                              nn, par, _ptr(out),
                                              _ptr(ws), 0 if ws is None else ws.numel(),
                                              _stream_ptr(self.device, stream)))
        return out

    def gqa_attention_tree(self, layer: int, q: torch.Tensor, n_new, parents, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """``gqa_attention`` of a chunk already appended, for a draft tree (parents [B, T])."""
        if q.dim() != 4:
            raise KVCError(1, "q must be [B, Hq, T, d]")
        B, Hq, T, d = q.shape
        self._check_tensor(q, (self.B, Hq, T, self.d), "q")
        if out is None:
            out = torch.empty_like(q)
        self._check_tensor(out, q.shape, "out")
        ws = workspace if workspace is not None else self.workspace(Hq, T)
        keep, nn = _i32(n_new, self.B)
        keep_par, par = _i32(parents, self.B * T)
        check(lib().kvc_gqa_attention_tree(self._h, layer, _ptr(q), Hq, T, nn,
                                           par, _ptr(out), _ptr(ws),
                                           0 if ws is None else ws.numel(), _stream_ptr(self.device, stream)))
        return out

    def selftest_bounded_wait(self, limit_ns: int, workspace: torch.Tensor | None = None, stream=None) -> None:
        """Launch the bounded-wait self-test into the workspace's error word."""
        ws = workspace if workspace is not None else self._ws
        if ws is None:
            raise KVCError(7, "no workspace")
        check(lib().kvc_selftest_bounded_wait(_ptr(ws), int(limit_ns), _stream_ptr(self.device, stream)))

    def noalloc_status(self, stream=None) -> int:
        """Synchronize and read the allocation-free calls' error word (0 = clean); raises on a non-zero code."""
        code = ctypes.c_int32(0)
        check(lib().kvc_noalloc_status(_stream_ptr(self.device, stream), ctypes.byref(code)))
        return code.value

    def device_status(self, workspace: torch.Tensor | None = None, stream=None) -> int:
        """Synchronize and read the workspace error word (0 = clean); raises on a non-zero code."""
        ws = workspace if workspace is not None else self._ws
        if ws is None:
            return 0
        code = ctypes.c_int32(0)
        check(lib().kvc_device_status(self._h, _ptr(ws), _stream_ptr(self.device, stream), ctypes.byref(code)))
        return code.value


class PagedKVCache(KVCache):
    """K/V in pages [num_pages, Hkv, page_size, d] per layer behind a device block table.

    ``block_table`` (int32 [B, max_pages_per_row], on the device, owned by
    this object) maps row b's logical page i to a physical page; it starts as
    row b owning pages b * max_pages_per_row .. (as long as num_pages allows,
    else -1) and may be rewritten between calls.  Every call works on the
    logical sequence, with max_len = max_pages_per_row * page_size.  With
    ``dtype="q4"`` the pages hold codes and ``k_scale`` / ``v_scale`` their
    scale words, as in ``KVCache``.
    """

    def __init__(self, layers: int, batch: int, kv_heads: int, page_size: int, num_pages: int,
                 max_pages_per_row: int, head_dim: int, dtype=torch.bfloat16, device="cuda"):
        if dtype not in _DTYPES:
            raise KVCError(1, f"unsupported dtype {dtype}")
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.layers, self.B, self.Hkv, self.d = layers, batch, kv_heads, head_dim
        self.page_size, self.num_pages, self.max_pages_per_row = page_size, num_pages, max_pages_per_row
        self.max_len = max_pages_per_row * page_size
        self.dtype, self.device = dtype, dev
        self.io_dtype = _io_dtype(dtype)
        self.k, self.v, self.k_scale, self.v_scale = _layer_buffers(
            dtype, layers, (num_pages, kv_heads, page_size), head_dim, dev, None, None, None, None)
        ids = torch.arange(batch * max_pages_per_row, dtype=torch.int32, device=dev)
        self.block_table = torch.where(ids < num_pages, ids, torch.full_like(ids, -1)).view(batch, max_pages_per_row)
        h = ctypes.c_void_p()
        if dtype == "q4":
            check(lib().kvc_create_quantized_paged(ctypes.byref(h), layers, batch, kv_heads, page_size, num_pages,
                                                   max_pages_per_row, head_dim, _pointers(self.k), _pointers(self.v),
                                                   _pointers(self.k_scale), _pointers(self.v_scale),
                                                   self.block_table.data_ptr()))
        else:
            check(lib().kvc_create_paged(ctypes.byref(h), layers, batch, kv_heads, page_size, num_pages,
                                         max_pages_per_row, head_dim, _DTYPES[dtype], _pointers(self.k),
                                         _pointers(self.v), self.block_table.data_ptr()))
        self._h = h
        self._ws = None
        self._dev_lens = None


def gqa_attention(q: torch.Tensor, cache: KVCache, n_new, layer: int = 0, **kw) -> torch.Tensor:
    """Module-level form of ``KVCache.gqa_attention`` (the pages' call signature)."""
    return cache.gqa_attention(layer, q, n_new, **kw)
