"""GB300 (sm_103a) Gated DeltaNet decode: Python binding of the C ABI.

The functions here only marshal torch tensors (device pointers, sizes, the
current CUDA stream) into calls of ``libgdn_decode.so``; every step of the
decode path runs in the library's CUDA kernels.  The names follow the C ABI
(``include/gdn_decode.h``):

  GDNStatePool / ConvStatePool   slot-indexed pools (slot 0 = null slot)
  causal_conv1d_decode           depthwise causal conv, one token a row
  gdn_decode_step                gated delta rule per row and value head
  gdn_layer_decode               both in one kernel
  gdn_commit                     twin-slot commit (swap read/write slots)
  linear_attention_decode, linear_attention_prefill   recurrent layers with a
                                 decay for each head and no delta rule
  attn_prologue, paged_attention, kv_pages_*   the attention layers beside the
                                 GDN layers, over a paged cache (KVPagePool)

The operation is the decode step of "mstar PR #1139" ("Why": the GDN rule is
the recurrent state update of one token a row; "What changed": twin slots,
the decode-only conv), with padding on the null slot of "mstar PR #1127".
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _lib
from ._lib import (GDN_BF16, GDN_DEVERR_BAD_PAGE, GDN_DEVERR_BAD_SLOT, GDN_DEVERR_NO_PAGES, GDN_DEVERR_NONE, GDN_DEVERR_TIMEOUT, GDN_F32,
                   GDN_NOALLOC_SCRATCH_SLOTS,
                   GDN_PROBE_INPLACE, GDN_PROBE_READ, GDN_PROBE_TWIN, GDN_PROBE_WRITE, gdn_dims)

__all__ = [
    "GDNError", "load", "lib_path", "GDNStatePool", "ConvStatePool", "causal_conv1d_decode",
    "gdn_decode_step", "gdn_layer_decode", "gdn_layer_decode_noalloc", "gdn_commit", "gdn_validate_slots",
    "gdn_prefill", "gdn_prefill_chunked", "gdn_prefill_chunked_workspace_bytes", "gdn_verify", "causal_conv1d_prefill", "gdn_layer_decode_bucket",
    "get_device_error", "selftest_wait_timeout", "probe_traffic", "GDN_F32", "GDN_BF16", "GDN_DEVERR_NONE",
    "GDN_DEVERR_BAD_SLOT", "GDN_DEVERR_TIMEOUT", "GDN_PROBE_TWIN", "GDN_PROBE_INPLACE", "GDN_PROBE_READ",
    "GDN_PROBE_WRITE", "GDN_NOALLOC_SCRATCH_SLOTS",
]


class GDNError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[gdn status {code}] {msg}")
        self.code = code


def load():
    return _lib.load()


def lib_path() -> str:
    return _lib.lib_path()


def _check(rc: int):
    if rc != 0:
        msg = _lib.load().gdn_last_error().decode(errors="replace")
        raise GDNError(rc, msg)


_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


def _dtype_code(t: torch.dtype) -> int:
    if t not in _DTYPES:
        raise TypeError(f"activation dtype must be float32 or bfloat16, got {t}")
    return _DTYPES[t]


def _stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _ptr(t: Optional[torch.Tensor], what: str, dtype=None, device=None, contiguous=True, host_ok=False):
    """Device pointer of a tensor.  With host_ok, a page-locked (pinned) host
    tensor is accepted too: under unified addressing its pointer is valid on
    the device, and the kernels read or write it across the host link."""
    if t is None:
        return None
    if not t.is_cuda:
        if host_ok and t.is_pinned():
            if dtype is not None and t.dtype != dtype:
                raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
            if contiguous and not t.is_contiguous():
                raise ValueError(f"{what} must be contiguous")
            return t.data_ptr()
        raise ValueError(f"{what} must be a CUDA tensor" + (" or pinned host memory" if host_ok else ""))
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _numel(t: torch.Tensor, n: int, what: str):
    if t.numel() != n:
        raise ValueError(f"{what} has {t.numel()} elements, expected {n}")


class GDNStatePool:
    """Recurrent state pool [num_slots][hv][dv][dk] fp32 in torch-owned memory.

    The library wraps the tensor (it never frees it).  Slot 0 is the null slot.
    The pool also holds its in-place counters (`inplace_counters`, zeroed
    int32 device memory the library's in-place layer launches schedule with);
    `inplace_counters=False` leaves them out, and in-place launches then give
    each CTA whole qk heads.
    """

    def __init__(self, num_slots: int, hk: int, hv: int, dk: int, dv: int, device=None,
                 tensor: Optional[torch.Tensor] = None, inplace_counters: bool = True):
        L = _lib.load()
        device = torch.device(device if device is not None else "cuda")
        if tensor is None:
            tensor = torch.zeros((num_slots, hv, dv, dk), dtype=torch.float32, device=device)
        if tuple(tensor.shape) != (num_slots, hv, dv, dk) or tensor.dtype != torch.float32:
            raise ValueError("state tensor must be float32 [num_slots][hv][dv][dk]")
        self.tensor = tensor
        self.num_slots, self.hk, self.hv, self.dk, self.dv = num_slots, hk, hv, dk, dv
        h = ctypes.c_void_p()
        _check(L.gdn_state_pool_wrap(_ptr(tensor, "state"), num_slots, gdn_dims(hk, hv, dk, dv),
                                     ctypes.byref(h)))
        self._h = h
        self.counters = None
        if inplace_counters:
            nbytes = L.gdn_pool_inplace_counter_bytes(num_slots, gdn_dims(hk, hv, dk, dv))
            self.counters = torch.zeros((nbytes + 3) // 4, dtype=torch.int32, device=tensor.device)
            _check(L.gdn_pool_attach_inplace_counters(h, _ptr(self.counters, "in-place counters"),
                                                      self.counters.numel() * 4))
        self._fast = _lib.fast()  # the C++ binding and the pool as it takes it
        self._p = self._fast.make_state(h.value, hk, hv, dk, dv, tensor.device.index) if self._fast else None

    @property
    def handle(self):
        return self._h

    def zero_slots(self, slots: torch.Tensor):
        _check(_lib.load().gdn_pool_zero_slots(self._h, _ptr(slots, "slots", torch.int32),
                                               slots.numel(), _stream(self.tensor.device)))

    def copy_slots(self, src: torch.Tensor, dst: torch.Tensor):
        """Slot dst[i] receives a copy of slot src[i] (snapshots, forks)."""
        _numel(dst, src.numel(), "dst")
        _check(_lib.load().gdn_pool_copy_slots(self._h, _ptr(src, "src", torch.int32),
                                               _ptr(dst, "dst", torch.int32), src.numel(),
                                               _stream(self.tensor.device)))

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            try:
                if getattr(self, "_p", None):
                    self._fast.drop_state(self._p)
                _lib.load().gdn_state_pool_destroy(h)
            except Exception:
                pass
            self._h = self._p = None


class ConvStatePool:
    """Conv window pool [num_slots][width-1][channels] in the activation dtype."""

    def __init__(self, num_slots: int, channels: int, width: int, dtype=torch.bfloat16, device=None,
                 tensor: Optional[torch.Tensor] = None):
        L = _lib.load()
        device = torch.device(device if device is not None else "cuda")
        if tensor is None:
            tensor = torch.zeros((num_slots, width - 1, channels), dtype=dtype, device=device)
        if tuple(tensor.shape) != (num_slots, width - 1, channels) or tensor.dtype != dtype:
            raise ValueError("conv tensor must be [num_slots][width-1][channels] of the given dtype")
        self.tensor = tensor
        self.num_slots, self.channels, self.width, self.dtype = num_slots, channels, width, dtype
        h = ctypes.c_void_p()
        _check(L.conv_state_pool_wrap(_ptr(tensor, "conv state"), num_slots, channels, width,
                                      _dtype_code(dtype), ctypes.byref(h)))
        self._h = h

    @property
    def handle(self):
        return self._h

    def zero_slots(self, slots: torch.Tensor):
        _check(_lib.load().conv_pool_zero_slots(self._h, _ptr(slots, "slots", torch.int32),
                                                slots.numel(), _stream(self.tensor.device)))

    def copy_slots(self, src: torch.Tensor, dst: torch.Tensor):
        """Slot dst[i] receives a copy of slot src[i] (snapshots, forks)."""
        _numel(dst, src.numel(), "dst")
        _check(_lib.load().conv_pool_copy_slots(self._h, _ptr(src, "src", torch.int32),
                                                _ptr(dst, "dst", torch.int32), src.numel(),
                                                _stream(self.tensor.device)))

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            try:
                _lib.load().conv_state_pool_destroy(h)
            except Exception:
                pass
            self._h = None


def causal_conv1d_decode(x: torch.Tensor, conv_pool: ConvStatePool, slot_idx: torch.Tensor,
                         w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None, write_slot: Optional[torch.Tensor] = None,
                         silu: bool = True) -> torch.Tensor:
    """Conv state update for one token a row. x: [rows][C] (row stride allowed)."""
    rows, C = x.shape
    dt = conv_pool.dtype
    dev = conv_pool.tensor.device
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    if out is None:
        out = torch.empty((rows, C), dtype=dt, device=dev)
    _numel(slot_idx, rows, "slot_idx")
    if write_slot is not None:
        _numel(write_slot, rows, "write_slot")
    _numel(w, C * conv_pool.width, "w")
    if bias is not None:
        _numel(bias, C, "bias")
    _check(_lib.load().causal_conv1d_decode(
        _ptr(x, "x", dt, dev, contiguous=False), x.stride(0), conv_pool.handle,
        _ptr(slot_idx, "slot_idx", torch.int32, dev), _ptr(write_slot, "write_slot", torch.int32, dev),
        _ptr(w, "w", dt, dev), _ptr(bias, "bias", dt, dev), int(bool(silu)),
        _ptr(out, "out", dt, dev, host_ok=True), rows, _dtype_code(dt), _stream(dev)))
    return out


def gdn_decode_step(q, k, v, a, b, A_log, dt_bias, pool: GDNStatePool, read_slot, write_slot=None,
                    out: Optional[torch.Tensor] = None, keep_in_place: bool = False) -> torch.Tensor:
    """Gated delta rule for one token a row. q,k: [rows][hk][dk]; v: [rows][hv][dv]; a,b: [rows][hv].
    q, k, v, a, b and out may be pinned host tensors (read and written across the host link)."""
    rows = q.shape[0]
    dt = q.dtype
    dev = pool.tensor.device
    _numel(q, rows * pool.hk * pool.dk, "q")
    _numel(k, rows * pool.hk * pool.dk, "k")
    _numel(v, rows * pool.hv * pool.dv, "v")
    _numel(a, rows * pool.hv, "a")
    _numel(b, rows * pool.hv, "b")
    _numel(A_log, pool.hv, "A_log")
    _numel(dt_bias, pool.hv, "dt_bias")
    _numel(read_slot, rows, "read_slot")
    if write_slot is not None:
        _numel(write_slot, rows, "write_slot")
    if out is None:
        out = torch.empty((rows, pool.hv, pool.dv), dtype=dt, device=dev)
    _numel(out, rows * pool.hv * pool.dv, "out")
    _check(_lib.load().gdn_decode_step(
        _ptr(q, "q", dt, dev, host_ok=True), _ptr(k, "k", dt, dev, host_ok=True),
        _ptr(v, "v", dt, dev, host_ok=True), _ptr(a, "a", dt, dev, host_ok=True),
        _ptr(b, "b", dt, dev, host_ok=True), _ptr(A_log, "A_log", torch.float32, dev),
        _ptr(dt_bias, "dt_bias", torch.float32, dev), pool.handle,
        _ptr(read_slot, "read_slot", torch.int32, dev), _ptr(write_slot, "write_slot", torch.int32, dev),
        _ptr(out, "out", dt, dev, host_ok=True), rows, pool.hv, int(bool(keep_in_place)), _dtype_code(dt),
        _stream(dev)))
    return out


def _prefill_checks(q, k, v, a, b, A_log, dt_bias, pool, cu_seqlens, read_slot):
    T = q.shape[0]
    nseq = cu_seqlens.numel() - 1
    if nseq < 0:
        raise ValueError("cu_seqlens needs nseq + 1 entries")
    _numel(q, T * pool.hk * pool.dk, "q")
    _numel(k, T * pool.hk * pool.dk, "k")
    _numel(v, T * pool.hv * pool.dv, "v")
    _numel(a, T * pool.hv, "a")
    _numel(b, T * pool.hv, "b")
    _numel(A_log, pool.hv, "A_log")
    _numel(dt_bias, pool.hv, "dt_bias")
    _numel(read_slot, nseq, "read_slot")
    return T, nseq


def gdn_prefill(q, k, v, a, b, A_log, dt_bias, pool: GDNStatePool, cu_seqlens, read_slot, write_slot=None,
                out: Optional[torch.Tensor] = None, keep_in_place: bool = False) -> torch.Tensor:
    """The rule over many tokens a sequence (packed, token-major: q,k [T][hk][dk],
    v [T][hv][dv], a,b [T][hv]; sequence r is tokens cu_seqlens[r]..cu_seqlens[r+1]).
    The final state goes to write_slot (twin) or back to read_slot (in place)."""
    T, nseq = _prefill_checks(q, k, v, a, b, A_log, dt_bias, pool, cu_seqlens, read_slot)
    dt, dev = q.dtype, pool.tensor.device
    if write_slot is not None:
        _numel(write_slot, nseq, "write_slot")
    if out is None:
        out = torch.empty((T, pool.hv, pool.dv), dtype=dt, device=dev)
    _numel(out, T * pool.hv * pool.dv, "out")
    _check(_lib.load().gdn_prefill(
        _ptr(q, "q", dt, dev, host_ok=True), _ptr(k, "k", dt, dev, host_ok=True), _ptr(v, "v", dt, dev, host_ok=True), _ptr(a, "a", dt, dev, host_ok=True),
        _ptr(b, "b", dt, dev, host_ok=True), _ptr(A_log, "A_log", torch.float32, dev),
        _ptr(dt_bias, "dt_bias", torch.float32, dev), pool.handle,
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, dev), _ptr(read_slot, "read_slot", torch.int32, dev),
        _ptr(write_slot, "write_slot", torch.int32, dev), _ptr(out, "out", dt, dev, host_ok=True), nseq, T,
        int(bool(keep_in_place)), _dtype_code(dt), _stream(dev)))
    return out


def gdn_prefill_chunked_workspace_bytes(nseq: int, total_tokens: int, hv: int) -> int:
    """Bytes of the device workspace gdn_prefill_chunked needs for bf16 activations."""
    return int(_lib.load().gdn_prefill_chunked_workspace_bytes(int(nseq), int(total_tokens), int(hv)))


def gdn_prefill_chunked(q, k, v, a, b, A_log, dt_bias, pool: GDNStatePool, cu_seqlens, read_slot,
                        write_slot=None, out: Optional[torch.Tensor] = None,
                        keep_in_place: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gdn_prefill's operation in chunks of 64 tokens on the tensor cores
    (dk = dv = 128): the same arguments and slot semantics, results within
    about 1e-5 relative of gdn_prefill instead of bit-identical.  Its
    activations must be device memory.  bf16 activations use a device
    workspace (a uint8 tensor of at least gdn_prefill_chunked_workspace_bytes;
    allocated here when none is given)."""
    T, nseq = _prefill_checks(q, k, v, a, b, A_log, dt_bias, pool, cu_seqlens, read_slot)
    dt, dev = q.dtype, pool.tensor.device
    if write_slot is not None:
        _numel(write_slot, nseq, "write_slot")
    if out is None:
        out = torch.empty((T, pool.hv, pool.dv), dtype=dt, device=dev)
    _numel(out, T * pool.hv * pool.dv, "out")
    need = gdn_prefill_chunked_workspace_bytes(nseq, T, pool.hv) if dt == torch.bfloat16 else 0
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the pool's device")
        ws_ptr, ws_bytes = ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()
    _check(_lib.load().gdn_prefill_chunked(
        _ptr(q, "q", dt, dev), _ptr(k, "k", dt, dev),
        _ptr(v, "v", dt, dev), _ptr(a, "a", dt, dev),
        _ptr(b, "b", dt, dev), _ptr(A_log, "A_log", torch.float32, dev),
        _ptr(dt_bias, "dt_bias", torch.float32, dev), pool.handle,
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, dev), _ptr(read_slot, "read_slot", torch.int32, dev),
        _ptr(write_slot, "write_slot", torch.int32, dev), _ptr(out, "out", dt, dev), nseq, T,
        int(bool(keep_in_place)), ws_ptr, ctypes.c_size_t(ws_bytes), _dtype_code(dt), _stream(dev)))
    return out


def gdn_verify(q, k, v, a, b, A_log, dt_bias, pool: GDNStatePool, cu_seqlens, read_slot, token_slot,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """As gdn_prefill, but the state after token t goes to token_slot[t] (a
    state a token) and the read slot is left alone."""
    T, nseq = _prefill_checks(q, k, v, a, b, A_log, dt_bias, pool, cu_seqlens, read_slot)
    dt, dev = q.dtype, pool.tensor.device
    _numel(token_slot, T, "token_slot")
    if out is None:
        out = torch.empty((T, pool.hv, pool.dv), dtype=dt, device=dev)
    _numel(out, T * pool.hv * pool.dv, "out")
    _check(_lib.load().gdn_verify(
        _ptr(q, "q", dt, dev, host_ok=True), _ptr(k, "k", dt, dev, host_ok=True), _ptr(v, "v", dt, dev, host_ok=True), _ptr(a, "a", dt, dev, host_ok=True),
        _ptr(b, "b", dt, dev, host_ok=True), _ptr(A_log, "A_log", torch.float32, dev),
        _ptr(dt_bias, "dt_bias", torch.float32, dev), pool.handle,
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, dev), _ptr(read_slot, "read_slot", torch.int32, dev),
        _ptr(token_slot, "token_slot", torch.int32, dev), _ptr(out, "out", dt, dev, host_ok=True), nseq, T,
        _dtype_code(dt), _stream(dev)))
    return out


def causal_conv1d_prefill(x, conv_pool: ConvStatePool, cu_seqlens, read_slot, w, bias, write_slot=None,
                          token_slot=None, out: Optional[torch.Tensor] = None, silu: bool = True) -> torch.Tensor:
    """The conv over many tokens a sequence: x [T][C] packed token-major; the
    window continues from read_slot and ends in write_slot (None: in place), or
    with token_slot [T] the window after each token goes to its slot."""
    T = x.shape[0]
    C = conv_pool.channels
    nseq = cu_seqlens.numel() - 1
    dt, dev = x.dtype, conv_pool.tensor.device
    _numel(x, T * C, "x")
    _numel(w, C * conv_pool.width, "w")
    if bias is not None:
        _numel(bias, C, "bias")
    _numel(read_slot, nseq, "read_slot")
    if write_slot is not None:
        _numel(write_slot, nseq, "write_slot")
    if token_slot is not None:
        _numel(token_slot, T, "token_slot")
    if out is None:
        out = torch.empty((T, C), dtype=dt, device=dev)
    _numel(out, T * C, "out")
    _check(_lib.load().causal_conv1d_prefill(
        _ptr(x, "x", dt, dev, host_ok=True), conv_pool.handle, _ptr(cu_seqlens, "cu_seqlens", torch.int32, dev),
        _ptr(read_slot, "read_slot", torch.int32, dev), _ptr(write_slot, "write_slot", torch.int32, dev),
        _ptr(token_slot, "token_slot", torch.int32, dev), _ptr(w, "w", dt, dev), _ptr(bias, "bias", dt, dev),
        int(bool(silu)), _ptr(out, "out", dt, dev, host_ok=True), nseq, T, _dtype_code(dt), _stream(dev)))
    return out


def gdn_layer_decode(x, conv_pool: ConvStatePool, w, bias, A_log, dt_bias, a, b, pool: GDNStatePool,
                     read_slot, write_slot=None, out: Optional[torch.Tensor] = None,
                     keep_in_place: bool = False, silu: bool = True, commit: bool = False) -> torch.Tensor:
    """Fused conv + gated delta rule. x: [rows][2*hk*dk + hv*dv] packed q|k|v.
    With commit (twin only) the slot tables are swapped in the same launch
    (gdn_layer_decode_commit)."""
    if commit and (keep_in_place or write_slot is None):
        raise ValueError("commit needs twin slots (a write_slot table, keep_in_place False)")
    rows = x.shape[0]
    dt = x.dtype
    dev = pool.tensor.device
    C = 2 * pool.hk * pool.dk + pool.hv * pool.dv
    _numel(x, rows * C, "x")
    _numel(w, C * conv_pool.width, "w")
    if bias is not None:
        _numel(bias, C, "bias")
    _numel(a, rows * pool.hv, "a")
    _numel(b, rows * pool.hv, "b")
    _numel(A_log, pool.hv, "A_log")
    _numel(dt_bias, pool.hv, "dt_bias")
    _numel(read_slot, rows, "read_slot")
    if write_slot is not None:
        _numel(write_slot, rows, "write_slot")
    if out is None:
        out = torch.empty((rows, pool.hv, pool.dv), dtype=dt, device=dev)
    _numel(out, rows * pool.hv * pool.dv, "out")
    args = (_ptr(x, "x", dt, dev, host_ok=True), conv_pool.handle, _ptr(w, "w", dt, dev), _ptr(bias, "bias", dt, dev),
            int(bool(silu)), _ptr(A_log, "A_log", torch.float32, dev),
            _ptr(dt_bias, "dt_bias", torch.float32, dev), _ptr(a, "a", dt, dev, host_ok=True), _ptr(b, "b", dt, dev, host_ok=True),
            pool.handle, _ptr(read_slot, "read_slot", torch.int32, dev),
            _ptr(write_slot, "write_slot", torch.int32, dev), _ptr(out, "out", dt, dev, host_ok=True), rows)
    if commit:
        _check(_lib.load().gdn_layer_decode_commit(*args, _dtype_code(dt), _stream(dev)))
    else:
        _check(_lib.load().gdn_layer_decode(*args, int(bool(keep_in_place)), _dtype_code(dt), _stream(dev)))
    return out


def gdn_layer_decode_noalloc(x, conv_pool: ConvStatePool, w, bias, A_log, dt_bias, a, b,
                             pool: GDNStatePool, read_slot, write_slot, out: torch.Tensor,
                             keep_in_place: bool = False, silu: bool = True,
                             scratch_slot: int = 0) -> torch.Tensor:
    """gdn_layer_decode with its work counters in the library's fixed scratch
    slot `scratch_slot` instead of the pool's; allocates nothing, so `out`
    is required."""
    rows = x.shape[0]
    dt = x.dtype
    dev = pool.tensor.device
    C = 2 * pool.hk * pool.dk + pool.hv * pool.dv
    _numel(x, rows * C, "x")
    _numel(w, C * conv_pool.width, "w")
    if bias is not None:
        _numel(bias, C, "bias")
    _numel(a, rows * pool.hv, "a")
    _numel(b, rows * pool.hv, "b")
    _numel(A_log, pool.hv, "A_log")
    _numel(dt_bias, pool.hv, "dt_bias")
    _numel(read_slot, rows, "read_slot")
    if write_slot is not None:
        _numel(write_slot, rows, "write_slot")
    _numel(out, rows * pool.hv * pool.dv, "out")
    _check(_lib.load().gdn_layer_decode_noalloc(
        _ptr(x, "x", dt, dev, host_ok=True), conv_pool.handle, _ptr(w, "w", dt, dev), _ptr(bias, "bias", dt, dev),
        int(bool(silu)), _ptr(A_log, "A_log", torch.float32, dev),
        _ptr(dt_bias, "dt_bias", torch.float32, dev), _ptr(a, "a", dt, dev, host_ok=True), _ptr(b, "b", dt, dev, host_ok=True),
        pool.handle, _ptr(read_slot, "read_slot", torch.int32, dev),
        _ptr(write_slot, "write_slot", torch.int32, dev), _ptr(out, "out", dt, dev, host_ok=True), rows,
        int(bool(keep_in_place)), int(scratch_slot), _dtype_code(dt), _stream(dev)))
    return out


def gdn_layer_decode_bucket(x, conv_pool: ConvStatePool, w, bias, A_log, dt_bias, a, b, pool: GDNStatePool,
                            read_slot, write_slot, n_decode: torch.Tensor, out: Optional[torch.Tensor] = None,
                            keep_in_place: bool = False, commit: bool = False,
                            silu: bool = True) -> torch.Tensor:
    """The decode half of a mixed step: the launch covers the bucket (x's rows);
    only rows below the device int32 n_decode are decoded, the rest are left
    alone (outputs zero).  With commit (twin only) the decoded rows' tables are
    swapped in the same launch."""
    if commit and (keep_in_place or write_slot is None):
        raise ValueError("commit needs twin slots (a write_slot table, keep_in_place False)")
    rows = x.shape[0]
    dt = x.dtype
    dev = pool.tensor.device
    C = 2 * pool.hk * pool.dk + pool.hv * pool.dv
    _numel(x, rows * C, "x")
    _numel(w, C * conv_pool.width, "w")
    if bias is not None:
        _numel(bias, C, "bias")
    for tname, tt, n in (("a", a, rows * pool.hv), ("b", b, rows * pool.hv), ("A_log", A_log, pool.hv),
                         ("dt_bias", dt_bias, pool.hv), ("read_slot", read_slot, rows), ("n_decode", n_decode, 1)):
        _numel(tt, n, tname)
    if write_slot is not None:
        _numel(write_slot, rows, "write_slot")
    if out is None:
        out = torch.empty((rows, pool.hv, pool.dv), dtype=dt, device=dev)
    _numel(out, rows * pool.hv * pool.dv, "out")
    _check(_lib.load().gdn_layer_decode_bucket(
        _ptr(x, "x", dt, dev, host_ok=True), conv_pool.handle, _ptr(w, "w", dt, dev), _ptr(bias, "bias", dt, dev),
        int(bool(silu)), _ptr(A_log, "A_log", torch.float32, dev),
        _ptr(dt_bias, "dt_bias", torch.float32, dev), _ptr(a, "a", dt, dev, host_ok=True), _ptr(b, "b", dt, dev, host_ok=True),
        pool.handle, _ptr(read_slot, "read_slot", torch.int32, dev),
        _ptr(write_slot, "write_slot", torch.int32, dev), _ptr(out, "out", dt, dev, host_ok=True), rows,
        _ptr(n_decode, "n_decode", torch.int32, dev), int(bool(keep_in_place)), int(bool(commit)),
        _dtype_code(dt), _stream(dev)))
    return out


def gdn_commit(read_slot: torch.Tensor, write_slot: torch.Tensor) -> None:
    """Swap the read and write slot tables on the device (twin-slot commit)."""
    n = read_slot.numel()
    _numel(write_slot, n, "write_slot")
    dev = read_slot.device
    _check(_lib.load().gdn_commit(_ptr(read_slot, "read_slot", torch.int32, dev),
                                  _ptr(write_slot, "write_slot", torch.int32, dev), n, _stream(dev)))


def gdn_validate_slots(read_slot: torch.Tensor, write_slot: Optional[torch.Tensor], num_slots: int,
                       keep_in_place: bool = False) -> None:
    """Debug check of the slot tables (synchronises). Raises GDNError on a violation."""
    dev = read_slot.device
    _check(_lib.load().gdn_validate_slots(_ptr(read_slot, "read_slot", torch.int32, dev),
                                          _ptr(write_slot, "write_slot", torch.int32, dev),
                                          read_slot.numel(), num_slots, int(bool(keep_in_place)),
                                          _stream(dev)))


def get_device_error(device=None) -> int:
    """Read and clear the sticky device error word of `device` (synchronises)."""
    device = torch.device(device if device is not None else "cuda")
    code = ctypes.c_int(0)
    with torch.cuda.device(device):
        _check(_lib.load().gdn_get_device_error(ctypes.byref(code), _stream(device)))
    return code.value


def selftest_wait_timeout(limit_us: int = 1000, device=None) -> None:
    """Run a kernel whose bounded wait cannot end (it gives up after
    `limit_us` microseconds); afterwards the device error word reads
    GDN_DEVERR_TIMEOUT.  Asynchronous."""
    device = torch.device(device if device is not None else "cuda")
    with torch.cuda.device(device):
        _check(_lib.load().gdn_selftest_wait_timeout(int(limit_us), _stream(device)))


def probe_traffic(pool: GDNStatePool, read_slot: torch.Tensor, write_slot: Optional[torch.Tensor],
                  mode: int, sink: Optional[torch.Tensor] = None) -> None:
    """Move a step's state bytes with no arithmetic (roofline probe)."""
    dev = read_slot.device
    _check(_lib.load().gdn_probe_traffic(pool.handle, _ptr(read_slot, "read_slot", torch.int32, dev),
                                         _ptr(write_slot, "write_slot", torch.int32, dev),
                                         read_slot.numel(), mode,
                                         _ptr(sink, "sink", torch.float32, dev), _stream(dev)))


class PreparedCall:
    """A validated C-ABI call with its pointer arguments bound once.

    Calling it launches the same entry point again on the same buffers and
    stream, without re-marshalling the tensors: a decode loop (or a graph
    capture) then costs one ctypes call per launch.  The tensors must stay
    alive and keep their addresses while the call is used.
    """

    def __init__(self, fn_name: str, args: tuple, keep: tuple):
        self._fn = getattr(_lib.load(), fn_name)
        self._args = args
        self._keep = keep  # hold references to the tensors whose pointers are bound

    def __call__(self) -> None:
        rc = self._fn(*self._args)
        if rc:
            _check(rc)


def prepare_layer_decode(x, conv_pool: ConvStatePool, w, bias, A_log, dt_bias, a, b, pool: GDNStatePool,
                         read_slot, write_slot, out, keep_in_place: bool = False, silu: bool = True,
                         stream: Optional[torch.cuda.Stream] = None, commit: bool = False) -> PreparedCall:
    """gdn_layer_decode (or, with commit, gdn_layer_decode_commit) bound to
    fixed buffers (validated here, once)."""
    if commit and (keep_in_place or write_slot is None):
        raise ValueError("commit needs twin slots (a write_slot table, keep_in_place False)")
    rows = x.shape[0]
    dt = x.dtype
    dev = pool.tensor.device
    C = 2 * pool.hk * pool.dk + pool.hv * pool.dv
    _numel(x, rows * C, "x")
    _numel(w, C * conv_pool.width, "w")
    if bias is not None:
        _numel(bias, C, "bias")
    for tname, tt, n in (("a", a, rows * pool.hv), ("b", b, rows * pool.hv), ("A_log", A_log, pool.hv),
                         ("dt_bias", dt_bias, pool.hv), ("read_slot", read_slot, rows),
                         ("out", out, rows * pool.hv * pool.dv)):
        _numel(tt, n, tname)
    if write_slot is not None:
        _numel(write_slot, rows, "write_slot")
    s = (stream or torch.cuda.current_stream(dev)).cuda_stream
    args = (_ptr(x, "x", dt, dev, host_ok=True), conv_pool.handle, _ptr(w, "w", dt, dev), _ptr(bias, "bias", dt, dev),
            int(bool(silu)), _ptr(A_log, "A_log", torch.float32, dev),
            _ptr(dt_bias, "dt_bias", torch.float32, dev), _ptr(a, "a", dt, dev, host_ok=True), _ptr(b, "b", dt, dev, host_ok=True),
            pool.handle, _ptr(read_slot, "read_slot", torch.int32, dev),
            _ptr(write_slot, "write_slot", torch.int32, dev), _ptr(out, "out", dt, dev, host_ok=True), rows)
    if commit:
        args += (_dtype_code(dt), s)
    else:
        args += (int(bool(keep_in_place)), _dtype_code(dt), s)
    return PreparedCall("gdn_layer_decode_commit" if commit else "gdn_layer_decode", args,
                        (x, conv_pool, w, bias, A_log, dt_bias, a, b, pool, read_slot, write_slot, out))


def prepare_commit(read_slot: torch.Tensor, write_slot: torch.Tensor,
                   stream: Optional[torch.cuda.Stream] = None) -> PreparedCall:
    """gdn_commit bound to fixed slot tables."""
    n = read_slot.numel()
    _numel(write_slot, n, "write_slot")
    dev = read_slot.device
    s = (stream or torch.cuda.current_stream(dev)).cuda_stream
    args = (_ptr(read_slot, "read_slot", torch.int32, dev), _ptr(write_slot, "write_slot", torch.int32, dev),
            n, s)
    return PreparedCall("gdn_commit", args, (read_slot, write_slot))


__all__ += ["PreparedCall", "prepare_layer_decode", "prepare_commit"]


# ---- attention layers over a paged cache ------------------------------------


def rope_inv_freq(rot: int, base: float = 10000.0, scaling: Optional[dict] = None):
    """(inverse frequencies [rot/2] as float64 on the CPU, mscale) of rotary positions.

    scaling, for contexts longer than the model was trained on, is None or one of
      {"type": "linear", "factor": f}    position interpolation: every frequency over f
      {"type": "ntk", "factor": f}       base * f^(rot / (rot - 2)): the lowest frequency over f, the highest kept
      {"type": "yarn", "factor": f, "original": n, "fast": 32, "slow": 1, "mscale": m}
                                         frequencies that turn more than `fast` times in the n positions of training are
                                         kept, those that turn less than `slow` times are taken over f, with a linear
                                         ramp over the dimensions between; mscale (default 0.1 ln f + 1) scales the table
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and positive, got {rot}")
    i = torch.arange(rot // 2, dtype=torch.float64)
    kind = scaling.get("type") if scaling else None
    f = float(scaling["factor"]) if scaling else 1.0
    if f <= 0:
        raise ValueError("the scaling factor must be positive")
    if kind == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2))
    freq = float(base) ** (-2.0 * i / rot)
    if kind in (None, "ntk"):
        return freq, 1.0
    if kind == "linear":
        return freq / f, 1.0
    if kind != "yarn":
        raise ValueError(f"unknown rotary scaling {kind!r}")
    n = float(scaling["original"])

    def dim(turns):  # the (real) index of the frequency that turns so often in n positions
        return rot * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo = max(math.floor(dim(scaling.get("fast", 32))), 0)
    hi = min(math.ceil(dim(scaling.get("slow", 1))), rot - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    mscale = scaling.get("mscale")
    if mscale is None:
        mscale = 0.1 * math.log(f) + 1.0 if f > 1 else 1.0
    return freq / f * ramp + freq * (1 - ramp), float(mscale)


def rope_table(rot: int, positions: int, base: float = 10000.0, scaling: Optional[dict] = None, device=None) -> torch.Tensor:
    """The rotation table [positions][rot] fp32 (cosines, then sines) that attn_prologue reads; made once for a model."""
    device = torch.device(device if device is not None else "cuda")
    freq, mscale = rope_inv_freq(rot, base, scaling)
    freq = freq.to(device)
    table = torch.empty((positions, rot), dtype=torch.float32, device=device)
    with torch.cuda.device(device):
        _check(_lib.load().rope_table(_ptr(freq, "inv_freq"), rot, positions, mscale, _ptr(table, "table"),
                                      _stream(device)))
    return table


class KVPagePool:
    """K and V of attention layers, each [layers][num_pages][hkv][page_size][d], in torch-owned memory (`k`, `v`).

    Page 0 is the null page.  The library wraps the tensors (it never frees them)."""

    def __init__(self, num_pages: int, page_size: int, hkv: int, d: int, layers: int = 1, dtype=torch.bfloat16,
                 device=None, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
        L = _lib.load()
        shape = (layers, num_pages, hkv, page_size, d)
        if (k is None) != (v is None):
            raise ValueError("give both k and v, or neither")
        if k is None:
            device = torch.device(device if device is not None else "cuda")
            k = torch.zeros(shape, dtype=dtype, device=device)
            v = torch.zeros(shape, dtype=dtype, device=device)
        if tuple(k.shape) != shape or tuple(v.shape) != shape or k.dtype != dtype or v.dtype != dtype:
            raise ValueError("k and v must be [layers][num_pages][hkv][page_size][d] of the given dtype")
        self.k, self.v, self.device = k, v, k.device
        self.num_pages, self.page_size, self.hkv, self.d = num_pages, page_size, hkv, d
        self.layers, self.dtype, self._code = layers, dtype, _dtype_code(dtype)
        h = ctypes.c_void_p()
        _check(L.kv_page_pool_wrap(_ptr(k, "k"), _ptr(v, "v", None, k.device), num_pages, page_size, layers, hkv, d,
                                   self._code, ctypes.byref(h)))
        self._h = h
        self._fast = _lib.fast()  # the C++ binding and the pool as it takes it
        self._p = self._fast.make_pool(h.value, hkv, d, self._code, self.device.index) if self._fast else None

    @property
    def handle(self):
        return self._h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            try:
                if self._p:
                    self._fast.drop_pool(self._p)
                _lib.load().kv_page_pool_destroy(h)
            except Exception:
                pass
            self._h = self._p = None


class KVPageMoves:
    """Pages to copy, as kv_pages_fork and kv_pages_compact list them on the device: src[j] -> dst[j] for j < count[0]
    (zeros past it, up to the call's forks or pages).  `n` is the capacity: the most forks of a call, or the pool's pages.
    `status` is 0 for every fork of the last call that was done; a compaction uses its room."""

    def __init__(self, n: int, device=None):
        device = torch.device(device if device is not None else "cuda")
        self.src = torch.zeros(n, dtype=torch.int32, device=device)
        self.dst = torch.zeros(n, dtype=torch.int32, device=device)
        self.count = torch.zeros(1, dtype=torch.int32, device=device)
        self.status = torch.zeros(n, dtype=torch.int32, device=device)

    def _pointers(self, n: int, dev: torch.device):
        """Device pointers of the lists, of at least n entries, and of the count."""
        i32, room = torch.int32, min(self.src.numel(), self.dst.numel(), self.status.numel())
        if room < n:
            raise ValueError(f"moves has room for {room} entries, {n} are needed")
        return (_arg(self.src, self.src.numel(), i32, dev, "moves"), _arg(self.dst, self.dst.numel(), i32, dev, "moves"),
                _arg(self.count, 1, i32, dev, "moves"))


# A decode step makes a few of these calls a layer, each of some microseconds on the GPU.  The C++ binding makes those
# that are in order; the helpers below, for the others and where it was not built, look at a tensor once, and only then at
# what is wrong with it.


def _made(r):
    """What the C++ binding returned, with a status raised as an error."""
    if type(r) is int:
        _check(r)
    return r


def _raw_stream(dev: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _on(dev: torch.device, call, *args):
    """call(*args, dev's stream) with dev as the current device: a stream's handle need not name its device, as 0,
    PyTorch's default stream, is the current device's."""
    if torch.cuda.current_device() == dev.index:
        _check(call(*args, _raw_stream(dev)))
    else:
        with torch.cuda.device(dev):
            _check(call(*args, _raw_stream(dev)))


def _arg(t: Optional[torch.Tensor], n: int, dtype, dev: torch.device, what: str):
    """Device pointer of a contiguous tensor of n elements (or None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.device == dev and t.is_contiguous() and t.numel() == n:
        return t.data_ptr()
    _numel(t, n, what)
    return _ptr(t, what, dtype, dev)


def _token_rows(x: torch.Tensor, tokens: int, heads: int, pool: KVPagePool, what: str):
    """Device pointer and token stride of x [tokens][heads][d], whose tokens may be apart but whose heads are dense."""
    shape, st = x.shape, x.stride()
    if len(shape) != 3 or shape[0] != tokens or shape[1] != heads or shape[2] != pool.d:
        raise ValueError(f"{what} must be [{tokens}][{heads}][{pool.d}], got {tuple(shape)}")
    if st[2] != 1 or (st[1] != pool.d and heads > 1):
        raise ValueError(f"{what}: the heads of a token must be dense")
    if x.dtype is not pool.dtype or x.device != pool.device:
        _ptr(x, what, pool.dtype, pool.device, False)
    return x.data_ptr(), st[0] if tokens > 1 else heads * pool.d


def _table(table: torch.Tensor, dev: torch.device, what: str = "table"):
    """Device pointer, rows and width of a page table."""
    shape = table.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be [rows][max_pages]")
    return _arg(table, shape[0] * shape[1], torch.int32, dev, what), shape[0], shape[1]


def attn_prologue(q, k, v, pool: KVPagePool, rope: Optional[torch.Tensor], table, seq_len, cu_seqlens, layer: int = 0,
                  q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  interleaved: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """RMS norm (optional) and rotary positions of q and k, and the append of k and v to the pages of each token's row.

    q [T][hq][d], k, v [T][hkv][d] (views of a packed projection are fine); row r's tokens are cu_seqlens[r] ..
    cu_seqlens[r+1], and seq_len[r] counts them already.  rope is a table of rope_table (its width says how much of a
    head is rotated) or None.  Returns the rotated q, [T][hq][d]."""
    if pool._p:
        r = pool._fast.attn_prologue(q, k, v, pool._p, rope, table, seq_len, cu_seqlens, layer, q_norm, k_norm, eps,
                                     interleaved, out)
        if r is not None:
            return _made(r)
    dev, d, hkv, i32, f32 = pool.device, pool.d, pool.hkv, torch.int32, torch.float32
    T, hq = q.shape[:2]
    tab, rows, max_pages = _table(table, dev)
    qp, qs = _token_rows(q, T, hq, pool, "q")
    kp, ks = _token_rows(k, T, hkv, pool, "k")
    vp, vs = _token_rows(v, T, hkv, pool, "v")
    positions = rot = 0
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError("rope must be [positions][rot]")
        positions, rot = rope.shape
    if out is None:
        out = torch.empty((T, hq, d), dtype=pool.dtype, device=dev)
        op = out.data_ptr()
    else:
        op = _arg(out, T * hq * d, pool.dtype, dev, "out")
    _on(dev, _lib.load().attn_prologue,
        qp, qs, kp, ks, vp, vs, pool._h, layer, _arg(rope, positions * rot, f32, dev, "rope"), positions, rot,
        1 if interleaved else 0, _arg(q_norm, d, f32, dev, "q_norm"), _arg(k_norm, d, f32, dev, "k_norm"), eps, tab,
        max_pages, _arg(seq_len, rows, i32, dev, "seq_len"), _arg(cu_seqlens, rows + 1, i32, dev, "cu_seqlens"),
        op, hq, rows, T, pool._code)
    return out


def paged_attention_workspace_bytes(pool: KVPagePool, hq: int, rows: int, total_tokens: int) -> int:
    """Bytes of the device workspace of paged_attention."""
    return int(_lib.load().paged_attention_workspace_bytes(pool._h, int(hq), int(rows), int(total_tokens)))


def paged_attention(q, pool: KVPagePool, table, seq_len, cu_seqlens, layer: int = 0, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of new tokens (q [T][hq][d], rotated) over their rows' pages, the tokens' own keys included.

    scale defaults to d^-1/2.  workspace is a uint8 tensor of paged_attention_workspace_bytes (allocated here when none
    is given).  Returns [T][hq][d]."""
    if scale is None:
        scale = pool.d ** -0.5
    if pool._p:
        r = pool._fast.paged_attention(q, pool._p, table, seq_len, cu_seqlens, layer, scale, out, workspace)
        if r is not None:
            return _made(r)
    dev, d, i32 = pool.device, pool.d, torch.int32
    T, hq = q.shape[:2]
    tab, rows, max_pages = _table(table, dev)
    qp, qs = _token_rows(q, T, hq, pool, "q")
    if out is None:
        out = torch.empty((T, hq, d), dtype=pool.dtype, device=dev)
        op = out.data_ptr()
    else:
        op = _arg(out, T * hq * d, pool.dtype, dev, "out")
    L = _lib.load()
    if workspace is None:
        nbytes = L.paged_attention_workspace_bytes(pool._h, hq, rows, T)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp, nbytes = _ptr(workspace, "workspace", None, dev), workspace.numel() * workspace.element_size()
    _on(dev, L.paged_attention,
        qp, qs, pool._h, layer, tab, max_pages, _arg(seq_len, rows, i32, dev, "seq_len"),
        _arg(cu_seqlens, rows + 1, i32, dev, "cu_seqlens"), scale,
        op, hq, rows, T, wp, nbytes, pool._code)
    return out


def kv_pages_shared(table, seq_len, cu_seqlens, bounds, page_size: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """What the rows of each group share, for paged_attention_shared: group g is rows bounds[g] .. bounds[g+1].  Returns
    [rows][2] int32: the group's first live row, and the leading pages that all live rows of the group have alike, before
    their new tokens."""
    f = _lib.fast()
    if f:
        r = f.kv_pages_shared(table, seq_len, cu_seqlens, bounds, page_size, out)
        if r is not None:
            return _made(r)
    dev, i32 = table.device, torch.int32
    tab, rows, max_pages = _table(table, dev)
    if out is None:
        out = torch.empty((rows, 2), dtype=i32, device=dev)
    _on(dev, _lib.load().kv_pages_shared,
        tab, rows, max_pages, _arg(seq_len, rows, i32, dev, "seq_len"), _arg(cu_seqlens, rows + 1, i32, dev, "cu_seqlens"),
        _arg(bounds, bounds.numel(), i32, dev, "bounds"), bounds.numel() - 1, page_size, _arg(out, 2 * rows, i32, dev, "out"))
    return out


def paged_attention_shared_workspace_bytes(pool: KVPagePool, hq: int, rows: int, total_tokens: int) -> int:
    """Bytes of the device workspace of paged_attention_shared."""
    return int(_lib.load().paged_attention_shared_workspace_bytes(pool._h, int(hq), int(rows), int(total_tokens)))


def paged_attention_shared(q, pool: KVPagePool, table, seq_len, cu_seqlens, bounds, prefix, layer: int = 0,
                           scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_attention with the pages that a group's rows share read once for all of them, for rows that were forked.

    It pays from about 512 shared tokens on in bf16 and 2,000 in fp32, with eight rows a group or more; elsewhere
    paged_attention takes up to 4 us less a call (fp32: up to 10).

    bounds [groups + 1] and prefix [rows][2] are kv_pages_shared's (which a step calls once, for all of its layers)."""
    if scale is None:
        scale = pool.d ** -0.5
    if pool._p:
        r = pool._fast.paged_attention_shared(q, pool._p, table, seq_len, cu_seqlens, layer, scale, out, workspace, bounds, prefix)
        if r is not None:
            return _made(r)
    dev, d, i32 = pool.device, pool.d, torch.int32
    T, hq = q.shape[:2]
    tab, rows, max_pages = _table(table, dev)
    qp, qs = _token_rows(q, T, hq, pool, "q")
    if out is None:
        out = torch.empty((T, hq, d), dtype=pool.dtype, device=dev)
        op = out.data_ptr()
    else:
        op = _arg(out, T * hq * d, pool.dtype, dev, "out")
    L = _lib.load()
    if workspace is None:
        nbytes = L.paged_attention_shared_workspace_bytes(pool._h, hq, rows, T)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp, nbytes = _ptr(workspace, "workspace", None, dev), workspace.numel() * workspace.element_size()
    _on(dev, L.paged_attention_shared,
        qp, qs, pool._h, layer, tab, max_pages, _arg(seq_len, rows, i32, dev, "seq_len"),
        _arg(cu_seqlens, rows + 1, i32, dev, "cu_seqlens"), _arg(bounds, bounds.numel(), i32, dev, "bounds"), bounds.numel() - 1,
        _arg(prefix, 2 * rows, i32, dev, "prefix"), scale, op, hq, rows, T, wp, nbytes, pool._code)
    return out


def kv_pages_reserve(table, refs, rows, tokens, page_size: int, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Give row rows[i] of the table the pages for tokens[i] tokens in all.  Returns status (0 where done)."""
    dev, n, i32 = table.device, rows.numel(), torch.int32
    tab, trows, max_pages = _table(table, dev)
    if status is None:
        status = torch.empty(n, dtype=i32, device=dev)
    pages = refs.numel()
    _on(dev, _lib.load().kv_pages_reserve,
        tab, trows, max_pages, _arg(refs, pages, i32, dev, "refs"), pages, page_size, _arg(rows, n, i32, dev, "rows"),
        _arg(tokens, n, i32, dev, "tokens"), n, _arg(status, n, i32, dev, "status"))
    return status


def kv_pages_fork(table, seq_len, refs, src_rows, dst_rows, page_size: int, moves: KVPageMoves) -> KVPageMoves:
    """Make the empty rows dst_rows copies of src_rows: full pages are shared, partial last pages get a free page each,
    whose copies are listed in `moves` (then kv_pages_copy(pool, moves))."""
    f = _lib.fast()
    if f:
        r = f.kv_pages_fork(table, seq_len, refs, src_rows, dst_rows, page_size, moves.src, moves.dst, moves.count,
                            moves.status)
        if r is not None:
            _made(r)
            return moves
    dev, n, i32 = table.device, src_rows.numel(), torch.int32
    tab, trows, max_pages = _table(table, dev)
    pages = refs.numel()
    _on(dev, _lib.load().kv_pages_fork,
        tab, trows, max_pages, _arg(seq_len, trows, i32, dev, "seq_len"), _arg(refs, pages, i32, dev, "refs"), pages,
        page_size, _arg(src_rows, n, i32, dev, "src_rows"), _arg(dst_rows, n, i32, dev, "dst_rows"), n,
        *moves._pointers(n, dev), _arg(moves.status, moves.status.numel(), i32, dev, "moves"))
    return moves


def kv_pages_free(table, seq_len, refs, rows) -> None:
    """Give up the pages of the listed rows and set their lengths to 0."""
    f = _lib.fast()
    if f:
        r = f.kv_pages_free(table, seq_len, refs, rows)
        if r is not None:
            _made(r)
            return
    dev, n, i32 = table.device, rows.numel(), torch.int32
    tab, trows, max_pages = _table(table, dev)
    pages = refs.numel()
    _on(dev, _lib.load().kv_pages_free,
        tab, trows, max_pages, _arg(seq_len, trows, i32, dev, "seq_len"), _arg(refs, pages, i32, dev, "refs"), pages,
        _arg(rows, n, i32, dev, "rows"), n)


def kv_pages_compact(table, refs, moves: KVPageMoves, table_out: Optional[torch.Tensor] = None,
                     refs_out: Optional[torch.Tensor] = None, remap: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Renumber the pages in use to the lowest numbers, in place or into table_out and refs_out; the copies are listed
    in `moves` (with room for the pool's pages), then kv_pages_copy(pool, moves).  Returns remap: each page's
    new number, 0 for a free page."""
    dev, i32, n = table.device, torch.int32, refs.numel()
    tab, trows, max_pages = _table(table, dev)
    remap = torch.empty(n, dtype=i32, device=dev) if remap is None else remap
    refp = _arg(refs, n, i32, dev, "refs")
    _on(dev, _lib.load().kv_pages_compact,
        tab, trows, max_pages, refp, n,
        tab if table_out is None else _arg(table_out, trows * max_pages, i32, dev, "table_out"),
        refp if refs_out is None else _arg(refs_out, n, i32, dev, "refs_out"), _arg(remap, n, i32, dev, "remap"),
        *moves._pointers(n, dev), _arg(moves.status, moves.status.numel(), i32, dev, "moves"))
    return remap


def kv_pages_copy(pool: KVPagePool, moves: KVPageMoves) -> None:
    """Copy the listed pages, K and V of all layers."""
    if pool._p:
        r = pool._fast.kv_pages_copy(pool._p, moves.src, moves.dst, moves.count)
        if r is not None:
            _made(r)
            return
    dev, n = pool.device, moves.src.numel()
    src, dst, count = moves._pointers(n, dev)
    _on(dev, _lib.load().kv_pages_copy, pool._h, src, dst, n, count)


__all__ += ["rope_inv_freq", "rope_table", "KVPagePool", "KVPageMoves", "attn_prologue",
            "paged_attention", "paged_attention_workspace_bytes", "kv_pages_reserve", "kv_pages_fork", "kv_pages_free",
            "kv_pages_compact", "kv_pages_copy", "kv_pages_shared", "paged_attention_shared",
            "paged_attention_shared_workspace_bytes", "GDN_DEVERR_BAD_PAGE", "GDN_DEVERR_NO_PAGES"]


# ---- linear attention with a decay for each head -----------------------------


def _linear_args(q, k, v, log_decay, pool: GDNStatePool, out):
    """What both forms check alike: the C ABI's arguments up to the pool's handle, the output and its pointer."""
    dev, dt = pool.tensor.device, q.dtype
    _dtype_code(dt)
    T = q.shape[0]
    if T > 0x7FFFFFFF:
        raise ValueError(f"{T} tokens are more than a call takes")

    def rows(x, heads, d, what):
        shape, st = x.shape, x.stride()
        if len(shape) != 3 or shape[0] != T or shape[1] != heads or shape[2] != d:
            raise ValueError(f"{what} must be [{T}][{heads}][{d}], got {tuple(shape)}")
        if T and ((st[2] != 1 and d > 1) or (st[1] != d and heads > 1)):
            raise ValueError(f"{what}: the heads of a token must be dense")
        return _ptr(x, what, dt, dev, False), st[0] if T > 1 else heads * d

    args = (*rows(q, pool.hk, pool.dk, "q"), *rows(k, pool.hk, pool.dk, "k"), *rows(v, pool.hv, pool.dv, "v"))
    if log_decay.dim() not in (1, 2):
        raise ValueError("log_decay must be [hv] or [tokens][hv]")
    per_token = log_decay.dim() == 2
    decay = _arg(log_decay, pool.hv * (T if per_token else 1), torch.float32, dev, "log_decay")
    if out is None:
        out = torch.empty((T, pool.hv, pool.dv), dtype=dt, device=dev)
        op = out.data_ptr()
    else:
        op = _arg(out, T * pool.hv * pool.dv, dt, dev, "out")
    return (*args, decay, 1 if per_token else 0, pool.handle), out, op


def _slots(read_slot, write_slot, rows: int, dev, keep_in_place: bool):
    i32 = torch.int32
    return (_arg(read_slot, rows, i32, dev, "read_slot"),
            None if keep_in_place else _arg(write_slot, rows, i32, dev, "write_slot"))


def linear_attention_decode(q, k, v, log_decay, pool: GDNStatePool, read_slot, write_slot=None,
                            scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                            keep_in_place: bool = False) -> torch.Tensor:
    """Linear attention with a decay for each head, one token a row: S' = exp(g) S + v k^T, o = scale S' q.

    q, k [rows][hk][dk], v [rows][hv][dv] (views of a packed projection are fine); log_decay g is fp32, [hv] or
    [rows][hv], at most 0 (what is above counts as 0).  The state goes from read_slot to write_slot (twin) or stays in
    read_slot (keep_in_place).  scale defaults to dk^-1/2.  Returns o, [rows][hv][dv]."""
    if scale is None:
        scale = pool.dk ** -0.5
    if pool._p:
        r = pool._fast.linear_decode(q, k, v, log_decay, pool._p, read_slot, None if keep_in_place else write_slot, scale,
                                     out, keep_in_place)
        if r is not None:
            return _made(r)
    args, out, op = _linear_args(q, k, v, log_decay, pool, out)
    rows, dev = q.shape[0], pool.tensor.device
    _on(dev, _lib.load().linear_attention_decode, *args, *_slots(read_slot, write_slot, rows, dev, keep_in_place), scale, op,
        rows, int(bool(keep_in_place)), _dtype_code(q.dtype))
    return out


def linear_attention_prefill_workspace_bytes(pool: GDNStatePool, nseq: int, total_tokens: int, dtype=torch.bfloat16) -> int:
    """Bytes of the device workspace of linear_attention_prefill."""
    return int(_lib.load().linear_attention_prefill_workspace_bytes(pool.handle, int(nseq), int(total_tokens),
                                                                    _dtype_code(dtype)))


def linear_attention_prefill(q, k, v, log_decay, pool: GDNStatePool, cu_seqlens, read_slot, write_slot=None,
                             scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                             keep_in_place: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """linear_attention_decode's rule over packed sequences: sequence r is tokens cu_seqlens[r] .. cu_seqlens[r+1] of q, k
    [T][hk][dk], v [T][hv][dv] and, where it is a number a token, log_decay [T][hv].

    workspace is a uint8 tensor of linear_attention_prefill_workspace_bytes (allocated here when none is given).  Tokens
    of no sequence are left alone.  Returns [T][hv][dv]."""
    if scale is None:
        scale = pool.dk ** -0.5
    if pool._p:
        r = pool._fast.linear_prefill(q, k, v, log_decay, pool._p, cu_seqlens, read_slot,
                                      None if keep_in_place else write_slot, scale, out, keep_in_place, workspace)
        if r is not None:
            return _made(r)
    args, out, op = _linear_args(q, k, v, log_decay, pool, out)
    T, nseq, dev, code = q.shape[0], cu_seqlens.numel() - 1, pool.tensor.device, _dtype_code(q.dtype)
    if nseq < 0:
        raise ValueError("cu_seqlens needs nseq + 1 entries")
    L = _lib.load()
    if workspace is None:
        nbytes = L.linear_attention_prefill_workspace_bytes(pool.handle, nseq, T, code)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp, nbytes = _ptr(workspace, "workspace", None, dev), workspace.numel() * workspace.element_size()
    _on(dev, L.linear_attention_prefill, *args, _arg(cu_seqlens, nseq + 1, torch.int32, dev, "cu_seqlens"),
        *_slots(read_slot, write_slot, nseq, dev, keep_in_place), scale, op, nseq, T, int(bool(keep_in_place)), wp, nbytes, code)
    return out


__all__ += ["linear_attention_decode", "linear_attention_prefill", "linear_attention_prefill_workspace_bytes"]
