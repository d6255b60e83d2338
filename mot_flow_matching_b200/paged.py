"""Python binding of the paged prefix-KV cache (include/mot_paged.h):
argument marshalling only; norm, rotation, quantisation, copies and attention
run in libmotattn.so.

    paged = MotPaged({"q_norm": .., "k_norm": ..}, page_size=64, kv_dtype="e4m3", ...)
    pool = paged.new_pool(n_pages)            # one layer's pages
    batch = paged.new_batch()
    batch.set(q_len, kv_len, table, n_pages)  # host lists; once per step, for all layers
    q = paged.append(batch, qkv, pool)        # norm, rotate, cache the chunk
    o = paged.attend(batch, q, pool)          # attention of the chunk over the pages
    paged.store(batch, k, v, pool)            # dense cache -> pages
    k, v = paged.load(batch, pool)            # pages -> dense cache
"""
from __future__ import annotations

from contextlib import nullcontext
from ctypes import byref, c_size_t, c_void_p
from typing import Dict, Optional, Sequence

import torch

from ._abi import MotPagedConfig, MotPagedPoolC, MotPagedWeights, check, lib
from .layer import _BF16, _F32, _dptr, _stream

KV_DTYPES = {"bf16": 0, "e4m3": 1}

_raw_stream = torch._C._cuda_getCurrentRawStream


def mot_paged_create(cfg: MotPagedConfig, weights: Dict[str, torch.Tensor], stream=None) -> c_void_p:
    for n in ("q_norm", "k_norm"):
        t = weights[n]
        if t.shape != (128,):
            raise ValueError(f"{n} must be [128] (got {list(t.shape)})")
        if t.is_cuda and t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{n} must be on the current device, {torch.cuda.current_device()} (got {t.device})")
    w = MotPagedWeights(*[_dptr(weights[n], _BF16, n) for n in ("q_norm", "k_norm")])
    h = c_void_p()
    check(lib().mot_paged_create(byref(cfg), byref(w), _stream(stream), byref(h)), "mot_paged_create")
    return h


def _external(stream) -> torch.cuda.Stream:
    return torch.cuda.ExternalStream(_stream(stream).value or 0)


def _on_stream(stream):
    """Memory allocated under it may be reused once work of `stream` is done (None: the current stream)."""
    return nullcontext() if stream is None else torch.cuda.stream(_external(stream))


def _host_i32(v, name: str) -> Optional[torch.Tensor]:
    if v is None:
        return None
    t = torch.as_tensor(v)
    if t.is_cuda:
        raise ValueError(f"{name} must be host memory (got {t.device})")
    if t.dtype != torch.int32 and t.numel():
        if t.is_floating_point() or t.is_complex():
            raise ValueError(f"{name} must be integers (got {t.dtype})")
        t = t.to(torch.int64)
        if int(t.min()) < -2 ** 31 or int(t.max()) >= 2 ** 31:
            raise ValueError(f"{name} must fit in 32 bits (got {int(t.min())} to {int(t.max())})")
    return t.to(torch.int32).contiguous()


def mot_paged_batch_set(bt, q_len, kv_len, table, n_pages: int, visible=None, stream=None) -> None:
    """q_len, kv_len, visible: host integers per sequence; table: host int32
    [batch, width] of page numbers."""
    q, kv, vis = _host_i32(q_len, "q_len"), _host_i32(kv_len, "kv_len"), _host_i32(visible, "visible")
    tab = _host_i32(table, "table")
    n = q.numel()
    if q.dim() != 1 or kv.shape != q.shape or (vis is not None and vis.shape != q.shape):
        raise ValueError("q_len, kv_len and visible must be one integer per sequence")
    if tab.dim() != 2 or tab.shape[0] != n:
        raise ValueError(f"table must be [{n}, width] (got {list(tab.shape)})")
    check(lib().mot_paged_batch_set(bt, n, q.data_ptr(), kv.data_ptr(), vis.data_ptr() if vis is not None else None,
                                    tab.data_ptr() if tab.numel() else None, tab.shape[1], n_pages, _stream(stream)),
          "mot_paged_batch_set")


class MotPagedPool:
    """One layer's pages: k, v [n_pages, Hkv, page_size, 128] in bf16, or in
    e4m3 with e8m0 scales k_scale, v_scale [n_pages, Hkv, page_size]."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        e4m3 = k_scale is not None or v_scale is not None
        kv_dtype = torch.float8_e4m3fn if e4m3 else _BF16
        if k.dim() != 4 or k.shape != v.shape or k.shape[3] != 128:
            raise ValueError(f"pages must be [n_pages, Hkv, page_size, 128] (got {list(k.shape)}, {list(v.shape)})")
        if e4m3 and (k_scale is None or v_scale is None or k_scale.shape != k.shape[:3] or v_scale.shape != k.shape[:3]):
            raise ValueError("an e4m3 pool needs both scales, [n_pages, Hkv, page_size]")
        e8m0 = torch.float8_e8m0fnu
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kv_dtype = "e4m3" if e4m3 else "bf16"
        self.c = MotPagedPoolC(_dptr(k, kv_dtype, "k"), _dptr(v, kv_dtype, "v"), _dptr(k_scale, e8m0, "k_scale"),
                               _dptr(v_scale, e8m0, "v_scale"), k.shape[0])
        if any(t is not None and t.device != k.device for t in (v, k_scale, v_scale)):
            raise ValueError("a pool's tensors must be on one device")
        self.ref = byref(self.c)
        self.page_shape, self.device = tuple(k.shape[1:]), k.get_device()


class MotPagedBatch:
    """The sequences of a step; see mot_paged_batch_set."""

    def __init__(self, paged: "MotPaged"):
        self.paged = paged
        self.handle = c_void_p()
        check(lib().mot_paged_batch_create(paged.handle, byref(self.handle)), "mot_paged_batch_create")
        n = c_size_t(0)
        check(lib().mot_paged_query_workspace(self.handle, byref(n)), "mot_paged_query_workspace")
        self.workspace_bytes = n.value
        self._ws, self._ws_streams = None, set()
        self.batch = self.tokens = self.kv_max = 0

    def set(self, q_len: Sequence[int], kv_len: Sequence[int], table, n_pages: int,
            visible: Optional[Sequence[int]] = None, stream=None) -> None:
        self.batch = 0
        if self.paged.handle is None or not self.handle:
            raise ValueError("the batch or its handle has been closed")
        q_len, kv_len = _host_i32(q_len, "q_len"), _host_i32(kv_len, "kv_len")
        mot_paged_batch_set(self.handle, q_len, kv_len, table, n_pages, visible, stream)
        # of the 32-bit lengths: sums in the caller's type may wrap
        self.batch, self.tokens, self.kv_max = q_len.numel(), int(q_len.sum()), int(kv_len.max())
        c = self.paged.cfg
        self.q_shape = (self.tokens, c.n_q_heads, 128)
        self.qkv_shape = (self.tokens, (c.n_q_heads + 2 * c.n_kv_heads) * 128)

    def workspace(self, device="cuda", stream=None) -> torch.Tensor:
        """The batch's own workspace, for work on `stream` (None: the current one)."""
        raw = self.paged._on(stream)
        if self._ws is None:
            with _on_stream(stream):
                self._ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
            self._ws_streams = {raw}
        if raw not in self._ws_streams:
            self._ws.record_stream(_external(raw))  # not another's memory before this stream is done with it
            self._ws_streams.add(raw)
        return self._ws

    def close(self):
        if self.handle:
            lib().mot_paged_batch_destroy(self.handle)
            self.handle = c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MotPaged:
    """A paged-cache handle."""

    def __init__(self, weights: Dict[str, torch.Tensor], n_q_heads: int = 32, n_kv_heads: int = 8, head_dim: int = 128,
                 page_size: int = 64, kv_dtype: str = "bf16", rms_eps: float = 1e-6, rope_theta: float = 1e6,
                 max_positions: int = 8192, max_batch: int = 64, max_tokens: int = 8192, max_pages: int = 8192,
                 stream=None):
        if kv_dtype not in KV_DTYPES:
            raise ValueError(f"kv_dtype must be one of {sorted(KV_DTYPES)} (got {kv_dtype!r})")
        self.kv_dtype = kv_dtype
        self.handle = None
        self.cfg = MotPagedConfig(n_q_heads, n_kv_heads, head_dim, page_size, KV_DTYPES[kv_dtype], float(rms_eps),
                                  float(rope_theta), max_positions, max_batch, max_tokens, max_pages)
        self.device = weights["q_norm"].device
        self.handle = mot_paged_create(self.cfg, weights, stream)
        self._index = weights["q_norm"].get_device()
        self._page_shape = (n_kv_heads, page_size, 128)
        L = lib()
        self._append, self._store, self._load, self._attend = (L.mot_paged_append, L.mot_paged_store, L.mot_paged_load,
                                                               L.mot_paged_attend)

    def new_pool(self, n_pages: int) -> MotPagedPool:
        """One layer's pages, uninitialised."""
        shape = (n_pages, self.cfg.n_kv_heads, self.cfg.page_size, 128)
        if self.kv_dtype == "bf16":
            return MotPagedPool(*[torch.empty(shape, dtype=_BF16, device=self.device) for _ in range(2)])
        kv = [torch.empty(shape, dtype=torch.float8_e4m3fn, device=self.device) for _ in range(2)]
        sc = [torch.empty(shape[:3], dtype=torch.float8_e8m0fnu, device=self.device) for _ in range(2)]
        return MotPagedPool(*kv, *sc)

    def new_batch(self) -> MotPagedBatch:
        return MotPagedBatch(self)

    # With `stream` the outputs and the workspace that a call allocates are that stream's: a tensor that the caller frees
    # goes back to it. Tensors that the caller passes are the caller's to keep until the stream is done with them.
    #
    # The calls below run once per layer and step, where a single token's kernel takes a few microseconds: the
    # checks are written to cost little (plain integers for pointers, no intermediate objects).

    def _check(self, batch: MotPagedBatch, pool: MotPagedPool) -> None:
        if batch.paged is not self:
            raise ValueError("the batch belongs to another handle")
        if batch.batch == 0:
            raise ValueError("the batch has not been set")
        if pool.kv_dtype != self.kv_dtype or pool.page_shape != self._page_shape or pool.device != self._index:
            raise ValueError(f"the pool's pages ({pool.kv_dtype}, {list(pool.page_shape)}, device {pool.device}) are not "
                             f"this handle's")

    def _ptr(self, t: torch.Tensor, dtype, shape, name: str) -> int:
        """Address of a contiguous tensor of this shape and type on the handle's device."""
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
        if t.dtype is not dtype or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor on device {self._index} (got {t.dtype}, "
                             f"{t.device}, strides {t.stride()})")
        return t.data_ptr()

    def _on(self, stream) -> int:
        if stream is None:
            return _raw_stream(self._index)
        return _stream(stream).value or 0

    def append(self, batch: MotPagedBatch, qkv: torch.Tensor, pool: MotPagedPool, q: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """Norms and rotates the chunk's queries (returned, [T, Hq, 128]) and
        keys, and writes its keys and values into the pages.
        qkv: [T, (Hq + 2 Hkv) * 128]."""
        self._check(batch, pool)
        if q is None:
            with _on_stream(stream):
                q = torch.empty(batch.q_shape, dtype=_BF16, device=qkv.device)
        st = self._append(self.handle, batch.handle, self._ptr(qkv, _BF16, batch.qkv_shape, "qkv"), pool.ref,
                          self._ptr(q, _BF16, batch.q_shape, "q"), self._on(stream))
        if st:
            check(st, "mot_paged_append")
        return q

    def store(self, batch: MotPagedBatch, k: torch.Tensor, v: torch.Tensor, pool: MotPagedPool, stream=None) -> None:
        """Dense cache k, v [batch, Hkv, rows, 128] (keys normed and rotated)
        into the pages, kv_len rows of each sequence."""
        self._check(batch, pool)
        rows = k.shape[2] if k.dim() == 4 else -1
        shape = (batch.batch, self.cfg.n_kv_heads, rows, 128)
        st = self._store(self.handle, batch.handle, self._ptr(k, _BF16, shape, "k"), self._ptr(v, _BF16, shape, "v"),
                         rows, pool.ref, self._on(stream))
        if st:
            check(st, "mot_paged_store")

    def load(self, batch: MotPagedBatch, pool: MotPagedPool, k: Optional[torch.Tensor] = None,
             v: Optional[torch.Tensor] = None, stream=None):
        """The pages' rows as the dense cache [batch, Hkv, rows, 128] that
        MotAttnLayer.forward takes (rows: that of k, v when given, else the
        longest sequence's; rows behind a sequence are not written)."""
        self._check(batch, pool)
        if k is None or v is None:
            with _on_stream(stream):
                if k is None:
                    k = torch.empty((batch.batch, self.cfg.n_kv_heads, batch.kv_max, 128) if v is None else v.shape,
                                    dtype=_BF16, device=pool.k.device)
                if v is None:
                    v = torch.empty_like(k)
        rows = k.shape[2] if k.dim() == 4 else -1
        shape = (batch.batch, self.cfg.n_kv_heads, rows, 128)
        st = self._load(self.handle, batch.handle, pool.ref, self._ptr(k, _BF16, shape, "k"),
                        self._ptr(v, _BF16, shape, "v"), rows, self._on(stream))
        if st:
            check(st, "mot_paged_load")
        return k, v

    def attend(self, batch: MotPagedBatch, q: torch.Tensor, pool: MotPagedPool, o: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """Attention of the chunk's queries [T, Hq, 128] over the pages;
        returns o [T, Hq, 128], and writes lse f32 [T, Hq] when given."""
        self._check(batch, pool)
        shape = batch.q_shape
        if o is None:
            with _on_stream(stream):
                o = torch.empty_like(q)
        if workspace is None:
            workspace = batch.workspace(q.device, stream)
        st = self._attend(self.handle, batch.handle, self._ptr(q, _BF16, shape, "q"), pool.ref,
                          self._ptr(o, _BF16, shape, "o"),
                          None if lse is None else self._ptr(lse, _F32, shape[:2], "lse"),
                          self._ptr(workspace, workspace.dtype, workspace.shape, "workspace"),
                          workspace.numel() * workspace.element_size(), self._on(stream))
        if st:
            check(st, "mot_paged_attend")
        return o

    def device_status(self, stream=None) -> int:
        return int(lib().mot_paged_get_device_status(self.handle, _stream(stream)))

    def close(self):
        if self.handle is not None:
            lib().mot_paged_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
