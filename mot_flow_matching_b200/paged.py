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

from ctypes import byref, c_size_t, c_void_p
from typing import Dict, Optional, Sequence

import torch

from ._abi import MotPagedConfig, MotPagedPoolC, MotPagedWeights, check, lib
from .layer import _BF16, _F32, _dptr, _stream

KV_DTYPES = {"bf16": 0, "e4m3": 1}


def mot_paged_create(cfg: MotPagedConfig, weights: Dict[str, torch.Tensor], stream=None) -> c_void_p:
    w = MotPagedWeights(*[_dptr(weights[n], _BF16, n) for n in ("q_norm", "k_norm")])
    h = c_void_p()
    check(lib().mot_paged_create(byref(cfg), byref(w), _stream(stream), byref(h)), "mot_paged_create")
    return h


def _host_i32(v, name: str) -> Optional[torch.Tensor]:
    if v is None:
        return None
    t = torch.as_tensor(v, dtype=torch.int32)
    if t.is_cuda:
        raise ValueError(f"{name} must be host memory (got {t.device})")
    return t.contiguous()


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


class MotPagedBatch:
    """The sequences of a step; see mot_paged_batch_set."""

    def __init__(self, paged: "MotPaged"):
        self.paged = paged
        self.handle = c_void_p()
        check(lib().mot_paged_batch_create(paged.handle, byref(self.handle)), "mot_paged_batch_create")
        n = c_size_t(0)
        check(lib().mot_paged_query_workspace(self.handle, byref(n)), "mot_paged_query_workspace")
        self.workspace_bytes = n.value
        self._ws = None
        self.batch = self.tokens = self.kv_max = 0

    def set(self, q_len: Sequence[int], kv_len: Sequence[int], table, n_pages: int,
            visible: Optional[Sequence[int]] = None, stream=None) -> None:
        self.batch = 0
        mot_paged_batch_set(self.handle, q_len, kv_len, table, n_pages, visible, stream)
        self.batch, self.tokens, self.kv_max = len(q_len), int(sum(q_len)), int(max(kv_len))

    def workspace(self, device="cuda") -> torch.Tensor:
        if self._ws is None:
            self._ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
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

    def _check(self, batch: MotPagedBatch, pool: MotPagedPool) -> None:
        if batch.paged is not self:
            raise ValueError("the batch belongs to another handle")
        if batch.batch == 0:
            raise ValueError("the batch has not been set")
        if pool.kv_dtype != self.kv_dtype or tuple(pool.k.shape[1:]) != (self.cfg.n_kv_heads, self.cfg.page_size, 128):
            raise ValueError(f"the pool's pages ({pool.kv_dtype}, {list(pool.k.shape[1:])}) are not this handle's")

    @staticmethod
    def _shape(t: torch.Tensor, shape, name: str) -> torch.Tensor:
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
        return t

    def append(self, batch: MotPagedBatch, qkv: torch.Tensor, pool: MotPagedPool, q: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """Norms and rotates the chunk's queries (returned, [T, Hq, 128]) and
        keys, and writes its keys and values into the pages.
        qkv: [T, (Hq + 2 Hkv) * 128]."""
        self._check(batch, pool)
        c = self.cfg
        self._shape(qkv, (batch.tokens, (c.n_q_heads + 2 * c.n_kv_heads) * 128), "qkv")
        if q is None:
            q = torch.empty(batch.tokens, c.n_q_heads, 128, dtype=_BF16, device=qkv.device)
        self._shape(q, (batch.tokens, c.n_q_heads, 128), "q")
        check(lib().mot_paged_append(self.handle, batch.handle, _dptr(qkv, _BF16, "qkv"), byref(pool.c),
                                     _dptr(q, _BF16, "q"), _stream(stream)), "mot_paged_append")
        return q

    def _dense(self, batch, k, v):
        rows = k.shape[2] if k.dim() == 4 else -1
        for t, name in ((k, "k"), (v, "v")):
            self._shape(t, (batch.batch, self.cfg.n_kv_heads, rows, 128), name)
        return rows

    def store(self, batch: MotPagedBatch, k: torch.Tensor, v: torch.Tensor, pool: MotPagedPool, stream=None) -> None:
        """Dense cache k, v [batch, Hkv, rows, 128] (keys normed and rotated)
        into the pages, kv_len rows of each sequence."""
        self._check(batch, pool)
        rows = self._dense(batch, k, v)
        check(lib().mot_paged_store(self.handle, batch.handle, _dptr(k, _BF16, "k"), _dptr(v, _BF16, "v"), rows,
                                    byref(pool.c), _stream(stream)), "mot_paged_store")

    def load(self, batch: MotPagedBatch, pool: MotPagedPool, k: Optional[torch.Tensor] = None,
             v: Optional[torch.Tensor] = None, stream=None):
        """The pages' rows as the dense cache [batch, Hkv, rows, 128] that
        MotAttnLayer.forward takes (rows: that of k, v when given, else the
        longest sequence's; rows behind a sequence are not written)."""
        self._check(batch, pool)
        shape = (batch.batch, self.cfg.n_kv_heads, batch.kv_max, 128)
        if k is None:
            k = torch.empty(shape if v is None else v.shape, dtype=_BF16, device=pool.k.device)
        if v is None:
            v = torch.empty_like(k)
        rows = self._dense(batch, k, v)
        check(lib().mot_paged_load(self.handle, batch.handle, byref(pool.c), _dptr(k, _BF16, "k"), _dptr(v, _BF16, "v"),
                                   rows, _stream(stream)), "mot_paged_load")
        return k, v

    def attend(self, batch: MotPagedBatch, q: torch.Tensor, pool: MotPagedPool, o: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """Attention of the chunk's queries [T, Hq, 128] over the pages;
        returns o [T, Hq, 128], and writes lse f32 [T, Hq] when given."""
        self._check(batch, pool)
        shape = (batch.tokens, self.cfg.n_q_heads, 128)
        self._shape(q, shape, "q")
        if o is None:
            o = torch.empty_like(q)
        self._shape(o, shape, "o")
        if lse is not None:
            self._shape(lse, shape[:2], "lse")
        if workspace is None:
            workspace = batch.workspace(q.device)
        check(lib().mot_paged_attend(self.handle, batch.handle, _dptr(q, _BF16, "q"), byref(pool.c),
                                     _dptr(o, _BF16, "o"), _dptr(lse, _F32, "lse"), _dptr(workspace, None, "workspace"),
                                     workspace.numel(), _stream(stream)), "mot_paged_attend")
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
