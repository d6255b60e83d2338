"""Host-only checks of the paged-cache C ABI (include/mot_paged.h): what a
configuration, a batch and a call may say is decided on the host before any
CUDA call, and the attention's work is cut so that every key of every tile is
taken exactly once (no GPU needed)."""
import ctypes
from ctypes import byref, c_int32, c_size_t, c_void_p

import numpy as np
import pytest
import torch

from mot_flow_matching_b200 import _abi
from mot_flow_matching_b200 import build as build_mod

INVALID, SHAPE = _abi.MOT_ERR_INVALID_ARGUMENT, _abi.MOT_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return _abi.lib()


def cfg(**kw):
    c = _abi.MotPagedConfig(32, 8, 128, 64, 0, 1e-6, 1e6, 8192, 8, 4096, 256)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def arr(v):
    return np.ascontiguousarray(v, dtype=np.int32)


def check(L, c, q_len, kv_len, table, n_pages, visible=None, stride=None):
    q, k, t = arr(q_len), arr(kv_len), arr(table)
    v = arr(visible) if visible is not None else None
    return L.mot_paged_batch_check(byref(c), len(q), q.ctypes.data, k.ctypes.data, v.ctypes.data if v is not None else None,
                                   t.ctypes.data, t.shape[1] if stride is None else stride, n_pages)


@pytest.mark.parametrize("field,value,status", [
    ("head_dim", 64, SHAPE), ("n_kv_heads", 5, SHAPE), ("n_kv_heads", 0, INVALID), ("n_q_heads", -32, INVALID),
    ("page_size", 8, SHAPE), ("page_size", 48, SHAPE), ("page_size", 256, SHAPE), ("page_size", 0, INVALID),
    ("kv_dtype", 2, INVALID), ("kv_dtype", -1, INVALID), ("rms_eps", -1.0, INVALID), ("rms_eps", float("nan"), INVALID),
    ("rope_theta", 0.0, INVALID), ("max_positions", 0, INVALID), ("max_positions", 1 << 23, SHAPE),
    ("max_batch", 0, INVALID), ("max_batch", 5000, SHAPE), ("max_tokens", 0, INVALID), ("max_pages", -3, INVALID),
])
def test_config_validation(L, field, value, status):
    out = c_void_p(1)
    w = _abi.MotPagedWeights(4096, 8192)
    assert L.mot_paged_create(byref(cfg(**{field: value})), byref(w), None, byref(out)) == status
    assert out.value is None
    assert check(L, cfg(**{field: value}), [1], [1], [[0]], 1) == status


def test_create_rejects_bad_arguments_before_cuda(L):
    out = c_void_p(1)
    assert L.mot_paged_create(byref(cfg()), byref(_abi.MotPagedWeights()), None, byref(out)) == INVALID
    assert out.value is None
    assert L.mot_paged_create(byref(cfg()), byref(_abi.MotPagedWeights(4096, 8194)), None, byref(out)) == \
        _abi.MOT_ERR_ALIGNMENT
    assert L.mot_paged_create(byref(cfg()), None, None, byref(out)) == INVALID
    assert L.mot_paged_create(byref(cfg()), byref(_abi.MotPagedWeights(4096, 8192)), None, None) == INVALID
    assert L.mot_paged_create(byref(cfg(n_q_heads=8 * 65)), byref(_abi.MotPagedWeights(4096, 8192)), None,
                              byref(out)) == SHAPE


def test_batch_validation(L):
    c = cfg()
    assert check(L, c, [4, 1], [130, 64], [[0, 1, 2], [3, -1, -1]], 4) == _abi.MOT_OK
    assert check(L, c, [0, 0], [0, 64], [[-1], [0]], 1) == _abi.MOT_OK
    for table in ([[0, 1, 4], [3, 0, 0]], [[0, -1, 2], [3, 0, 0]], [[0, 1, 2], [4, 0, 0]], [[0, 1, -2 ** 31], [3, 0, 0]]):
        assert check(L, c, [4, 1], [130, 64], table, 4) == INVALID, table  # a page that is not in the pool
    assert check(L, c, [4, 1], [130, 65], [[0, 1], [2, 3]], 4) == INVALID  # the table is too narrow
    assert check(L, c, [131, 1], [130, 64], [[0, 1, 2], [3, 0, 0]], 4) == INVALID
    assert check(L, c, [-1, 1], [130, 64], [[0, 1, 2], [3, 0, 0]], 4) == INVALID
    assert check(L, c, [0, 0], [-1, 64], [[0, 1, 2], [3, 0, 0]], 4) == INVALID
    assert check(L, c, [4, 1], [130, 64], [[0, 1, 2], [3, 0, 0]], 4, visible=[131, 0]) == INVALID
    assert check(L, c, [4, 1], [130, 64], [[0, 1, 2], [3, 0, 0]], 4, visible=[-1, 0]) == INVALID
    assert check(L, c, [4, 1], [130, 64], [[0, 1, 2], [3, 0, 0]], 4, visible=[130, 64]) == _abi.MOT_OK
    assert check(L, c, [1], [8193], [list(range(129))], 129) == SHAPE
    assert check(L, c, [1] * 9, [1] * 9, [[i] for i in range(9)], 9) == SHAPE
    assert check(L, c, [4096, 1], [4096, 1], [list(range(64))] * 2, 64) == SHAPE  # too many tokens
    assert check(L, cfg(max_pages=2), [1], [129], [[0, 1, 2]], 3) == SHAPE
    assert check(L, c, [1], [1], [[0]], 1 << 30) == SHAPE  # more pool rows than a TMA coordinate holds
    assert check(L, c, [1], [1], [[0]], 0) == INVALID
    assert L.mot_paged_batch_check(byref(c), 1, None, None, None, None, 0, 1) == INVALID
    assert L.mot_paged_batch_check(None, 1, None, None, None, None, 0, 1) == INVALID


def test_calls_refuse_null_handles(L):
    pool = _abi.MotPagedPoolC(16, 16, None, None, 1)
    assert L.mot_paged_batch_create(None, byref(c_void_p())) == INVALID
    assert L.mot_paged_batch_set(None, 1, None, None, None, None, 0, 1, None) == INVALID
    assert L.mot_paged_query_workspace(None, byref(c_size_t())) == INVALID
    assert L.mot_paged_append(None, None, 16, byref(pool), 16, None) == INVALID
    assert L.mot_paged_store(None, None, 16, 16, 1, byref(pool), None) == INVALID
    assert L.mot_paged_load(None, None, byref(pool), 16, 16, 1, None) == INVALID
    assert L.mot_paged_attend(None, None, 16, byref(pool), 16, None, 16, 16, None) == INVALID
    assert L.mot_paged_get_device_status(None, None) == INVALID
    L.mot_paged_destroy(None)
    L.mot_paged_batch_destroy(None)


def test_bindings_refuse_host_tensors():
    from mot_flow_matching_b200.paged import MotPaged, MotPagedPool
    gains = {n: torch.ones(128, dtype=torch.bfloat16) for n in ("q_norm", "k_norm")}
    with pytest.raises(ValueError, match="CUDA"):
        MotPaged(gains)
    with pytest.raises(ValueError, match="kv_dtype"):
        MotPaged(gains, kv_dtype="int8")
    pages = torch.zeros(2, 8, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        MotPagedPool(pages, pages)
    with pytest.raises(ValueError, match="pages must be"):
        MotPagedPool(pages[..., :64], pages[..., :64])


class FakeCudaTensor:
    # what the binding looks at before it hands over an address
    is_cuda, dtype = True, torch.bfloat16

    def __init__(self, device, shape=(128,)):
        self.index, self.shape, self.device = device, torch.Size(shape), f"cuda:{device}"

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


def test_gains_elsewhere_or_of_another_size_reach_no_kernel(monkeypatch):
    # the kernels of create read 128 values of each gain on the current device
    from mot_flow_matching_b200 import paged as binding

    def no_library():
        raise AssertionError("the library was called")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(binding, "lib", no_library)
    monkeypatch.setattr(binding, "_stream", lambda s: c_void_p(0))
    good = FakeCudaTensor(0)
    for bad in (FakeCudaTensor(1), FakeCudaTensor(0, (64,)), FakeCudaTensor(0, (1, 128))):
        for weights in ({"q_norm": bad, "k_norm": good}, {"q_norm": good, "k_norm": bad}, {"q_norm": bad, "k_norm": bad}):
            with pytest.raises(ValueError, match="_norm must be"):
                binding.MotPaged(weights)
    with pytest.raises(AssertionError, match="library"):
        binding.MotPaged({"q_norm": good, "k_norm": good})


def test_bindings_refuse_lengths_and_pages_that_are_not_32_bit_integers():
    from mot_flow_matching_b200.paged import mot_paged_batch_set
    good = dict(q_len=[1, 1], kv_len=[3, 4], table=[[0], [1]], visible=[0, 0])
    for name in good:
        for bad in (torch.tensor(good[name]).double(), torch.tensor(good[name]) + 2 ** 32,
                    torch.tensor(good[name]) - 2 ** 32):
            with pytest.raises(ValueError, match=name):
                mot_paged_batch_set(None, n_pages=2, **{**good, name: bad})
    with pytest.raises(ValueError, match="q_len must be integers"):
        mot_paged_batch_set(None, n_pages=2, **{**good, "q_len": [1.5, 1]})


@pytest.mark.parametrize("q_len,kv_len", [([200, 100], [250, 130]), ([1, 0, 127], [1, 5, 127])])
def test_lengths_of_any_integer_type_add_up(monkeypatch, q_len, kv_len):
    # 200 + 100 is 44 in 8 bits
    from mot_flow_matching_b200 import paged as binding
    monkeypatch.setattr(binding, "mot_paged_batch_set", lambda *a, **k: None)
    paged, batch = object.__new__(binding.MotPaged), object.__new__(binding.MotPagedBatch)
    paged.handle, paged.cfg, batch.paged, batch.handle = None, cfg(), paged, c_void_p(16)
    try:
        for kind in (list, tuple, np.uint8, np.int16, np.int64, torch.uint8, torch.int16, torch.int64):
            make = (lambda x: torch.tensor(x, dtype=kind)) if isinstance(kind, torch.dtype) else \
                kind if kind in (list, tuple) else (lambda x: np.array(x, dtype=kind))
            paged.handle = c_void_p(16)
            batch.set(make(q_len), make(kv_len), [[0]], 1)
            assert (batch.batch, batch.tokens, batch.kv_max) == (len(q_len), sum(q_len), max(kv_len)), kind
            assert batch.q_shape == (sum(q_len), 32, 128)
    finally:
        paged.handle, batch.handle = None, c_void_p()  # not the library's: nothing to free


def test_a_closed_handle_sets_no_batch():
    # the batch object's memory in the library refers to the handle's
    from mot_flow_matching_b200.paged import MotPaged, MotPagedBatch
    paged, batch = object.__new__(MotPaged), object.__new__(MotPagedBatch)
    paged.handle, batch.paged, batch.handle = None, paged, c_void_p(16)
    try:
        with pytest.raises(ValueError, match="closed"):
            batch.set([1], [1], [[0]], 1)
    finally:
        batch.handle = c_void_p()  # not the library's: nothing to free


def plan(L, kind, tiles, heads, ctas, cap=None):
    t = arr(tiles).reshape(-1, 3)
    cap = len(t) * heads + ctas if cap is None else cap
    units, first, n = np.full((cap + 1, 16), -7, dtype=np.int32), arr(np.zeros(ctas + 1)), c_int32()
    st = L.mot_dev_paged_plan(kind, t.ctypes.data, len(t), heads, ctas, units.ctypes.data, cap, first.ctypes.data, byref(n))
    assert (units[cap] == -7).all()
    return st, units[: n.value], first


@pytest.mark.parametrize("kind,granule,ctas", [(0, 128, 296), (1, 128, 148), (0, 128, 7), (1, 128, 3)])
@pytest.mark.parametrize("seed", range(6))
def test_plan_covers_every_key_once(L, kind, granule, ctas, seed):
    g = np.random.default_rng(seed)
    heads = int(g.choice([1, 2, 8]))
    n = int(g.choice([1, 2, 5, 64, 300]))
    top = int(g.choice([1, 130, 5000, 100000]))
    tiles = [(i, 8 * i, int(g.integers(1, top + 1))) for i in range(n)]
    st, units, first = plan(L, kind, tiles, heads, ctas)
    assert st == _abi.MOT_OK
    assert first[0] == 0 and first[-1] == len(units) and (np.diff(first) >= 0).all()
    seen, slots, counters = {}, set(), {}
    for u in units:
        seq, head, row0, k0, k1, slot0, split, counter = (int(x) for x in u[:8])
        assert row0 == 8 * seq and 0 <= head < heads and k0 % granule == 0 and k0 < k1
        number, of = split & 0xFFFF, split >> 16
        seen.setdefault((seq, head), []).append((number, of, k0, k1, slot0, counter))
        if of > 1:
            assert slot0 + number not in slots  # a partial of its own
            slots.add(slot0 + number)
            assert counters.setdefault(counter, (seq, head)) == (seq, head)
    assert len(seen) == n * heads
    for (seq, head), parts in seen.items():
        at = 0
        for i, (number, of, k0, k1, _, _) in enumerate(parts):
            assert number == i and of == len(parts) and k0 == at
            at = k1
        assert at == tiles[seq][2]
    assert max(slots, default=0) < 2 * ctas and max(counters, default=0) < ctas  # what the workspace holds


def test_plan_shares_the_work(L):
    # one long sequence, 8 heads: no CTA gets more than the average and a few granules
    for kind, ctas in ((0, 296), (1, 148)):
        st, units, first = plan(L, kind, [(0, 0, 100000)], 8, ctas)
        work = [sum(-(-(int(u[4]) - int(u[3])) // 128) for u in units[a:b]) for a, b in zip(first[:-1], first[1:])]
        assert max(work) <= 8 * 782 / ctas * 1.1 + 4
    # as many equal tiles as CTAs stay whole
    st, units, first = plan(L, 1, [(i, 0, 4096) for i in range(148)], 1, 148)
    assert len(units) == 148 and (np.diff(first) == 1).all()


def test_plan_of_nothing_and_too_little_room(L):
    st, units, first = plan(L, 0, np.zeros((0, 3)), 8, 296)
    assert st == _abi.MOT_OK and len(units) == 0 and (first == 0).all()
    assert plan(L, 0, [(0, 0, 5000)], 8, 296, cap=3)[0] == SHAPE
