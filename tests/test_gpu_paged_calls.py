"""Calls of the paged prefix-KV cache (include/mot_paged.h) around the kernels:
addresses that are no device memory of the current device, the `stream` argument, what a failed call leaves behind."""
import gc
from ctypes import byref, c_void_p

import pytest
import torch

from mot_flow_matching_b200 import _abi, synth
from mot_flow_matching_b200.paged import MotPaged
from tests.gpu_helpers import ensure_built, make_layer, run_forward, to_dev
from tests.test_gpu_paged import fill_pool, make_paged, make_table, write_sequences

pytestmark = pytest.mark.gpu


def test_create_refuses_gains_in_host_memory(cuda_ready):
    # on the host, before the kernels that would read them
    ensure_built()
    cfg = _abi.MotPagedConfig(4, 2, 128, 16, 0, 1e-6, 1e6, 64, 1, 8, 4)
    dev = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    host, pinned = torch.ones(128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16).pin_memory()
    for q, k in ((host, dev), (dev, host), (pinned, dev), (dev, pinned)):
        out = c_void_p(1)
        w = _abi.MotPagedWeights(q.data_ptr(), k.data_ptr())
        assert _abi.lib().mot_paged_create(byref(cfg), byref(w), None, byref(out)) == _abi.MOT_ERR_INVALID_ARGUMENT
        assert out.value is None
    w = _abi.MotPagedWeights(dev.data_ptr(), dev.data_ptr())
    out = c_void_p()
    assert _abi.lib().mot_paged_create(byref(cfg), byref(w), None, byref(out)) == _abi.MOT_OK
    _abi.lib().mot_paged_destroy(out)


@pytest.mark.parametrize("as_int", [False, True])
def test_outputs_allocated_for_a_stream_are_that_streams(cuda_ready, as_int):
    # Memory that the current stream has freed but not yet finished writing must not become an output of work on
    # another stream: the current stream sleeps, then fills tensors of the outputs' sizes, which are freed at once.
    q_len, kv_len = [40, 1], [300, 500]
    paged, _ = make_paged(8, 2, 16, "bf16", q_len, kv_len)
    table, n_pages = make_table(kv_len, 16)
    pool = fill_pool(paged, n_pages, 0)
    write_sequences(paged, pool, table, kv_len, 1)
    batch = paged.new_batch()
    batch.set(q_len, kv_len, table, n_pages)
    qkv = torch.randn(41, 12 * 128).to(torch.bfloat16).cuda()
    q = paged.append(batch, qkv, pool)
    o, (k, v) = paged.attend(batch, q, pool), paged.load(batch, pool)
    side = torch.cuda.Stream()
    s = side.cuda_stream if as_int else side
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for like in (q, o, k, v):
        torch.empty_like(like).fill_(7.0)
    # and a workspace
    torch.empty(batch.workspace_bytes, dtype=torch.uint8, device="cuda").fill_(255)
    b2 = paged.new_batch()
    b2.set(q_len, kv_len, table, n_pages, stream=s)
    q2 = paged.append(b2, qkv, pool, stream=s)
    o2 = paged.attend(b2, q2, pool, stream=s)
    k2, v2 = paged.load(b2, pool, stream=s)
    torch.cuda.synchronize()
    for a, b, rows in ((q, q2, None), (o, o2, None), (k, k2, kv_len), (v, v2, kv_len)):
        for i in range(len(kv_len) if rows else 1):
            x, y = (a[i, :, :rows[i]], b[i, :, :rows[i]]) if rows else (a, b)
            assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))


def test_a_workspace_is_kept_for_every_stream_that_uses_it(cuda_ready):
    q_len, kv_len = [1], [5000]
    paged, _ = make_paged(8, 2, 16, "bf16", q_len, kv_len)
    table, n_pages = make_table(kv_len, 16)
    pool = fill_pool(paged, n_pages, 0)
    write_sequences(paged, pool, table, kv_len, 1)
    q = torch.randn(1, 8, 128, device="cuda", dtype=torch.bfloat16)
    batch, side = paged.new_batch(), torch.cuda.Stream()
    batch.set(q_len, kv_len, table, n_pages)
    o = paged.attend(batch, q, pool)
    at, n = batch.workspace().data_ptr(), batch.workspace_bytes
    gc.collect()  # handles of other tests
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(500_000_000)
    paged.attend(batch, q, pool, o=o, stream=side)
    batch._ws = None  # as when the batch goes, but without the wait of its cudaFree
    fresh = torch.empty(n, dtype=torch.uint8, device="cuda")
    # not its memory while the side stream is at work (any cudaFree in this process waits for it: then nothing is shown)
    assert fresh.data_ptr() != at or side.query()
    torch.cuda.synchronize()


def test_a_failed_create_leaves_no_error_behind(cuda_ready):
    # no room for the RoPE table of 2^22 positions (2 GiB); the next create, and the other handles', find no error of it
    gains = {n: torch.ones(128, dtype=torch.bfloat16, device="cuda") for n in ("q_norm", "k_norm")}
    torch.cuda.empty_cache()
    held = torch.empty(torch.cuda.mem_get_info()[0] - (1 << 30), dtype=torch.uint8, device="cuda")
    try:
        with pytest.raises(_abi.MotError) as e:
            MotPaged(gains, max_positions=1 << 22)
        assert e.value.status == _abi.MOT_ERR_CUDA
        wl = synth.Workload("gen", 1, 64, 0, 0, 0.0, dims=synth.LayerDims(hidden=512, n_q_heads=4, n_kv_heads=2))
        td = to_dev(synth.make_inputs(wl, 8300, with_dy=False))
        layer = make_layer(wl, td)
        assert run_forward(layer, td)[3] == 0
        layer.close()
        MotPaged(gains, max_positions=64).close()
    finally:
        del held
        torch.cuda.empty_cache()


def test_a_workspace_from_another_stream_serves_the_default_one(cuda_ready):
    q_len, kv_len = [1], [5000]
    paged, _ = make_paged(8, 2, 16, "bf16", q_len, kv_len)
    table, n_pages = make_table(kv_len, 16)
    pool = fill_pool(paged, n_pages, 0)
    write_sequences(paged, pool, table, kv_len, 1)
    q = torch.randn(1, 8, 128, device="cuda", dtype=torch.bfloat16)
    batch, side = paged.new_batch(), torch.cuda.Stream()
    batch.set(q_len, kv_len, table, n_pages)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        o = paged.attend(batch, q, pool)
    side.synchronize()
    for stream in (None, 0, torch.cuda.default_stream(), side):
        o2 = paged.attend(batch, q, pool, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16))
