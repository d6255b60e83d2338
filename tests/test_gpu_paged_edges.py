"""The paged prefix-KV cache at the ends of what its calls allow: pages far into
a large pool, sequences of a million keys, the largest head groups, thousands of
sequences, scales that no call of this library writes."""
import numpy as np
import pytest
import torch

from oracle import mot_paged_oracle as PG
from tests.test_gpu_paged import (EPS, HALF_BF16, THETA, as_f64, attend_tolerance, fill_pool, lse_tolerance, make_paged, make_table,
                                  pool_values, run_attend, sequence_rows, small_weights, write_sequences)

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages_behind_four_gigabytes(cuda_ready, kv):
    # the same batch in a small pool and in the last pages of a large one: bit for bit, all four operators
    q_len, kv_len, page, hkv = [1, 90, 3], [200, 300, 77], 64, 8
    n_far = 45000 if kv == "bf16" else 90000  # 128 or 64 KB a page, k and v each
    paged, _ = make_paged(32, hkv, page, kv, q_len, kv_len)
    table, n = make_table(kv_len, page, 5, spare=0)
    near, far = fill_pool(paged, n, 0), paged.new_pool(n_far)
    assert far.k.numel() * far.k.element_size() > 2 ** 32
    far_table = np.where(table >= 0, n_far - n + table, table)
    qkv = torch.randn(sum(q_len), 48 * 128, device="cuda", dtype=torch.bfloat16)
    dense = [torch.randn(3, hkv, 300, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    got = []
    for pool, tab, pages in ((near, table, n), (far, far_table, n_far)):
        batch = paged.new_batch()
        batch.set(q_len, kv_len, tab, pages)
        paged.store(batch, *dense, pool)
        q = paged.append(batch, qkv, pool)
        o = paged.attend(batch, q, pool)
        k, v = (torch.zeros_like(d) for d in dense)
        paged.load(batch, pool, k, v)
        torch.cuda.synchronize()
        got.append((q, o, k, v))
    assert paged.device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(bits(a), bits(b))
    assert torch.isfinite(got[0][1]).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 3, 40])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (4, 4)])
def test_a_million_keys(cuda_ready, q_len, hq, hkv, kv):
    # One page listed 8000 times and one of its own at the end, where the chunk is: the softmax counts a key of the
    # first 8000 times. The bound's sums are over 2^20 keys here: f32 adds in a tree of at most 2^14 sequential steps (a
    # CTA's share of the keys, a few at a time), 2^-10.
    page, reps, tail = 128, 8000, 57
    n = page * reps + tail
    paged, _ = make_paged(hq, hkv, page, kv, [q_len], [2 * page], max_positions=n, max_pages=reps + 1)
    pool = fill_pool(paged, 2, 0)
    write_sequences(paged, pool, np.array([[0, 1]], dtype=np.int32), [page + tail], 3)
    batch = paged.new_batch()
    batch.set([q_len], [n], np.array([[0] * reps + [1]], dtype=np.int32), 2)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(q_len, hq, 128, generator=g).to(torch.bfloat16).cuda()
    lse = torch.empty(q_len, hq, device="cuda")
    o = paged.attend(batch, q, pool, lse=lse)
    torch.cuda.synchronize()
    assert paged.device_status() == 0
    k, v = (np.concatenate([x[0], x[1][:, :tail]], axis=1) for x in pool_values(pool))
    o, lse, qf = as_f64(o), as_f64(lse), as_f64(q)
    count = np.concatenate([np.full(page, float(reps)), np.ones(tail)])
    for i in sorted({0, q_len // 2, q_len - 1}):
        for h in range(hq):
            limit = page + tail - q_len + i + 1
            kk, vv, c = k[h * hkv // hq, :limit], v[h * hkv // hq, :limit], count[:limit]
            s = kk @ qf[i, h] / np.sqrt(128)
            w = c * np.exp(s - s.max())
            ref, absv = (w / w.sum()) @ vv, (w / w.sum()) @ np.abs(vv)
            mag = (np.abs(kk) @ np.abs(qf[i, h])).max() / np.sqrt(128)
            tol = attend_tolerance(ref, absv, np.float64(mag).reshape(()), 0.0) + absv * 2.0 ** -10
            if kv == "e4m3":  # n * 2^-24 * max|v| over the weights' sum, which here is at least `reps` times the largest
                tol = tol + n * 2.0 ** -24 * np.abs(vv).max() / w.sum()
            assert np.all(np.abs(o[i, h] - ref) <= tol), (i, h, np.abs(o[i, h] - ref).max())
            assert abs(lse[i, h] - (s.max() + np.log(w.sum()))) <= lse_tolerance(np.float64(20.0), mag) + 2.0 ** -10


def test_append_at_far_positions(cuda_ready):
    # positions around 2^20: the angles are taken in f64
    page, n, q_len = 128, 2 ** 20, 150
    paged, w = make_paged(4, 2, page, "bf16", [q_len], [page], max_positions=n, max_pages=n // page)
    pool = fill_pool(paged, 3, 0)
    batch = paged.new_batch()
    batch.set([q_len], [n - 1], np.array([[0] * (n // page - 2) + [1, 2]], dtype=np.int32), 3)
    g = torch.Generator().manual_seed(6)
    qkv = torch.randn(q_len, 8 * 128, generator=g).to(torch.bfloat16).cuda()
    q = paged.append(batch, qkv, pool)
    pos = np.arange(n - 1 - q_len, n - 1)
    gains = {x: as_f64(w[x]) for x in w}
    qr, kr, vr = PG.chunk_qkv(as_f64(qkv).reshape(q_len, 8, 128), pos, gains["q_norm"], gains["k_norm"], 4, 2, EPS, THETA)
    kval, vval = pool_values(pool)
    ids = 1 + (pos // page - (n // page - 2))

    def tau(r):
        pair = np.hypot(r[..., :64], r[..., 64:])
        return 2.0 ** -16 * np.concatenate([pair, pair], -1)
    assert np.all(np.abs(as_f64(q) - qr) <= HALF_BF16 * (np.abs(qr) + tau(qr)) + tau(qr))
    assert np.all(np.abs(kval[ids, :, pos % page] - kr) <= HALF_BF16 * (np.abs(kr) + tau(kr)) + tau(kr))
    assert np.array_equal(vval[ids, :, pos % page], vr)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", [(64, 1), (48, 1), (128, 2), (33, 3)])
def test_the_largest_head_groups(cuda_ready, hq, hkv, kv):
    run_attend(hq, hkv, 32, kv, [1, 7, 40], [300, 77, 290], [0, 0, 290], seed=hq, sample=3)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_thousands_of_sequences(cuda_ready, kv):
    g = np.random.default_rng(0)
    kv_len = g.integers(1, 60, size=3000).tolist()
    q_len = [min(k, int(x)) for k, x in zip(kv_len, g.integers(0, 3, size=3000))]
    q_len[17], kv_len[17] = 50, 59
    run_attend(4, 2, 16, kv, q_len, kv_len, seed=8, sample=1)


@pytest.mark.parametrize("q_len", [1, 3, 100])
@pytest.mark.parametrize("k_byte,v_byte,q_power", [(0, 127, 126), (1, 20, 100), (254, 127, -125), (127, 250, 0), (130, 0, -3), (132, 254, -4)])
def test_scales_that_no_call_writes(cuda_ready, k_byte, v_byte, q_power, q_len):
    # a pool that comes from elsewhere may have any scale byte over any payload
    n = 300
    paged, _ = make_paged(4, 2, 16, "e4m3", [q_len], [n])
    table, n_pages = make_table([n], 16)
    pool = fill_pool(paged, n_pages, 0)
    g = torch.Generator().manual_seed(k_byte)
    for pages, scale, byte in ((pool.k, pool.k_scale, k_byte), (pool.v, pool.v_scale, v_byte)):
        # magnitudes of at most 1: below 2^128 with the largest scale
        x = torch.randn(*pages.shape, generator=g).clamp(-3, 3) * 0.25
        pages.copy_(x.to(torch.float8_e4m3fn).cuda())
        scale.view(torch.uint8).fill_(byte)
    batch = paged.new_batch()
    batch.set([q_len], [n], table, n_pages)
    q = (torch.randn(q_len, 4, 128, generator=g) * 2.0 ** q_power).to(torch.bfloat16).cuda()
    lse = torch.empty(q_len, 4, device="cuda")
    o, lse = as_f64(paged.attend(batch, q, pool, lse=lse)), as_f64(lse)
    k, v = (sequence_rows(x, table, 0, n, 16) for x in pool_values(pool))
    ref, l, absv, mag = PG.chunk_attention(as_f64(q), k, v, 0)
    # An output below 2^-126 is a multiple of 2^-133. Weights before they are divided by their sum are at most 2^8: where
    # n * 2^8 * max|v| is no f32, the sum may be infinite although the output would not be.
    near = np.abs(o - ref) <= attend_tolerance(ref, absv, mag, small_weights("e4m3", v)) + 2.0 ** -133
    over = n * 2.0 ** 8 * np.abs(v).max() >= 2.0 ** 128
    fine = np.isfinite(as_f64(q)).all(-1)  # 2^126 times a normal value is infinite now and then
    assert np.all(near[fine] | (over & ~np.isfinite(o[fine])))
    assert not np.isfinite(o[~fine]).any()
    assert np.all(np.abs(lse - l)[fine] <= lse_tolerance(l, mag)[fine])
