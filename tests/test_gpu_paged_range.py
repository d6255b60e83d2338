"""The paged attention over its whole range of magnitudes: cached rows of very
different size, seen and unseen, queries near the ends of f32. Every query is
held to the fp64 oracle over the keys that it sees, and every bound is taken
from those keys alone."""
import numpy as np
import pytest
import torch

from oracle import mot_paged_oracle as PG
from tests.test_gpu_paged import (as_f64, attend_tolerance, fill_pool, lse_tolerance, make_paged, make_table, pool_values,
                                  sequence_rows, small_weights)

pytestmark = pytest.mark.gpu


def cached(hq, hkv, page, kv, q_len, kv_len, k, v, visible=None, **kw):
    """A pool and a batch of sequences whose dense keys and values are k, v [B, Hkv, rows, 128]."""
    paged, _ = make_paged(hq, hkv, page, kv, q_len, kv_len, **kw)
    table, n_pages = make_table(kv_len, page, 3)
    pool = fill_pool(paged, n_pages, 0)
    batch = paged.new_batch()
    batch.set(q_len, kv_len, table, n_pages, visible=visible)
    paged.store(batch, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), pool)
    return paged, pool, table, batch


def attend(paged, pool, batch, q):
    lse = torch.full(q.shape[:2], -7.0, device="cuda")
    o = paged.attend(batch, q, pool, lse=lse)
    torch.cuda.synchronize()
    assert paged.device_status() == 0
    return as_f64(o), as_f64(lse)


def check_rows(paged, pool, table, q, q_len, kv_len, visible, o, lse, small=small_weights, rows=None):
    """The queries of one sequence (`rows` of them) against the oracle over what each sees."""
    k, v = (sequence_rows(x, table, 0, kv_len, paged.cfg.page_size) for x in pool_values(pool))
    qf = as_f64(q)
    for i in range(q_len) if rows is None else rows:
        limit = max(visible, kv_len - q_len + i + 1)
        ref, l, absv, mag = PG.chunk_attention(qf[i:i + 1], k[:, :limit], v[:, :limit], limit)
        tol = attend_tolerance(ref, absv, mag, small(pool.kv_dtype, v[:, :limit]))
        err = np.abs(o[i:i + 1] - ref)
        assert np.all(err <= tol), (i, limit, float(np.nanmax(err / tol)), o[i, 0, :4], ref[0, 0, :4])
        assert np.all(np.abs(lse[i:i + 1] - l) <= lse_tolerance(l, mag)), (i, lse[i], l)


# 4 query heads over 2 KV heads: 2 or 3 tokens are 4 or 6 query rows of a unit of 8, 200 tokens 400 rows of two of 256
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("power", [10, 17, 24, 30, 60])
@pytest.mark.parametrize("q_len,past,where", [(2, 0, 1), (3, 300, 2), (4, 61, 1), (200, 0, 1), (200, 70, 130), (130, 300, 129)])
def test_rows_that_a_query_does_not_see_may_be_of_any_size(cuda_ready, q_len, past, where, power, what, kv):
    g = torch.Generator().manual_seed(q_len + power)
    n = past + q_len
    dense = {x: torch.randn(1, 2, n, 128, generator=g) for x in ("k", "v")}
    dense[what][0, :, past + where] *= 2.0 ** power
    paged, pool, table, batch = cached(4, 2, 16, kv, [q_len], [n], dense["k"], dense["v"])
    q = torch.randn(q_len, 4, 128, generator=g).to(torch.bfloat16).cuda()
    o, lse = attend(paged, pool, batch, q)
    check_rows(paged, pool, table, q, q_len, n, 0, o, lse, rows=sorted({0, 1, where // 2, where - 1, where, q_len - 1}))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("power", [20, 40, 90])
@pytest.mark.parametrize("big_first", [False, True])
@pytest.mark.parametrize("q_len,n", [(1, 40), (3, 700), (40, 90), (130, 700)])
def test_a_large_value_of_small_weight_leaves_the_others(cuda_ready, q_len, n, big_first, power, kv):
    # Half of the keys have score 22.6 and values of 1, the others score -22.6 (weights of 2^-65) and values of 2^power:
    # all of them seen by all queries. A weight that meets 8-bit values is a multiple of 2^-31 of the largest product of
    # weight and value (2^7 below 1, and 2^-24 of that), off by half of one, times 448 units of which the largest value
    # has at least 224.
    g = torch.Generator().manual_seed(n + power)
    u = torch.randint(0, 2, (2, 1, 128), generator=g).float() * 2 - 1
    v = torch.randn(1, 2, n, 128, generator=g)
    far = torch.arange(n) < n // 2
    far = far if big_first else ~far
    k = 0.25 * u[None] * torch.where(far, -1.0, 1.0)[None, None, :, None]
    v[:, :, far] *= 2.0 ** power
    paged, pool, table, batch = cached(4, 2, 16, kv, [q_len], [n], k, v, visible=[n])
    q = (8 * u.repeat_interleave(2, 0)[:, 0])[None].expand(q_len, 4, 128).contiguous().to(torch.bfloat16).cuda()
    o, lse = attend(paged, pool, batch, q)

    def small(kv_dtype, vv):
        s = np.where(far.numpy(), -22.6, 22.6)
        w = np.exp(s - 22.6)
        return len(w) * 2.0 ** -31 * (w / w.sum() * np.abs(vv).max(-1)).max() if kv_dtype == "e4m3" else 0.0
    check_rows(paged, pool, table, q, q_len, n, n, o, lse, small=small, rows=sorted({0, q_len // 2, q_len - 1}))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("power", [24, 60])
@pytest.mark.parametrize("q_len", [1, 100])
def test_keys_far_apart_keep_their_scores(cuda_ready, q_len, power, kv):
    # One seen key is 2^power times the others and at right angles to the queries (score 0 exactly): the scores of the
    # others count, and the bound on them does not have the large key's size in it.
    g = torch.Generator().manual_seed(power)
    n = 150
    k, v = (torch.randn(1, 2, n, 128, generator=g) for _ in range(2))
    k[0, :, 20, :64] = 0
    k[0, :, 20] *= 2.0 ** power
    paged, pool, table, batch = cached(4, 2, 16, kv, [q_len], [n], k, v, visible=[n])
    q = torch.randn(q_len, 4, 128, generator=g)
    q[..., 64:] = 0
    q = q.to(torch.bfloat16).cuda()
    o, lse = attend(paged, pool, batch, q)
    kk, vv = (sequence_rows(x, table, 0, n, 16) for x in pool_values(pool))
    kk[:, 20] = 0  # the same scores
    ref, l, absv, mag = PG.chunk_attention(as_f64(q), kk, vv, n)
    assert np.all(np.abs(o - ref) <= attend_tolerance(ref, absv, mag, small_weights(kv, vv)))
    assert np.all(np.abs(lse - l) <= lse_tolerance(l, mag))


@pytest.mark.parametrize("hq,hkv,page", [(4, 2, 16), (4, 4, 128), (6, 2, 64), (8, 1, 32)])
def test_units_of_both_kinds_in_turn(cuda_ready, hq, hkv, page):
    # many sequences a CTA, every other one with scales that f16 does not bear (large or small values or keys, rows of
    # zeros), lengths that end inside a tile, one row of NaN that only the last query of its sequence sees
    g = torch.Generator().manual_seed(hq)
    lengths = [200, 129, 300, 70, 257, 512, 90, 385] * 8
    q_len = [70, 129, 40, 70, 100, 33, 90, 260] * 8
    n, rows = len(lengths), max(lengths)
    k, v = (torch.randn(n, hkv, rows, 128, generator=g) for _ in range(2))
    for b in range(0, n, 2):
        at = torch.randint(0, lengths[b], (7,), generator=g)
        (v if b % 4 else k)[b, :, at] *= 2.0 ** (20 if b % 8 else -30)
    for b in range(1, n, 8):
        v[b, :, lengths[b] // 2] = 0
    v[5, :, lengths[5] - 1, 3] = float("nan")
    paged, pool, table, batch = cached(hq, hkv, page, "e4m3", q_len, lengths, k, v)
    q = torch.randn(sum(q_len), hq, 128, generator=g).to(torch.bfloat16).cuda()
    o, lse = attend(paged, pool, batch, q)
    at = 0
    for b in range(n):
        sl = slice(at, at + q_len[b])
        if b < 16 or b % 7 == 0:
            last = q_len[b] - 1
            check_rows(paged, pool, table[b:b + 1], q[sl], q_len[b], lengths[b], 0, o[sl], lse[sl],
                       rows=[0, q_len[b] // 2, last - (b == 5)])
        at += q_len[b]
    end = sum(q_len[:6]) - 1
    assert np.isnan(o[end]).all() and np.isfinite(o[:end]).all() and np.isfinite(o[end + 1:]).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 60])
def test_queries_of_the_largest_size(cuda_ready, q_len, kv):
    # magnitudes of 2^127 over small keys, one of a row's 128 products not zero: the scores are finite
    n = 60
    g = torch.Generator().manual_seed(1)
    k, v = torch.zeros(1, 2, n, 128), torch.randn(1, 2, n, 128, generator=g)
    k[..., 5] = 2.0 ** -60
    paged, pool, table, batch = cached(4, 2, 16, kv, [q_len], [n], k, v)
    q = torch.zeros(q_len, 4, 128)
    q[:, :, 5] = 1.5 * 2.0 ** 127
    q[:, 1, 5] = 2.0 ** 126
    q[:, 3, 5] = -2.0 ** 127
    q = q.to(torch.bfloat16).cuda()
    o, lse = attend(paged, pool, batch, q)
    check_rows(paged, pool, table, q, q_len, n, 0, o, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 3, 200])
@pytest.mark.parametrize("q_power,k_power", [(-100, None), (-120, None), (-90, -60), (100, 60), (126, 100), (60, 110)])
def test_scores_of_zero_from_factors_of_any_size(cuda_ready, q_len, q_power, k_power, kv):
    # keys of zeros (k_power None) or at right angles to the queries: every score is 0, the output the mean of the values
    n = 230
    g = torch.Generator().manual_seed(2)
    k, v = torch.zeros(1, 2, n, 128), torch.randn(1, 2, n, 128, generator=g)
    if k_power is not None:
        k[..., 64:] = torch.randn(1, 2, n, 64, generator=g) * 2.0 ** k_power
    paged, pool, table, batch = cached(4, 2, 16, kv, [q_len], [n], k, v)
    q = torch.zeros(q_len, 4, 128)
    q[..., :64] = torch.rand(q_len, 4, 64, generator=g) * 2.0 ** q_power
    q = q.to(torch.bfloat16).cuda()
    o, lse = attend(paged, pool, batch, q)
    check_rows(paged, pool, table, q, q_len, n, 0, o, lse, rows=sorted({0, q_len // 2, q_len - 1}))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 3, 150])
@pytest.mark.parametrize("power", [-50, 60, 110, 125, 127])
def test_small_queries_over_large_keys_and_the_reverse(cuda_ready, q_len, power, kv):
    # queries of 2^-power over keys of 2^(power - 2): scores of order 1 from factors at either end of f32 (2^-127 is a
    # subnormal)
    n = 180
    g = torch.Generator().manual_seed(power)
    k, v = torch.randn(1, 2, n, 128, generator=g).clamp(-2.5, 2.5) * 2.0 ** (power - 2), torch.randn(1, 2, n, 128, generator=g)
    paged, pool, table, batch = cached(4, 2, 16, kv, [q_len], [n], k, v)
    q = (torch.randn(q_len, 4, 128, generator=g).double() * 2.0 ** -power).to(torch.bfloat16).cuda()
    o, lse = attend(paged, pool, batch, q)
    check_rows(paged, pool, table, q, q_len, n, 0, o, lse, rows=sorted({0, q_len // 2, q_len - 1}))


@pytest.mark.parametrize("q_len", [200, 2])
def test_small_queries_beside_a_tile_of_nan_scales(cuda_ready, q_len):
    # keys 128.. have the NaN scale: queries of 2^-30 that see none of them, in one unit with some that do, get the
    # answer of the others
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(1, 2, 256, 128, generator=g) for _ in range(2))
    paged, pool, table, batch = cached(4, 2, 16, "e4m3", [q_len], [256], k, v)
    for i in table[0][8:16]:
        pool.k_scale.view(torch.uint8)[int(i)] = 255
        pool.v_scale.view(torch.uint8)[int(i)] = 255
    q = (torch.randn(q_len, 4, 128, generator=g) * 2.0 ** -30).to(torch.bfloat16).cuda()
    o, lse = attend(paged, pool, batch, q)
    free = max(0, q_len - 128)
    assert np.isnan(o[free:]).all() and np.isnan(lse[free:]).all()
    if free:
        check_rows(paged, pool, table, q, q_len, 256, 0, o, lse, rows=[0, 1, 40, free - 1])


def bad_rows(pool, table, page, head, bad):
    """Puts what is not finite into value rows of KV head `head`: {key: (dim or None for the whole row, value)}."""
    for j, (d, x) in bad.items():
        at = (int(table[0][j // page]), head, j % page)
        if pool.kv_dtype == "bf16":
            pool.v[at + ((slice(None) if d is None else d),)] = x
        elif d is None:
            pool.v_scale.view(torch.uint8)[at] = 255  # over a payload that is finite
        else:
            pool.v.view(torch.uint8)[at + (d,)] = 0x7F


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hkv,page,q_len,past,visible", [
    (4, 4, 16, 300, 0, 0), (4, 2, 64, 200, 1000, 0), (8, 2, 128, 129, 71, 150), (6, 2, 32, 260, 5000, 5100), (4, 4, 16, 90, 38, 0),
    (4, 2, 16, 3, 300, 0)])
def test_values_that_are_not_finite_reach_those_that_see_them(cuda_ready, hq, hkv, page, q_len, past, visible, wide, kv):
    # bad values in several tiles of the chunk and of what lies before it, each in a dim of its own or in a whole row:
    # a query has NaN or infinity in exactly the dims of the bad values that it sees
    g = torch.Generator().manual_seed(past)
    n = past + q_len
    k, v = (torch.randn(1, hkv, n, 128, generator=g) for _ in range(2))
    if wide:
        v[0, :, 0] *= 2.0 ** -20
    paged, pool, table, batch = cached(hq, hkv, page, kv, [q_len], [n], k, v, visible=[visible])
    q = torch.randn(q_len, hq, 128, generator=g).to(torch.bfloat16).cuda()
    clean = pool_values(pool)
    inf = float("inf")
    bad = {n - 1: (None, float("nan")), past + q_len // 3: (127, inf), past + q_len // 2: (64, float("nan")),
           past + q_len // 2 + 1: (7, -inf), past + 2 * q_len // 3: (7, inf)}
    bad_rows(pool, table, page, hkv - 1, bad)
    o, lse = attend(paged, pool, batch, q)
    kk, vv = (sequence_rows(x, table, 0, n, page) for x in clean)
    group = hq // hkv
    for i in sorted({0, q_len // 3 - 1, q_len // 3, q_len // 2 - 1, q_len // 2, q_len // 2 + 1, 2 * q_len // 3, q_len - 2, q_len - 1}):
        limit = max(visible, past + i + 1)
        hit = np.zeros((hq, 128), dtype=bool)
        for j, (d, _) in bad.items():
            if j < limit:
                hit[-group:, slice(None) if d is None else d] = True
        assert np.array_equal(~np.isfinite(o[i]), hit), i
        ref, l, absv, mag = PG.chunk_attention(as_f64(q[i:i + 1]), kk[:, :limit], vv[:, :limit], limit)
        tol = attend_tolerance(ref, absv, mag, small_weights(kv, vv[:, :limit]))
        assert np.all((np.abs(o[i] - ref[0]) <= tol[0]) | hit), i
        assert np.all(np.abs(lse[i] - l[0]) <= lse_tolerance(l, mag)[0])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_value_that_is_not_finite_costs_no_time(cuda_ready, kv):
    # whole sequences a CTA: one NaN in the last row of each, unseen by all queries but the last
    n, hkv, length, q_len = 38, 4, 6000, 64
    dense = [torch.randn(n, hkv, length, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    q = torch.randn(n * q_len, 16, 128, device="cuda", dtype=torch.bfloat16)
    times = []
    for bad in (False, True):
        if bad:
            dense[1][:, :, -1, 0] = float("nan")
        paged, pool, table, batch = cached(16, hkv, 64, kv, [q_len] * n, [length] * n, *dense)
        attend(paged, pool, batch, q)
        best = float("inf")
        for _ in range(3):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            for _ in range(5):
                o = paged.attend(batch, q, pool)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
        assert torch.isfinite(o.view(n, q_len, 16, 128)[:, :-1]).all()
    assert paged.device_status() == 0 and times[1] < 2 * times[0], times
