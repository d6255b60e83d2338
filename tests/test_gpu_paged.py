"""The paged prefix-KV cache (include/mot_paged.h) against its fp64 oracle:
norm + rotation + cache write of ragged chunks, dense <-> pages, attention of
chunks and single tokens over the pages, in bf16 and e4m3, at odd lengths,
page sizes and head groupings; masks, non-finite values in unseen places, rows
and pages that belong to nobody, refusals, streams, graphs, and the operators
together with the attention layer."""
import math

import numpy as np
import pytest
import torch

from mot_flow_matching_b200 import _abi, synth
from mot_flow_matching_b200.paged import MotPaged, mot_paged_batch_set
from oracle import mot_paged_oracle as PG
from tests.gpu_helpers import ensure_built, make_layer, run_forward, to_dev

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8  # half a step of bf16, relative
EPS, THETA = 1e-6, 1e6


def make_paged(hq, hkv, page, kv, q_len, kv_len, extra=0, **kw):
    ensure_built()
    g = torch.Generator().manual_seed(7)
    w = {n: (1 + 0.1 * torch.randn(128, generator=g)).to(torch.bfloat16).cuda() for n in ("q_norm", "k_norm")}
    used = sum(-(-k // page) for k in kv_len)
    kw = {"max_positions": max(max(kv_len), 1) + extra, "max_batch": len(kv_len), "max_tokens": max(1, sum(q_len)),
          "max_pages": max(1, used) + extra, **kw}
    return MotPaged(w, n_q_heads=hq, n_kv_heads=hkv, page_size=page, kv_dtype=kv, rms_eps=EPS, rope_theta=THETA,
                    **kw), w


def make_table(kv_len, page, seed=0, spare=3):
    used = [-(-k // page) for k in kv_len]
    n = sum(used) + spare
    order = np.random.default_rng(seed).permutation(n)
    table = np.full((len(kv_len), max(max(used), 1)), -1, dtype=np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    return table, n


def as_f64(t):
    return t.float().double().cpu().numpy()


def pool_values(pool):
    """(k, v) [n_pages, Hkv, page, 128] as the values they stand for."""
    if pool.kv_dtype == "bf16":
        return as_f64(pool.k), as_f64(pool.v)
    return (as_f64(pool.k) * as_f64(pool.k_scale)[..., None], as_f64(pool.v) * as_f64(pool.v_scale)[..., None])


def sequence_rows(values, table, b, length, page):
    ids = table[b][: -(-length // page)]
    if length == 0:
        return np.zeros((values.shape[1], 0, 128))
    return np.concatenate([values[i] for i in ids], axis=1)[:, :length]


def fill_pool(paged, n_pages, seed, poison=True):
    """A pool of normal values (unit RMS rows, as normed keys are); with `poison`, what the caller does
    not overwrite stays NaN."""
    pool = paged.new_pool(n_pages)
    if pool.kv_dtype == "bf16":
        pool.k.fill_(float("nan"))
        pool.v.fill_(float("inf"))
    else:
        for t in (pool.k, pool.v, pool.k_scale, pool.v_scale):
            t.view(torch.uint8).fill_(0x7F if t.dtype == torch.float8_e4m3fn else 255)
    return pool


def write_sequences(paged, pool, table, kv_len, seed, scale=1.0):
    """Random sequences into the pages through plain indexing; the rest of the pool is left alone."""
    g = np.random.default_rng(seed)
    page, hkv = paged.cfg.page_size, paged.cfg.n_kv_heads
    for what in ("k", "v"):
        pages = getattr(pool, what)
        for b, n in enumerate(kv_len):
            x = torch.from_numpy(g.normal(size=(n, hkv, 128)) * scale).to(torch.bfloat16)
            j = torch.arange(n)
            ids = torch.from_numpy(table[b])[j // page].long() if n else j
            if pool.kv_dtype == "bf16":
                pages[ids.cuda(), :, (j % page).cuda()] = x.cuda()
            else:
                # spread the rows' scales
                x = (x.double() * torch.exp2(torch.from_numpy(g.integers(-3, 4, size=(n, hkv, 1))).double())).numpy()
                payload, sc = PG.quantise_rows(x)
                raw = torch.from_numpy(payload).float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
                e = torch.from_numpy(np.log2(sc) + 127 if n else sc).to(torch.uint8).cuda()
                pages.view(torch.uint8)[ids.cuda(), :, (j % page).cuda()] = raw
                getattr(pool, what + "_scale").view(torch.uint8)[ids.cuda(), :, (j % page).cuda()] = e


def attend_tolerance(o, absv, mag, small=0.0):
    """Per element. Output: half a bf16 step. Scores: f32 sums of 128 exact products, off by at most
    128 * 2^-24 of the sum of magnitudes, then scaled and shifted (3 roundings), so each weight by twice that
    relative (numerator and denominator). Weights: at most half a bf16 step each where they meet bf16
    values, their sum none. Exponential 2^-21, sums over up to 2^13 keys of f32 adds in a tree of at most 2^8
    sequential steps: 2^-16. All times the weighted mean of |v|. `small`: what small f16 weights add."""
    score = (128 + 3) * 2.0 ** -24 * mag
    return (HALF_BF16 * np.abs(o) + absv * (HALF_BF16 * 1.01 + 2 * score[..., None] + 2.0 ** -16) + small) * (1 + HALF_BF16)


def small_weights(kv, v):
    """Over an 8-bit cache weights are f16 where they meet the values: those below 2^-14 are multiples of 2^-24, off by
    at most 2^-25 (not half a step of themselves, as normal ones are). They are relative to a running max that never
    exceeds the row's, so the row's sum that divides them is at least 1; each multiplies a value counted in units of
    the largest scale so far, 448 of which are at most twice the largest |v|: 2^-25 * 2 max|v| a key."""
    return v.shape[1] * 2.0 ** -24 * np.abs(v).max() if kv == "e4m3" and v.size else 0.0


def lse_tolerance(lse, mag):
    return (128 + 3) * 2.0 ** -24 * mag + 2.0 ** -16 + 2.0 ** -23 * np.abs(lse)


def check_attend(paged, pool, table, q, q_len, kv_len, visible, o, lse, what="", sample=None):
    k, v = pool_values(pool)
    at = 0
    for b, (n, length) in enumerate(zip(q_len, kv_len)):
        rows = range(n) if sample is None else sorted(set(list(range(0, n, max(1, n // sample))) + [n - 1]) if n else [])
        kk, vv = (sequence_rows(x, table, b, length, paged.cfg.page_size) for x in (k, v))
        for i in rows:
            limit_len = length - n + i + 1
            ref, l, absv, mag = PG.chunk_attention(as_f64(q[at + i:at + i + 1]), kk[:, :max(limit_len, visible[b])],
                                                   vv[:, :max(limit_len, visible[b])], max(limit_len, visible[b]))
            got = as_f64(o[at + i:at + i + 1])
            tol = attend_tolerance(ref, absv, mag, small_weights(pool.kv_dtype, vv))
            bad = ~(np.abs(got - ref) <= tol)
            assert not bad.any(), (what, b, i, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / tol)))
            if lse is not None:
                gl = as_f64(lse[at + i:at + i + 1])
                assert np.all(np.abs(gl - l) <= lse_tolerance(l, mag)), (what, b, i, np.abs(gl - l).max())
        at += n


def run_attend(hq, hkv, page, kv, q_len, kv_len, visible=None, seed=0, sample=None, scale=1.0):
    paged, _ = make_paged(hq, hkv, page, kv, q_len, kv_len)
    table, n_pages = make_table(kv_len, page, seed)
    pool = fill_pool(paged, n_pages, seed)
    write_sequences(paged, pool, table, kv_len, seed + 1, scale)
    visible = [0] * len(kv_len) if visible is None else visible
    batch = paged.new_batch()
    batch.set(q_len, kv_len, table, n_pages, visible=visible)
    T = sum(q_len)
    g = torch.Generator().manual_seed(seed + 2)
    q = (torch.randn(T, hq, 128, generator=g) * scale).to(torch.bfloat16).cuda()
    lse = torch.full((T, hq), -7.0, device="cuda")
    o = paged.attend(batch, q, pool, lse=lse)
    torch.cuda.synchronize()
    assert paged.device_status() == 0
    check_attend(paged, pool, table, q, q_len, kv_len, visible, o, lse, (hq, hkv, page, kv, q_len, kv_len), sample)
    return paged, pool, table, batch, q, o, lse


# ------------------------------------------------------------------ attend
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,page", [(4, 2, 64), (8, 2, 16), (4, 4, 128), (32, 8, 64), (16, 1, 32), (6, 2, 64)])
def test_attend_single_tokens(cuda_ready, hq, hkv, page, kv):
    kv_len = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 400, 1201]
    run_attend(hq, hkv, page, kv, [1] * len(kv_len), kv_len, seed=hq + page)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len,kv_len,visible", [
    ([1], [1], None),
    ([5], [5], None),
    ([3, 0, 1, 2], [10, 7, 1, 130], None),
    ([9, 31, 2], [9, 50, 400], [0, 50, 200]),
    ([33], [290], [290]),
    ([64, 1, 65], [64, 257, 200], [0, 0, 100]),
    ([130, 128, 127], [130, 513, 300], None),
    ([257], [700], [650]),
    ([300, 260], [300, 900], [300, 900]),
])
def test_attend_chunks(cuda_ready, q_len, kv_len, visible, kv):
    run_attend(4, 2, 64, kv, q_len, kv_len, visible, seed=len(q_len) + sum(q_len), sample=24)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,page", [(4, 4, 16), (16, 2, 32), (6, 2, 128), (20, 1, 64)])
def test_attend_chunks_other_groups_and_pages(cuda_ready, hq, hkv, page, kv):
    run_attend(hq, hkv, page, kv, [70, 1, 19, 200], [95, 300, 19, 1000], [0, 0, 0, 900], seed=hq, sample=12)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attend_long_cache(cuda_ready, kv):
    run_attend(8, 2, 64, kv, [1, 3, 40], [20011, 9000, 12345], [0, 0, 100], seed=3, sample=6)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attend_large_scores(cuda_ready, kv):
    # score spread of some hundreds: the running max moves many times
    run_attend(4, 2, 64, kv, [1, 6, 150], [700, 300, 500], seed=5, sample=20, scale=4.0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attend_zero_queries_give_the_mean(cuda_ready, kv):
    paged, pool, table, batch, q, _, _ = run_attend(4, 2, 32, kv, [1, 40], [100, 77], [0, 77])
    lse = torch.empty(41, 4, device="cuda")
    o = paged.attend(batch, torch.zeros_like(q), pool, lse=lse)
    check_attend(paged, pool, table, torch.zeros_like(q), [1, 40], [100, 77], [0, 77], o, lse)
    assert abs(lse[0, 0].item() - math.log(100)) < 1e-5


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("what,where", [("v", 0), ("v", 12), ("k", 12), ("k", 19), ("v", 19)])
@pytest.mark.parametrize("past", [0, 300])
def test_attend_unseen_values_have_no_influence(cuda_ready, what, where, kv, past):
    # a NaN or infinity at chunk token `where`: the queries before it are as without it -- bit for bit but for the
    # dims of a value that is not finite, whose sum may be taken again without it, in another order, and is held
    # to the oracle -- and those from it on are not finite (keys: every dim; values: that dim, or the row in 8 bits)
    q_len, kv_len = [20], [past + 20]
    paged, pool, table, batch, q, o, _ = run_attend(4, 2, 16, kv, q_len, kv_len, seed=11)
    j = past + where
    page_id, row = int(table[0][j // 16]), j % 16
    t = getattr(pool, what)
    if kv == "bf16":
        t[page_id, 1, row, 5] = float("nan") if what == "k" else float("inf")
    else:
        t.view(torch.uint8)[page_id, 1, row] = 0x7F
        getattr(pool, what + "_scale").view(torch.uint8)[page_id, 1, row] = 255
    o2 = paged.attend(batch, q, pool)
    torch.cuda.synchronize()
    assert torch.equal(o2[:, :2].view(torch.int16), o[:, :2].view(torch.int16))  # KV head 0
    same = [d for d in range(128) if what == "k" or (kv == "bf16" and d != 5)]
    assert torch.equal(o2[:where, 2:, same].view(torch.int16), o[:where, 2:, same].view(torch.int16))
    if where:
        k, v = (sequence_rows(x, table, 0, past + where, 16) for x in pool_values(pool))
        ref, _, absv, mag = PG.chunk_attention(as_f64(q[:where]), k, v, 0)
        fine = np.where(np.isfinite(v), v, 0.0)
        assert np.all(np.abs(as_f64(o2[:where]) - ref) <= attend_tolerance(ref, absv, mag, small_weights(kv, fine)))
    hit = o2[where:, 2:]
    assert not torch.isfinite(hit[..., 5]).any()
    if kv == "bf16" and what == "v":
        assert torch.equal(hit[..., :5].view(torch.int16), o[where:, 2:, :5].view(torch.int16))
    else:
        assert not torch.isfinite(hit).any()


@pytest.mark.parametrize("q_len", [256, 2])
def test_attend_tile_of_nan_scales(cuda_ready, q_len):
    # keys 128.. all have the NaN scale, over payloads that are finite (a pool need not come from append or store):
    # queries that see one of them get NaN, the others what the oracle says
    paged, pool, table, batch, q, _, _ = run_attend(4, 2, 16, "e4m3", [q_len], [256], seed=4, sample=4)
    for i in table[0][8:16]:
        pool.k_scale.view(torch.uint8)[int(i)] = 255
        pool.v_scale.view(torch.uint8)[int(i)] = 255
    lse = torch.empty(q_len, 4, device="cuda")
    o = paged.attend(batch, q, pool, lse=lse)
    free = max(0, q_len - 128)
    assert torch.isnan(o[free:]).all() and torch.isnan(lse[free:]).all()
    if free:
        k, v = (sequence_rows(x, table, 0, 128, 16) for x in pool_values(pool))
        ref, l, absv, mag = PG.chunk_attention(as_f64(q[:free]), k, v, 0)
        assert np.all(np.abs(as_f64(o[:free]) - ref) <= attend_tolerance(ref, absv, mag, small_weights("e4m3", v)))
        assert np.all(np.abs(as_f64(lse[:free]) - l) <= lse_tolerance(l, mag))


def test_attend_is_deterministic_and_leaves_its_inputs(cuda_ready):
    paged, pool, table, batch, q, o, lse = run_attend(32, 8, 64, "bf16", [1, 200, 1], [3000, 900, 17], sample=2)
    k0, v0, q0 = pool.k.clone(), pool.v.clone(), q.clone()
    for _ in range(5):
        lse2 = torch.empty_like(lse)
        o2 = paged.attend(batch, q, pool, lse=lse2)
        assert torch.equal(o2.view(torch.int16), o.view(torch.int16)) and torch.equal(lse2, lse)
    for a, b in ((pool.k, k0), (pool.v, v0), (q, q0)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows_per_seq", [1, 2, 3, 4, 6, 7, 8, 9])
def test_attend_around_the_choice_of_kernel(cuda_ready, rows_per_seq, kv):
    # 4 heads a group: 4 to 36 query rows, few and many sequences
    run_attend(8, 2, 32, kv, [rows_per_seq], [300], seed=rows_per_seq)
    kv_len = [rows_per_seq + 37 * i for i in range(40)]
    run_attend(8, 2, 32, kv, [rows_per_seq] * 40, kv_len, seed=rows_per_seq, sample=2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attend_scales_far_apart(cuda_ready, kv):
    # rows whose magnitudes span 2^-40 .. 2^20 within a tile (8-bit scales far from the tile's largest)
    q_len, kv_len = [1, 60], [200, 300]
    paged, _ = make_paged(4, 2, 16, kv, q_len, kv_len)
    table, n_pages = make_table(kv_len, 16, 3)
    pool = fill_pool(paged, n_pages, 0)
    g = np.random.default_rng(1)
    dense = []
    for what in range(2):
        e = g.integers(-40, -3, size=(2, 2, 300, 1)) if what == 0 else g.integers(-40, 20, size=(2, 2, 300, 1))
        dense.append(torch.from_numpy(g.normal(size=(2, 2, 300, 128)) * np.exp2(e)).to(torch.bfloat16).cuda())
    batch = paged.new_batch()
    batch.set(q_len, kv_len, table, n_pages)
    paged.store(batch, *dense, pool)
    q = torch.randn(61, 4, 128).to(torch.bfloat16).cuda()
    lse = torch.empty(61, 4, device="cuda")
    o = paged.attend(batch, q, pool, lse=lse)
    check_attend(paged, pool, table, q, q_len, kv_len, [0, 0], o, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attend_query_rows_that_are_not_finite_stay_alone(cuda_ready, kv):
    paged, pool, table, batch, q, o, lse = run_attend(4, 2, 32, kv, [1, 70], [100, 300], seed=21)
    q2 = q.clone()
    q2[0, 1, 3] = float("nan")
    q2[40, 2, 7] = float("inf")
    o2 = paged.attend(batch, q2, pool)
    bad = torch.zeros(71, 4, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[40, 2] = True
    assert torch.isnan(o2[bad]).all()
    assert torch.equal(o2[~bad].view(torch.int16), o[~bad].view(torch.int16))


def test_attend_and_load_into_16_byte_aligned_outputs(cuda_ready):
    # outputs that start in the middle of a 32-byte sector
    for kv in ("bf16", "e4m3"):
        paged, pool, table, batch, q, o, _ = run_attend(8, 2, 64, kv, [1, 100, 9], [70, 300, 600], seed=9, sample=3)
        buf = torch.zeros(o.numel() + 16, dtype=torch.bfloat16, device="cuda")
        o2 = buf[8:8 + o.numel()].view(o.shape)
        assert o2.data_ptr() % 32 == 16
        paged.attend(batch, q, pool, o=o2)
        assert torch.equal(o2.view(torch.int16), o.view(torch.int16)) and (buf[:8] == 0).all() and (buf[-8:] == 0).all()
        k, v = paged.load(batch, pool)
        kb = torch.zeros(k.numel() + 16, dtype=torch.bfloat16, device="cuda")
        k2 = kb[8:8 + k.numel()].view(k.shape)
        k2.copy_(k)
        paged.load(batch, pool, k=k2, v=v.clone())
        assert torch.equal(k2.view(torch.int16), k.view(torch.int16)) and (kb[:8] == 0).all() and (kb[-8:] == 0).all()
        p2 = paged.new_pool(pool.k.shape[0])
        for a, b in ((p2.k, pool.k), (p2.v, pool.v), (p2.k_scale, pool.k_scale), (p2.v_scale, pool.v_scale)):
            if a is not None:
                a.view(torch.uint8).copy_(b.view(torch.uint8))
        b0 = paged.new_batch()
        b0.set([0, 0, 0], [70, 300, 600], table, pool.k.shape[0])
        paged.store(b0, k2, v, p2)
        ka, va = paged.load(b0, p2)
        assert torch.equal(ka[2].view(torch.int16), k[2].view(torch.int16))


# ------------------------------------------------------------------ append
def check_append(paged, w, pool, before, table, qkv, q_len, kv_len, q):
    c = paged.cfg
    page = c.page_size
    x = as_f64(qkv).reshape(-1, c.n_q_heads + 2 * c.n_kv_heads, 128)
    gains = {n: as_f64(w[n]) for n in w}
    after = [t.view(torch.uint8).cpu().numpy() for t in (pool.k, pool.v, pool.k_scale, pool.v_scale) if t is not None]
    untouched = [a.copy() for a in before]
    kval, vval = pool_values(pool)
    at = 0
    for b, (n, length) in enumerate(zip(q_len, kv_len)):
        if n == 0:
            continue
        pos = np.arange(length - n, length)
        qr, kr, vr = PG.chunk_qkv(x[at:at + n], pos, gains["q_norm"], gains["k_norm"], c.n_q_heads, c.n_kv_heads, EPS,
                                  THETA)
        # f32: sum of 128 squares (2^-17 relative on the norm, halved by the root), four roundings, table 2^-24:
        # 2^-16 of the rotated pair's length
        def tau(r):
            pair = np.hypot(r[..., :64], r[..., 64:])
            return 2.0 ** -16 * np.concatenate([pair, pair], -1)

        got = as_f64(q[at:at + n])
        assert np.all(np.abs(got - qr) <= HALF_BF16 * (np.abs(qr) + tau(qr)) + tau(qr))
        ids = table[b][pos // page]
        kg, vg = kval[ids, :, pos % page], vval[ids, :, pos % page]
        if pool.kv_dtype == "bf16":
            assert np.all(np.abs(kg - kr) <= HALF_BF16 * (np.abs(kr) + tau(kr)) + tau(kr))
            assert np.array_equal(vg, vr)
        else:
            ks, vs = (as_f64(t)[ids, :, pos % page] for t in (pool.k_scale, pool.v_scale))
            payload, scale = PG.quantise_rows(vr)
            assert np.array_equal(vs, scale) and np.array_equal(vg, payload * scale[..., None])
            _, scale = PG.quantise_rows(kr)
            near = np.abs(np.abs(kr).max(-1) / (448 * np.minimum(scale, ks)) - 1) < 2.0 ** -15
            assert np.all((ks == scale) | near)
            step = np.maximum(2.0 ** -4 * (np.abs(kr) + tau(kr)), 2.0 ** -10 * ks[..., None])
            assert np.all(np.abs(kg - kr) <= step + tau(kr))
        for a, u in zip(after, untouched):
            u[ids, :, pos % page] = a[ids, :, pos % page]
        at += n
    for a, u in zip(after, untouched):
        assert np.array_equal(a, u)  # nothing else in the pool moved


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,page,q_len,kv_len", [
    (4, 2, 64, [1], [1]),
    (32, 8, 64, [1], [401]),
    (4, 2, 16, [1, 0, 5, 33], [17, 9, 5, 300]),
    (6, 2, 32, [31, 2], [31, 1000]),
    (16, 1, 128, [130, 129], [130, 500]),
    (32, 8, 64, [400, 231], [400, 631]),
    (5, 1, 16, [3], [3]),
    (32, 8, 64, [1000, 0, 701], [1100, 3, 701]),  # a warp a token
    (6, 2, 32, [3000, 1900], [3000, 2000]),
    (7, 7, 16, [700], [701]),
])
def test_append(cuda_ready, hq, hkv, page, q_len, kv_len, kv):
    paged, w = make_paged(hq, hkv, page, kv, q_len, kv_len)
    table, n_pages = make_table(kv_len, page, 4)
    pool = fill_pool(paged, n_pages, 0)
    before = [t.view(torch.uint8).cpu().numpy().copy() for t in (pool.k, pool.v, pool.k_scale, pool.v_scale) if t is not None]
    T = sum(q_len)
    g = torch.Generator().manual_seed(T)
    qkv = (torch.randn(T, (hq + 2 * hkv) * 128, generator=g) * 1.28).to(torch.bfloat16)
    qkv[0, -256:-128] = 0  # a row of zeros
    qkv = qkv.cuda()
    batch = paged.new_batch()
    batch.set(q_len, kv_len, table, n_pages)
    q = paged.append(batch, qkv, pool)
    torch.cuda.synchronize()
    check_append(paged, w, pool, before, table, qkv, q_len, kv_len, q)


def test_append_non_finite_rows_become_nan_rows(cuda_ready):
    paged, _ = make_paged(4, 2, 16, "e4m3", [3], [3])
    pool = paged.new_pool(1)
    for t in (pool.k, pool.v, pool.k_scale, pool.v_scale):
        t.view(torch.uint8).zero_()
    qkv = torch.randn(3, 8 * 128).to(torch.bfloat16)
    qkv[1, 6 * 128 + 3] = float("inf")   # v head 0 of token 1
    qkv[2, 5 * 128 + 3] = float("nan")   # k head 1 of token 2
    batch = paged.new_batch()
    batch.set([3], [3], [[0]], 1)
    paged.append(batch, qkv.cuda(), pool)
    k, v = pool_values(pool)
    nk, nv = np.isnan(k[0, :, :3]).all(-1), np.isnan(v[0, :, :3]).all(-1)
    assert nk.tolist() == [[False, False, False], [False, False, True]]
    assert nv.tolist() == [[False, True, False], [False, False, False]]
    assert np.isfinite(k[0, 0, :3]).all() and np.isfinite(v[0, 1, :3]).all()


# ------------------------------------------------------------------ store, load
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hkv,page,kv_len,rows", [
    (2, 64, [1], 1), (2, 16, [16, 0, 33, 1], 40), (8, 64, [400, 231], 400), (1, 128, [129, 127, 128], 200),
    (3, 32, [500] * 5, 513)])
def test_store_then_load(cuda_ready, hkv, page, kv_len, rows, kv):
    paged, _ = make_paged(2 * hkv, hkv, page, kv, [0] * len(kv_len), kv_len)
    table, n_pages = make_table(kv_len, page, 9)
    pool = fill_pool(paged, n_pages, 0)
    before = [t.view(torch.uint8).cpu().numpy().copy() for t in (pool.k, pool.v, pool.k_scale, pool.v_scale) if t is not None]
    g = torch.Generator().manual_seed(rows)
    dense = [torch.randn(len(kv_len), hkv, rows, 128, generator=g).to(torch.bfloat16) for _ in range(2)]
    dense[1][0, 0, 0] = 0
    dense[0][-1, 0, -1] = float("nan")
    batch = paged.new_batch()
    batch.set([0] * len(kv_len), kv_len, table, n_pages)
    paged.store(batch, dense[0].cuda(), dense[1].cuda(), pool)
    out = [torch.full_like(d, 3.0).cuda() for d in dense]
    paged.load(batch, pool, *out)
    torch.cuda.synchronize()
    for d, got in zip(dense, out):
        for b, n in enumerate(kv_len):
            x = d[b, :, :n].double().numpy()
            if kv == "e4m3":
                payload, scale = PG.quantise_rows(x)
                x = payload * scale[..., None]
            assert np.array_equal(as_f64(got[b, :, :n]), x, equal_nan=True)
            assert (got[b, :, n:] == 3.0).all()  # rows behind the sequence left as they were
    after = [t.view(torch.uint8).cpu().numpy() for t in (pool.k, pool.v, pool.k_scale, pool.v_scale) if t is not None]
    for a, old in zip(after, before):
        for b, n in enumerate(kv_len):
            for i in range(-(-n // page)):
                live = min(page, n - i * page)
                old[table[b][i], :, :live] = a[table[b][i], :, :live]
        assert np.array_equal(a, old)


# ------------------------------------------------------------------ together
def test_chunks_through_pages_equal_the_prefix_layer(cuda_ready):
    # a 300-token prompt encoded in chunks of 130, 1 and 169 tokens over the pages against the prefix layer's one
    # pass (which keeps q and the projections in f32 / f16; here they pass through bf16 twice)
    dims = synth.LayerDims(hidden=512, n_q_heads=4, n_kv_heads=2)
    wl = synth.Workload("prefix", 1, 300, 0, 0, 0.0, dims=dims)
    t = synth.make_inputs(wl, 8100, with_dy=False)
    td = to_dev({k: t[k] for k in ("x", "w_q", "w_k", "w_v", "w_o", "q_norm", "k_norm")})
    layer = make_layer(wl, td)
    y32 = torch.empty(1, 300, 512, device="cuda")
    _, kc, vc = layer.prefix_forward(td["x"], [300], y_f32=y32)
    paged = MotPaged(td, n_q_heads=4, n_kv_heads=2, page_size=16, rms_eps=dims.rms_eps, rope_theta=dims.rope_theta,
                     max_positions=300, max_batch=1, max_tokens=300, max_pages=19)
    pool, batch = paged.new_pool(24), paged.new_batch()
    table, _ = make_table([300], 16, 2, spare=5)
    w = torch.cat([td["w_q"], td["w_k"], td["w_v"]]).float()
    outs = []
    for a, b in ((0, 130), (130, 131), (131, 300)):
        qkv = (td["x"][0, a:b].float() @ w.T).to(torch.bfloat16)
        batch.set([b - a], [b], table[:, : -(-b // 16)], 24)
        q = paged.append(batch, qkv, pool)
        o = paged.attend(batch, q, pool)
        outs.append(o.float().reshape(b - a, 512) @ td["w_o"].float().T)
    y = torch.cat(outs)
    k, v = paged.load(batch, pool)
    torch.cuda.synchronize()
    # Cache: rounding the projection moves an element by at most 2^-8 of it and the row's norm by as much, so the
    # rotated pair by 2 * 2^-8 of its length; then both sides round once more (2^-8 each). f32 sums: 2^-10 of the RMS.
    kr, vr = as_f64(kc), as_f64(vc)
    pair = np.hypot(kr[..., :64], kr[..., 64:])
    noise = 2.0 ** -10
    assert np.all(np.abs(as_f64(k) - kr) <= 4.1 * HALF_BF16 * np.concatenate([pair, pair], -1) + noise)
    assert np.all(np.abs(as_f64(v) - vr) <= 2.1 * HALF_BF16 * np.abs(vr) + noise * np.sqrt(np.mean(vr ** 2)))
    # y, row by row (rows differ in size: the first see few keys): a bf16 rounding is 1.65e-3 rms relative. Scores
    # take four of them (q and k, each twice; scores have unit variance): 3.3e-3 rms on each weight; values and
    # outputs one each: sqrt(3.3^2 + 1.65^2 + 1.65^2) e-3 = 4.0e-3. 1200 head rows reach 4.5 sigma: 1.8e-2 < 2e-2.
    yr = y32[0].double().cpu().numpy()
    err = np.linalg.norm(y.double().cpu().numpy() - yr, axis=-1) / np.linalg.norm(yr, axis=-1)
    assert err.max() <= 2e-2 and np.sqrt(np.mean(err ** 2)) <= 8e-3, (err.max(), np.sqrt(np.mean(err ** 2)))
    layer.close()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_cache_through_pages_feeds_the_layer(cuda_ready, kv):
    # prefix layer -> store -> load -> gen layer: bit for bit the layer over the dense cache (bf16), or over the
    # cache rounded to e4m3 rows
    dims = synth.LayerDims(hidden=512, n_q_heads=4, n_kv_heads=2)
    wl = synth.Workload("gen", 2, 200, 77, 16, 16.0, dims=dims)
    t = synth.make_inputs(wl, 8200, with_dy=False)
    td = to_dev(t)
    lengths = [77, 40]
    paged, _ = make_paged(4, 2, 32, kv, [0, 0], lengths)
    table, n_pages = make_table(lengths, 32)
    pool, batch = paged.new_pool(n_pages), paged.new_batch()
    batch.set([0, 0], lengths, table, n_pages)
    paged.store(batch, td["k_cache"], td["v_cache"], pool)
    kl, vl = paged.load(batch, pool)
    ref = dict(td)
    if kv == "e4m3":
        for n in ("k_cache", "v_cache"):
            payload, scale = PG.quantise_rows(t[n].double().numpy())
            ref[n] = torch.from_numpy(payload * scale[..., None]).to(torch.bfloat16).cuda()
    got = dict(td, k_cache=kl, v_cache=vl)
    layer = make_layer(wl, td)
    y, y32, _, s = run_forward(layer, ref, prefix_len=lengths)
    y2, y32b, _, s2 = run_forward(layer, got, prefix_len=lengths)
    assert s == s2 == 0 and torch.equal(y32.view(torch.int32), y32b.view(torch.int32))
    layer.close()


def test_append_then_attend_in_a_graph_follows_the_batch(cuda_ready):
    # one captured step replayed over growing sequences (two single tokens and a chunk)
    hq, hkv, page = 8, 2, 16
    q_len, kv0 = [1, 1, 21], [30, 700, 21]
    steps = 3
    final = [k + q * (steps - 1) for k, q in zip(kv0, q_len)]
    paged, w = make_paged(hq, hkv, page, "e4m3", q_len, final)
    table, n_pages = make_table(final, page, 5)
    g = torch.Generator().manual_seed(3)
    qkvs = [torch.randn(23, 12 * 128, generator=g).to(torch.bfloat16).cuda() for _ in range(steps)]
    pools = []
    for _ in range(2):
        pool = fill_pool(paged, n_pages, 0)
        write_sequences(paged, pool, table, [k - q for k, q in zip(kv0, q_len)], 1)
        pools.append(pool)
    lens = [[k + q * i for k, q in zip(kv0, q_len)] for i in range(steps)]
    eager = []
    batch = paged.new_batch()
    for i in range(steps):
        batch.set(q_len, lens[i], table, n_pages)
        q = paged.append(batch, qkvs[i], pools[0])
        eager.append((q, paged.attend(batch, q, pools[0])))
    side = torch.cuda.Stream()
    b2 = paged.new_batch()
    x = qkvs[0].clone()
    q, o = torch.empty_like(eager[0][0]), torch.empty_like(eager[0][1])
    ws = b2.workspace()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b2.set(q_len, lens[0], table, n_pages)
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            paged.append(b2, x, pools[1], q=q)
            paged.attend(b2, q, pools[1], o=o, workspace=ws)
            with pytest.raises(_abi.MotError):  # not while capturing
                mot_paged_batch_set(b2.handle, q_len, lens[0], table, n_pages)
        for i in range(steps):
            b2.set(q_len, lens[i], table, n_pages)
            x.copy_(qkvs[i])
            graph.replay()
            side.synchronize()
            assert torch.equal(q.view(torch.int16), eager[i][0].view(torch.int16))
            assert torch.equal(o.view(torch.int16), eager[i][1].view(torch.int16))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_copies_captured_empty_follow_the_batch(cuda_ready, kv):
    # store and load captured while every sequence is empty, replayed over sequences that are not
    paged, _ = make_paged(4, 2, 16, kv, [0, 0], [40, 7])
    table, n_pages = make_table([40, 7], 16, 2)
    pool = fill_pool(paged, n_pages, 0)
    k, v = (torch.randn(2, 2, 40, 128).to(torch.bfloat16).cuda() for _ in range(2))
    k2, v2 = torch.full_like(k, -3.0), torch.full_like(v, -3.0)
    batch, side = paged.new_batch(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        batch.set([0, 0], [0, 0], table, n_pages)
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            paged.store(batch, k, v, pool)
            paged.load(batch, pool, k2, v2)
        graph.replay()
        side.synchronize()
        assert (k2 == -3).all() and (v2 == -3).all()
        batch.set([0, 0], [40, 7], table, n_pages)
        graph.replay()
        side.synchronize()
    for x, y, what in ((k, k2, 0), (v, v2, 1)):
        for b, n in enumerate((40, 7)):
            assert np.array_equal(as_f64(y[b, :, :n]), sequence_rows(pool_values(pool)[what], table, b, n, 16))
            if kv == "bf16":
                assert torch.equal(x[b, :, :n].view(torch.int16), y[b, :, :n].view(torch.int16))
        assert (y[1, :, 7:] == -3).all()


def test_load_refuses_one_tensor_for_both(cuda_ready):
    paged, _ = make_paged(4, 2, 16, "bf16", [1], [20])
    batch, pool = paged.new_batch(), paged.new_pool(2)
    batch.set([1], [20], [[0, 1]], 2)
    k = torch.empty(1, 2, 20, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(_abi.MotError) as e:
        paged.load(batch, pool, k, k)
    assert e.value.status == _abi.MOT_ERR_INVALID_ARGUMENT


def test_stream_order_without_synchronisation(cuda_ready):
    # set, append, attend, load issued back to back on a stream of its own equal the synchronised run
    hq, hkv, page, q_len, kv_len = 8, 2, 32, [40, 1], [300, 1000]
    paged, w = make_paged(hq, hkv, page, "bf16", q_len, kv_len)
    table, n_pages = make_table(kv_len, page)
    qkv = torch.randn(41, 12 * 128).to(torch.bfloat16).cuda()
    pools = []
    for _ in range(2):
        p = fill_pool(paged, n_pages, 0)
        write_sequences(paged, p, table, [260, 999], 2)
        pools.append(p)
    batch = paged.new_batch()
    batch.set(q_len, kv_len, table, n_pages)
    torch.cuda.synchronize()
    q = paged.append(batch, qkv, pools[0])
    torch.cuda.synchronize()
    o = paged.attend(batch, q, pools[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b2 = paged.new_batch()
        for _ in range(20):
            b2.set(q_len, kv_len, table, n_pages)
            q2 = paged.append(b2, qkv, pools[1])
            o2 = paged.attend(b2, q2, pools[1])
            k2, v2 = paged.load(b2, pools[1])
    side.synchronize()
    assert torch.equal(o2.view(torch.int16), o.view(torch.int16))
    k, v = paged.load(batch, pools[0])
    for a, b in ((k, k2), (v, v2)):
        for i, n in enumerate(kv_len):
            assert torch.equal(a[i, :, :n].view(torch.int16), b[i, :, :n].view(torch.int16))


def test_batches_set_in_turn_without_synchronisation(cuda_ready):
    # one batch object described anew before every call, different lengths, kinds of kernels and pages each time, and
    # two batches on one workspace: as each by itself
    paged, _ = make_paged(8, 2, 16, "bf16", [64, 64, 64], [500, 500, 500], max_batch=3)
    table, n_pages = make_table([500, 500, 500], 16, 1)
    pool = fill_pool(paged, n_pages, 0)
    write_sequences(paged, pool, table, [500, 500, 500], 3)
    cases = [([1, 1, 1], [500, 20, 3]), ([64, 1, 30], [64, 499, 77]), ([3, 0, 0], [3, 0, 0]), ([5, 64, 0], [400, 500, 9]),
             ([1, 2, 1], [17, 300, 450])]
    qs = [torch.randn(sum(q), 8, 128).to(torch.bfloat16).cuda() for q, _ in cases]
    alone = []
    for (q_len, kv_len), q in zip(cases, qs):
        b = paged.new_batch()
        b.set(q_len, kv_len, table, n_pages)
        alone.append(paged.attend(b, q, pool))
        torch.cuda.synchronize()
    one, two = paged.new_batch(), paged.new_batch()
    ws = one.workspace()
    got = []
    for turn in range(8):
        for i, ((q_len, kv_len), q) in enumerate(zip(cases, qs)):
            b = (one, two)[(turn + i) & 1]
            b.set(q_len, kv_len, table, n_pages)
            got.append((i, paged.attend(b, q, pool, workspace=ws), paged.load(b, pool)[0]))
    torch.cuda.synchronize()
    for i, o, k in got:
        assert torch.equal(o.view(torch.int16), alone[i].view(torch.int16)), i
        for s, n in enumerate(cases[i][1]):
            ref = sequence_rows(as_f64(pool.k), table, s, n, 16)
            assert np.array_equal(as_f64(k[s, :, :n]), ref)


# ------------------------------------------------------------------ refusals
def test_refusals(cuda_ready):
    paged, _ = make_paged(4, 2, 16, "bf16", [4, 4], [40, 40])
    batch, pool = paged.new_batch(), paged.new_pool(6)
    ok = dict(q_len=[4, 4], kv_len=[40, 40], table=[[0, 1, 2], [3, 4, 5]], n_pages=6)
    inv, shape = _abi.MOT_ERR_INVALID_ARGUMENT, _abi.MOT_ERR_UNSUPPORTED_SHAPE
    for change, status in ((dict(table=[[0, 1, 6], [3, 4, 5]]), inv), (dict(table=[[0, 1, -1], [3, 4, 5]]), inv),
                           (dict(table=[[0, 1], [3, 4]]), inv), (dict(q_len=[-1, 4]), inv), (dict(q_len=[41, 4]), inv),
                           (dict(visible=[41, 0]), inv), (dict(visible=[0, -1]), inv), (dict(n_pages=0), inv),
                           (dict(kv_len=[40, 41]), shape), (dict(q_len=[5, 4]), shape),
                           (dict(q_len=[1] * 3, kv_len=[1] * 3, table=[[0], [1], [2]]), shape)):
        with pytest.raises(_abi.MotError) as e:
            batch.set(**{**ok, **change})
        assert e.value.status == status, change
        with pytest.raises(ValueError):  # a refused set leaves nothing to run
            paged.attend(batch, torch.zeros(8, 4, 128, dtype=torch.bfloat16, device="cuda"), pool)
    qkv = torch.randn(8, 8 * 128).to(torch.bfloat16).cuda()
    dense = torch.randn(2, 2, 40, 128).to(torch.bfloat16).cuda()
    # the same page twice: read, but not written
    batch.set([4, 4], [40, 40], [[0, 1, 2], [0, 4, 5]], 6)
    paged.append(batch, qkv, pool)
    with pytest.raises(_abi.MotError):
        paged.store(batch, dense, dense, pool)
    batch.set([4, 4], [40, 40], [[0, 1, 2], [3, 4, 2]], 6)
    with pytest.raises(_abi.MotError):
        paged.append(batch, qkv, pool)
    batch.set(**ok)
    with pytest.raises(_abi.MotError):  # a pool with fewer pages than the table was checked against
        paged.append(batch, qkv, paged.new_pool(5))
    with pytest.raises(_abi.MotError):  # dense rows shorter than a sequence
        paged.store(batch, dense[:, :, :39].contiguous(), dense[:, :, :39].contiguous(), pool)
    q = torch.randn(8, 4, 128).to(torch.bfloat16).cuda()
    with pytest.raises(_abi.MotError) as e:
        paged.attend(batch, q, pool, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == _abi.MOT_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(_abi.MotError) as e:
        big = torch.empty(8 * 4 * 128 + 8, dtype=torch.bfloat16, device="cuda")
        paged.attend(batch, big[1:1 + 8 * 4 * 128].view(8, 4, 128), pool)
    assert e.value.status == _abi.MOT_ERR_ALIGNMENT
    with pytest.raises(_abi.MotError):
        paged.attend(batch, q, pool, o=q)  # over its own input
    for bad in (q[:7], q.float(), q.cpu(), q.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(ValueError):
            paged.attend(batch, bad, pool)
    other, _ = make_paged(4, 2, 32, "bf16", [1], [1])
    with pytest.raises(ValueError):
        other.attend(batch, q, pool)
    with pytest.raises(ValueError):
        paged.attend(batch, q, other.new_pool(9))
    o = paged.attend(batch, paged.append(batch, qkv, pool), pool)  # still usable
    torch.cuda.synchronize()
    assert paged.device_status() == 0 and o.shape == (8, 4, 128)


def test_empty_batches(cuda_ready):
    paged, _ = make_paged(4, 2, 16, "bf16", [0, 0], [0, 9])
    batch, pool = paged.new_batch(), paged.new_pool(2)
    batch.set([0, 0], [0, 9], [[-1], [1]], 2)
    q = paged.append(batch, torch.empty(0, 1024, dtype=torch.bfloat16, device="cuda"), pool)
    o = paged.attend(batch, q, pool)
    assert o.shape == (0, 4, 128)
    batch.set([0, 0], [0, 0], torch.empty(2, 0, dtype=torch.int32), 2)
    k, v = paged.load(batch, pool)
    paged.store(batch, k, v, pool)
    torch.cuda.synchronize()
    assert k.shape == (2, 2, 0, 128)
