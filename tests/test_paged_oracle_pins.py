"""Pins of the paged-cache oracle (oracle/mot_paged_oracle.py): the e4m3 row
against torch's float8 conversion and closed forms, the chunk's norm and
rotation against the whole sequence's, the chunk's attention against torch's
scaled_dot_product_attention and against one pass over the whole sequence."""
import numpy as np
import pytest
import torch

from oracle import mot_attn_oracle as O
from oracle import mot_paged_oracle as PG
from oracle import mot_prefix_oracle as PO


def test_round_to_e4m3_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    codes = codes[np.isfinite(codes)]
    assert np.array_equal(PG.round_to_e4m3(codes), codes)  # every e4m3 value stays
    g = np.random.default_rng(0)
    x = np.concatenate([g.uniform(-448, 448, 4000), g.normal(0, 2.0 ** -7, 4000),
                        (codes[:-1] + codes[1:]) / 2]).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(PG.round_to_e4m3(x), ref)


def test_scale_is_the_smallest_power_of_two_that_fits():
    rows = np.zeros((8, 128))
    amax = [448.0, np.nextafter(448.0, 449), 1.0, 0.0, 1e-30, 3.3e38, 1.75, np.nextafter(1.75, 2)]
    rows[:, 5] = amax
    payload, scale = PG.quantise_rows(rows)
    assert scale[0] == 1.0 and scale[1] == 2.0 and scale[3] == 2.0 ** -64 and scale[4] == 2.0 ** -64
    assert scale[6] == 2.0 ** -8 and scale[7] == 2.0 ** -7
    for a, s in zip(amax, scale):
        assert a <= 448 * s and (s == 2.0 ** -64 or a > 224 * s)
    assert payload[0, 5] == 448 and payload[3, 5] == 0
    bad = np.zeros((2, 128))
    bad[0, 0], bad[1, 3] = np.inf, np.nan
    payload, scale = PG.quantise_rows(bad)
    assert np.isnan(payload).all() and np.isnan(scale).all()


def test_stored_values_are_exact_in_bf16():
    x = np.random.default_rng(1).normal(size=(64, 128)) * np.exp2(np.arange(64) - 32)[:, None]
    payload, scale = PG.quantise_rows(x)
    y = payload * scale[:, None]
    assert np.array_equal(O.round_to_bf16(y), y)
    # half a step of a 4-bit significand, or of the subnormals
    assert np.all(np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale[:, None]))


def test_chunk_rows_are_the_whole_sequences():
    g = np.random.default_rng(2)
    qkv, qg, kg = g.normal(size=(9, 4, 128)), g.normal(1, 0.1, 128), g.normal(1, 0.1, 128)
    q, k, v = PG.chunk_qkv(qkv, np.arange(9), qg, kg, 2, 1, 1e-6, 1e6)
    q2, k2, v2 = PG.chunk_qkv(qkv[5:], np.arange(5, 9), qg, kg, 2, 1, 1e-6, 1e6)
    assert np.allclose(q[5:], q2, atol=1e-13) and np.allclose(k[5:], k2, atol=1e-13) and np.array_equal(v[5:], v2)
    # one head through torch's rms_norm and a complex rotation
    n = torch.nn.functional.rms_norm(torch.from_numpy(qkv[:, 0]), (128,), torch.from_numpy(qg), 1e-6).numpy()
    z = (n[:, :64] + 1j * n[:, 64:]) * np.exp(1j * np.arange(9)[:, None] * 1e6 ** (-np.arange(64) / 64))
    assert np.allclose(q[:, 0], np.concatenate([z.real, z.imag], -1), atol=1e-12)


@pytest.mark.parametrize("n,length,visible", [(1, 1, 0), (1, 40, 0), (7, 7, 0), (5, 33, 0), (5, 33, 33), (6, 20, 17)])
def test_chunk_attention_is_masked_sdpa(n, length, visible):
    g = np.random.default_rng(n * 100 + length)
    q, k, v = g.normal(size=(n, 4, 128)), g.normal(size=(2, length, 128)), g.normal(size=(2, length, 128))
    o, lse, absv, _ = PG.chunk_attention(q, k, v, visible)
    i, j = np.arange(n)[:, None], np.arange(length)[None]
    see = j < np.maximum(visible, length - n + i + 1)
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1)[None], torch.from_numpy(k)[None], torch.from_numpy(v)[None],
        attn_mask=torch.from_numpy(see), enable_gqa=True)[0].transpose(0, 1).numpy()
    assert np.allclose(o, ref, atol=1e-12)
    s = np.einsum("nhd,hjd->nhj", q, np.repeat(k, 2, 0)) / np.sqrt(128.0)
    s = np.where(see[:, None], s, -np.inf)
    assert np.allclose(lse, torch.logsumexp(torch.from_numpy(s), -1).numpy(), atol=1e-12)
    assert np.all(absv + 1e-12 >= np.abs(o))


def test_chunks_of_a_causal_sequence_are_the_prefix_oracles():
    g = np.random.default_rng(5)
    q, k, v = g.normal(size=(30, 4, 128)), g.normal(size=(2, 30, 128)), g.normal(size=(2, 30, 128))
    ref, lse = PO.causal_gqa_attention(np.moveaxis(q, 1, 0), k, v, 30)
    got = [PG.chunk_attention(q[a:b], k[:, :b], v[:, :b], 0) for a, b in ((0, 11), (11, 12), (12, 30))]
    assert np.allclose(np.concatenate([x[0] for x in got]), np.moveaxis(ref, 0, 1), atol=1e-12)
    assert np.allclose(np.concatenate([x[1] for x in got]), lse.T, atol=1e-12)


def test_unseen_keys_have_no_influence():
    g = np.random.default_rng(6)
    q, k, v = g.normal(size=(3, 2, 128)), g.normal(size=(1, 10, 128)), g.normal(size=(1, 10, 128))
    ref = PG.chunk_attention(q, k, v, 0)[0]
    v[0, 8, 3], k[0, 9, 0] = np.inf, np.nan
    o = PG.chunk_attention(q, k, v, 0)[0]
    assert np.array_equal(o[0], ref[0]) and np.isinf(o[1, :, 3]).all() and np.isfinite(o[1, :, :3]).all()
    assert np.isnan(o[2]).all()
