"""The oracle's 4-bit latents tied to fp16, to torch and to the E2M1 codec (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import latent4
from oracle.store import kvpack_store, read_record


def test_scale_codes_are_the_upper_bytes_of_fp16():
    c = np.arange(0xF8, dtype=np.uint16)
    want = (c << 7).astype(np.uint16).view(np.float16).astype(np.float64)
    assert np.array_equal(latent4.scale4_decode(c), want)
    assert latent4.scale4_decode(0xE2) == latent4.SCALE_MAX and np.all(np.diff(want) > 0)


def test_scale_rounding_against_brute_force():
    table = latent4.scale4_decode(np.arange(0xE3))
    s = np.concatenate([table, (table[1:] + table[:-1]) / 2, table * 1.03, [2.0 ** -18, 2.0 ** -18 * 1.001, 1e30, 0.0]])
    for v, c in zip(s, latent4.scale4_encode(s)):
        err = np.abs(table - v)
        near = np.flatnonzero(err == err.min())
        assert c in near and (len(near) == 1 or c % 2 == 0), (v, c)


def test_every_product_is_exact_in_fp16_and_bf16():
    v = np.outer(oracle.fp4.e2m1_decode(np.arange(16)), latent4.scale4_decode(np.arange(0xE3))).reshape(-1)
    assert np.array_equal(v.astype(np.float16).astype(np.float64), v)
    assert np.array_equal(torch.from_numpy(v).bfloat16().double().numpy(), v)
    assert not np.isfinite(np.float16(6.0 * latent4.scale4_decode(0xE3)))


@pytest.mark.parametrize("scale", [1e-7, 1e-3, 1.0, 300.0, 1e6])
def test_quantisation_error(scale):
    """The largest gap of E2M1 is 2 below 6 and a scale is off by 2^-4 of itself, or by half a step of its smallest: a value is
    off by at most one code step of the group plus what saturates, 6 s 2^-4; where amax leaves the scales' range, by what it leaves."""
    x = np.random.default_rng(0).standard_normal((40, 64)) * scale
    codes, scales = latent4.quantize_latent4(x)
    y = latent4.latent4_decode(codes, scales)
    amax = np.abs(x.reshape(40, 4, 16)).max(2).repeat(16, 1)
    assert np.all(np.abs(x - y) <= amax / 6 * (1 + 6 / 16) * (1 + 1 / 16) + 6 * 2.0 ** -18 + np.maximum(0, amax - 61440))


def test_layout_and_store_round_trip():
    lay = oracle.PoolLayout(16, 2, 512, 64, 16, 128, 3, "e4m3", "e2m1")
    assert (lay.rec_bytes, lay.rec_stride) == (416, 416)
    rng = np.random.default_rng(1)
    lat = torch.from_numpy(rng.standard_normal((5, 512))).bfloat16()
    bits = lambda t: t.view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    rope = torch.from_numpy(rng.standard_normal((5, 64))).bfloat16()
    pool = np.zeros(lay.pool_bytes, np.uint8)
    slots = np.array([0, 17, 47, -1, 5])
    kvpack_store(lay, pool, 1, bits(lat), bits(rope), rng.integers(0, 255, (5, 128)), np.ones(5, np.float32), slots)
    got, pe = read_record(lay, pool, 1, slots[slots >= 0])
    keep = slots >= 0
    assert np.array_equal(got, latent4.latent4_decode(*latent4.quantize_latent4(lat.double().numpy()[keep])))
    assert np.array_equal(pe, rope.double().numpy()[keep])
    rel = np.linalg.norm(got - lat.double().numpy()[keep]) / np.linalg.norm(got)
    assert 0.05 < rel < 0.12                       # four bits: about a tenth of a normal value's size


def test_planted_mistakes_are_seen():
    """Nibbles swapped, a scale's bias off by one, truncation instead of rounding: each gives other values."""
    x = np.random.default_rng(2).standard_normal((4, 32))
    codes, scales = latent4.quantize_latent4(x)
    y = latent4.latent4_decode(codes, scales)
    assert not np.array_equal(y, latent4.latent4_decode((codes >> 4 | codes << 4).astype(np.uint8), scales))
    assert not np.array_equal(y, latent4.latent4_decode(codes, scales + 8))
    assert np.any(scales != np.searchsorted(latent4._SCALES, (np.abs(x.reshape(4, 2, 16)).max(2) / 6), side="right") - 1)
