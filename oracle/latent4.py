"""4-bit latents: E2M1 codes in groups of 16 with an unsigned 8-bit scale each.

[GLM-5.3 "How to try"] keeps the KV cache in FP8, [AgentX "Hybrid KV cache management"] its indexer keys in FP4; the
pages have no 4-bit latents.

reading (codes): the OCP MX FP4 E2M1 element type of ``oracle.fp4``, value 2i in the low nibble of byte i.

reading (scale): an unsigned float of 5 exponent bits (bias 15) and 3 mantissa bits; exponent field 0 is subnormal:
code c = 8 e + m stands for (8 + m) 2^(e - 18), and for m 2^-17 where e = 0.  Fields 31 are not used.

reading (quantisation): per group, scale = amax / 6 rounded to the nearest code, ties to the even one, at most 10240
(6 x 10240 is inside fp16's range); code = E2M1 nearest-even, saturating, of fp32(x / scale); all codes zero (with the
values' signs) where the scale is 0.
"""

import numpy as np

from .fp4 import e2m1_decode, e2m1_encode, e2m1_pack, e2m1_unpack

GROUP = 16
SCALE_MAX = 10240.0


def scale4_decode(codes) -> np.ndarray:
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = c // 8, c % 8
    return np.where(e == 0, m * 2.0 ** -17, (8 + m) * 2.0 ** (e - 18.0))


_SCALES = scale4_decode(np.arange(0xE3))          # 0 .. 10240, increasing


def scale4_encode(s) -> np.ndarray:
    """Nearest scale code of values >= 0, ties to the even code, saturating."""
    s = np.asarray(s, dtype=np.float64)
    hi = np.clip(np.searchsorted(_SCALES, s), 1, len(_SCALES) - 1)   # _SCALES[hi - 1] < s <= _SCALES[hi]
    below, above = s - _SCALES[hi - 1], _SCALES[hi] - s
    down = (below < above) | ((below == above) & ((hi - 1) % 2 == 0))
    return np.where(down, hi - 1, hi).astype(np.uint8)


def quantize_latent4(x):
    """Values [T, D] (float64) -> (packed codes uint8 [T, D/2], scale codes uint8 [T, D/16])."""
    x = np.asarray(x, dtype=np.float64)
    t, d = x.shape
    g = x.reshape(t, d // GROUP, GROUP)
    amax = np.abs(g).max(axis=2)
    scales = scale4_encode((amax / 6.0).astype(np.float32))
    s = scale4_decode(scales)[:, :, None]
    q = np.where(s > 0, g / np.where(s > 0, s, 1.0), np.copysign(0.0, g)).astype(np.float32)
    return e2m1_pack(e2m1_encode(q).reshape(t, d)), scales


def latent4_decode(codes, scales) -> np.ndarray:
    """Packed codes [n, D/2] and scale codes [n, D/16] -> values [n, D] (float64, exact)."""
    v = e2m1_decode(e2m1_unpack(codes))
    n, d = v.shape
    return (v.reshape(n, d // GROUP, GROUP) * scale4_decode(scales)[:, :, None]).reshape(n, d)
