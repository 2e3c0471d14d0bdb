"""Norm, rotation and quantisation on the way into the cache and into the indexer.

[GLM-5.3 "How to try"]: the KV cache is FP8; [AgentX "DeepSeek V4"]: 64 indexer
heads a token.  The pages give no formulas; the readings taken here are the
common ones of latent attention: an RMS norm of the latent, a layer norm (or
RMS norm) of the indexer key, rotary position embedding of the rope dims, and
amax quantisation.  Everything is float64 and nothing is rounded: a quantised
vector is returned as the real values z * (F / amax) that its codes stand near,
with its scale amax / F.
"""

import numpy as np


def rotate(x, cos, sin, interleaved: bool):
    """x [..., d] turned pairwise by angles with cosines and sines [..., d / 2]."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    i = np.arange(d // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + d // 2)
    y = np.empty(np.broadcast_shapes(x.shape, cos.shape[:-1] + (d,)))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def rms_norm(x, weight, eps: float):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def layer_norm(x, weight, bias, eps: float):
    x = np.asarray(x, dtype=np.float64)
    c = x - x.mean(-1, keepdims=True)
    return c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * weight + bias


def quantise(z, top: float):
    """(unrounded code values, scale) of the last axis; vectors below 2^-100 take scale 1."""
    amax = np.abs(z).max(-1, keepdims=True)
    scale = np.where(amax < 2.0 ** -100, 1.0, amax / top)
    return z / scale, scale[..., 0]


def append_values(latent, rope_key, idx_k, cos, sin, *, quant_tile, top, latent_norm=None, idx_norm=None, idx_bias=None,
                  eps=1e-6, interleaved=False, idx_interleaved=False, idx_rope=True):
    """What kvpack_append puts into the cache for each token: (latent code values [n, d], scales [n, tiles],
    rope [n, d_rope], key code values [n, d_index], key scales [n]).  cos / sin None: no rotation."""
    y = np.asarray(latent, dtype=np.float64)
    if latent_norm is not None:
        y = rms_norm(y, latent_norm, eps)
    codes, scales = quantise(y.reshape(y.shape[0], -1, quant_tile), top=448.0)
    r = np.asarray(rope_key, dtype=np.float64)
    if cos is not None:
        r = rotate(r, cos, sin, interleaved)
    z = np.asarray(idx_k, dtype=np.float64)
    if idx_norm is not None:
        z = rms_norm(z, idx_norm, eps) if idx_bias is None else layer_norm(z, idx_norm, idx_bias, eps)
    if cos is not None and idx_rope:
        d = 2 * cos.shape[-1]
        z = np.concatenate([rotate(z[:, :d], cos, sin, idx_interleaved), z[:, d:]], axis=1)
    key, key_scale = quantise(z, top)
    return codes.reshape(y.shape), scales, r, key, key_scale


def query_values(q_idx, w, w_scale, cos, sin, *, idx_norm=None, eps=1e-6, idx_interleaved=False, idx_rope=True):
    """(code values [T, H, d], weights [T, H]) of smla_query_prep's indexer part."""
    z = np.asarray(q_idx, dtype=np.float64)
    if idx_norm is not None:
        z = rms_norm(z, idx_norm, eps)
    if cos is not None and idx_rope:
        d = 2 * cos.shape[-1]
        z = np.concatenate([rotate(z[..., :d], cos[:, None], sin[:, None], idx_interleaved), z[..., d:]], axis=-1)
    codes, scale = quantise(z, 448.0)
    return codes, np.asarray(w, dtype=np.float64) * w_scale * scale
