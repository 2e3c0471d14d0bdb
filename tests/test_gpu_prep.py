"""kvpack_append and smla_query_prep on the GPU against the float64 oracle.

Tolerances.  A stored scale is an fp32 quotient of an fp32 maximum: the norm's sum, reciprocal square
root and products and the rotation lose a few units of 2^-24 each, 2^-19 covers them; where a rotation
or a mean cancels, the loss is relative to the row's largest element, so values are compared within
2^-19 of the row's amax (448 or 6 in code units).  A code is the grid value nearest to the exact one,
or its neighbour where the exact one lies within that loss of the border between them: its distance is
at most the nearest value's plus twice the loss.  A bf16 result is within half a step (2^-8) of itself
plus the rotation's loss.
"""
import numpy as np
import pytest
import torch

import paged_sparse_mla_gb300 as smla
import oracle
from oracle import prep
from tests import gpu_helpers as G

pytestmark = pytest.mark.gpu

LOSS = 2.0 ** -19
E4M3 = np.array(sorted({float(v) for v in oracle.e4m3_decode(np.arange(256, dtype=np.uint8)) if np.isfinite(v)}))
E2M1 = np.array(sorted({float(v) for v in oracle.e2m1_decode(np.arange(16, dtype=np.uint8))}))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.ensure_built()


def nearest_ok(got, want, grid):
    """Every `got` is a grid value as near to `want` as any, within twice the loss of top * LOSS."""
    top = grid[-1]
    i = np.clip(np.searchsorted(grid, want), 1, len(grid) - 1)
    best = np.minimum(np.abs(grid[i] - want), np.abs(grid[i - 1] - want))
    worst = (np.abs(got - want) - best).max()
    assert worst <= 2 * top * LOSS, worst
    assert np.isin(got, grid).all()


def table(n, d, seed=0):
    f = 10000.0 ** (-np.arange(0, d, 2) / max(d, 1))
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def wide(n, width, total, g, scale=1.0, shift=0.0):
    """A [n, width] bf16 slice of a [n, total] tensor (rows `total` elements apart), from column 8 on if it fits."""
    x = (torch.randn(n, total, generator=g, device="cuda") * scale + shift).bfloat16()
    at = min(8, total - width)
    return x[:, at:at + width]


SHAPES = {"full": (64, 1, 512, 64, 128, 128), "layers": (48, 3, 512, 64, 128, 128), "tiny": (16, 1, 64, 16, 64, 32),
          "mid": (7, 2, 256, 32, 128, 64), "wide_index": (64, 1, 128, 64, 64, 256)}


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("shape,n,strided,interleaved,norm,bias,rot", [
    ("full", 1, False, True, True, True, True), ("full", 257, True, False, True, False, True),
    ("full", 33, True, True, False, False, False), ("layers", 50, True, True, True, True, True),
    ("tiny", 19, False, False, True, True, True), ("mid", 12, True, True, True, False, True),
    ("wide_index", 40, True, False, True, True, True), ("full", 9, True, True, True, True, "keys"),
])
def test_append_matches_the_oracle(shape, fmt, n, strided, interleaved, norm, bias, rot):
    bs, layers, dl, dr, tile, di = SHAPES[shape]
    g = torch.Generator(device="cuda").manual_seed(n + dl)
    blocks = -(-n // bs) + 3
    lay = smla.layout_init(bs, layers, dl, dr, tile, di, blocks, fmt)
    ref = oracle.PoolLayout(bs, layers, dl, dr, tile, di, blocks, fmt)
    layer = layers - 1
    pool = torch.randint(0, 256, (lay.pool_bytes,), dtype=torch.uint8, device="cuda", generator=g)
    before = pool.cpu().numpy().copy()
    if strided:
        lat, rk, ik = wide(n, dl, dl + dr + 16, g, 3.0), wide(n, dr, dr + 10, g), wide(n, di, di + 3, g, 2.0, 0.5)
    else:
        lat, rk, ik = wide(n, dl, dl, g, 0.01), wide(n, dr, dr, g), wide(n, di, di, g, 5.0)
    if n > 2:  # a token whose first tile is all zeros
        lat[1, :tile] = 0
    ln = 1 + 0.1 * torch.randn(dl, generator=g, device="cuda") if norm else None
    kn = 1 + 0.1 * torch.randn(di, generator=g, device="cuda") if norm else None
    kb = 0.1 * torch.randn(di, generator=g, device="cuda") if bias else None
    tab = torch.from_numpy(table(5000, dr)).cuda()
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda")
    idx_rope = rot is True
    rope = smla.make_rope(tab, interleaved=interleaved, idx_interleaved=not interleaved, idx_rope=idx_rope) if rot else None
    slots = torch.randperm(blocks * bs, generator=g, device="cuda")[:n].contiguous()
    if n > 4:
        slots[3] = -1
    smla.kvpack_append(lay, pool, layer, lat, rk, ik, rope, pos if rot else None, slots, latent_norm=ln, idx_norm=kn,
                       idx_bias=kb, eps=1e-5)
    assert smla.smla_get_last_error() == 0
    after = pool.cpu().numpy()
    f64 = lambda t: t.double().cpu().numpy() if t is not None else None  # noqa: E731
    cs = f64(tab)[pos.cpu().numpy()] if rot else None
    cos, sin = (cs[:, :dr // 2], cs[:, dr // 2:]) if rot else (None, None)
    top, grid = (448.0, E4M3) if fmt == "e4m3" else (6.0, E2M1)
    codes, scales, r, key, kscale = prep.append_values(
        f64(lat), f64(rk), f64(ik), cos, sin, quant_tile=tile, top=top, latent_norm=f64(ln), idx_norm=f64(kn),
        idx_bias=f64(kb), eps=1e-5, interleaved=interleaved, idx_interleaved=not interleaved, idx_rope=idx_rope)
    sl = slots.cpu().numpy()
    keep = np.flatnonzero(sl >= 0)
    from oracle.store import _offsets
    rec = _offsets(ref, sl[keep], layer, "record")[:, None]
    got_codes = oracle.e4m3_decode(after[rec + np.arange(dl)])
    got_scales = np.ascontiguousarray(after[rec + dl + np.arange(4 * (dl // tile))]).view(np.float32)
    nearest_ok(got_codes, codes[keep], E4M3)
    np.testing.assert_allclose(got_scales, scales[keep], rtol=LOSS)
    got_r = oracle.bf16_bits_to_f64(np.ascontiguousarray(after[rec + dl + 4 * (dl // tile) + np.arange(2 * dr)]).view(np.uint16))
    size = np.abs(f64(rk)[keep]).max(-1, keepdims=True) * 2
    assert (np.abs(got_r - r[keep]) <= 2.0 ** -8 * np.abs(r[keep]) + LOSS * size).all()
    got_key, got_ks = oracle.read_index_key(ref, after, layer, sl[keep])
    nearest_ok(got_key, key[keep], grid)
    np.testing.assert_allclose(got_ks, kscale[keep], rtol=LOSS)
    # nothing else of the pool changed: other slots, other layers, padding
    touched = np.zeros(lay.pool_bytes, dtype=bool)
    touched[(rec + np.arange(ref.rec_bytes)).ravel()] = True
    touched[(_offsets(ref, sl[keep], layer, "key")[:, None] + np.arange(ref.key_bytes)).ravel()] = True
    touched[(_offsets(ref, sl[keep], layer, "scale")[:, None] + np.arange(4)).ravel()] = True
    assert np.array_equal(before[~touched], after[~touched])


def test_append_without_an_indexer_leaves_its_regions():
    lay = smla.layout_init(16, 1, 512, 64, 128, 128, 4)
    g = torch.Generator(device="cuda").manual_seed(0)
    pool = torch.full((lay.pool_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
    smla.kvpack_append(lay, pool, 0, wide(5, 512, 512, g), wide(5, 64, 64, g), None, None, None,
                       torch.arange(5, device="cuda"))
    b = pool.view(4, lay.block_stride)
    assert (b[:, lay.idx_key_off:] == 0xA5).all() and (b[0, :5 * lay.rec_stride] != 0xA5).any()


def test_append_skips_and_latches_bad_slots_and_positions():
    lay = smla.layout_init(16, 1, 512, 64, 128, 128, 4)
    g = torch.Generator(device="cuda").manual_seed(0)
    rope = smla.make_rope(torch.from_numpy(table(100, 64)).cuda(), interleaved=True)
    lat, rk, ik = wide(4, 512, 512, g), wide(4, 64, 64, g), wide(4, 128, 128, g)
    for slots, pos in (([0, 64, 2, 3], [0, 1, 2, 3]), ([0, 1, 2, 3], [0, 100, 2, 3]), ([0, 1, 2, 3], [0, -1, 2, 3])):
        pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")
        smla.kvpack_append(lay, pool, 0, lat, rk, ik, rope, torch.tensor(pos, device="cuda"), torch.tensor(slots, device="cuda"))
        assert smla.smla_get_last_error() == 4
        rec = pool[:16 * lay.rec_stride].view(16, -1)
        assert (rec[[0, 2, 3]] != 0).any(1).all() and not rec[1].any() and not rec[4:].any()


def test_append_of_extreme_rows():
    """Rows of zeros, rows near bf16's ends and a single large element: finite scales, nearest codes."""
    lay = smla.layout_init(16, 1, 512, 64, 128, 128, 1)
    ref = oracle.PoolLayout(16, 1, 512, 64, 128, 128, 1, "e4m3")
    lat = torch.zeros(5, 512, dtype=torch.bfloat16, device="cuda")
    lat[1] = 2.0 ** -120
    lat[2] = torch.linspace(-1, 1, 512).cuda() * 2.0 ** 120
    lat[3, 300] = 1e4
    lat[4] = torch.linspace(-1, 1, 512).cuda() * 2.0 ** -90
    ik = torch.zeros(5, 128, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")
    smla.kvpack_append(lay, pool, 0, lat, torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda"), ik, None, None,
                       torch.arange(5, device="cuda"))
    p = pool.cpu().numpy()
    x = lat.double().cpu().numpy()
    codes, scales = prep.quantise(x.reshape(5, 4, 128), 448.0)
    rec = p[:5 * 656].reshape(5, 656)
    nearest_ok(oracle.e4m3_decode(rec[:, :512]), codes.reshape(5, 512), E4M3)
    np.testing.assert_allclose(np.ascontiguousarray(rec[:, 512:528]).view(np.float32), scales, rtol=LOSS)
    keys, ks = oracle.read_index_key(ref, p, 0, np.arange(5))
    assert (keys == 0).all() and (ks == 1).all()


@pytest.mark.parametrize("t,h,hi,dr,di,norm,interleaved,rot,pe,ix", [
    (1, 64, 64, 64, 128, False, True, True, True, True), (37, 64, 64, 64, 128, True, False, True, True, True),
    (3, 5, 4, 16, 32, True, True, True, True, True), (70, 128, 3, 64, 256, False, False, True, True, True),
    (11, 8, 64, 32, 64, True, True, "pe", True, True), (9, 16, 64, 64, 128, False, True, False, True, True),
    (21, 24, 64, 64, 128, True, True, True, False, True), (21, 24, 64, 64, 128, True, True, True, True, False),
])
@pytest.mark.parametrize("strided", [False, True])
def test_query_prep_matches_the_oracle(t, h, hi, dr, di, norm, interleaved, rot, pe, ix, strided):
    g = torch.Generator(device="cuda").manual_seed(t * h + di)
    lay = smla.layout_init(16, 1, 64, dr, 64, di, 1)
    prm = smla.make_params(h, hi, 16, 1.0)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    more = 129 if strided else 0                      # an odd head stride: 2-byte aligned slices
    q_pe = rnd(t, h, dr + more).bfloat16()[..., more:]
    q_idx = (rnd(t, hi, di + more) * 3).bfloat16()[..., more:]
    if t > 2:
        q_idx[1, 0] = 0
    kn = 1 + 0.1 * rnd(di) if norm else None
    w = rnd(t, hi)
    tab = torch.from_numpy(table(9000, dr)).cuda()
    pos = torch.randint(0, 9000, (t,), generator=g, device="cuda")
    idx_rope = rot is True
    rope = smla.make_rope(tab, interleaved=interleaved, idx_interleaved=not interleaved, idx_rope=idx_rope) if rot else None
    q_pe_out = torch.full((t, h, dr), 7.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((t, hi, di), 0x55, dtype=torch.uint8, device="cuda")
    w_out = torch.full((t, hi), 7.0, device="cuda")
    smla.smla_query_prep(lay, prm, rope, pos if rot else None, q_pe=q_pe if pe else None, q_pe_out=q_pe_out if pe else None,
                         q_idx=q_idx if ix else None, w=w if ix else None, w_scale=0.125, q_idx_out=codes if ix else None,
                         w_out=w_out if ix else None, idx_norm=kn if ix else None, eps=1e-5)
    assert smla.smla_get_last_error() == 0
    f64 = lambda x: x.double().cpu().numpy() if x is not None else None  # noqa: E731
    cs = f64(tab)[pos.cpu().numpy()] if rot else None
    cos, sin = (cs[:, :dr // 2], cs[:, dr // 2:]) if rot else (None, None)
    if pe:
        want = prep.rotate(f64(q_pe), cos[:, None], sin[:, None], interleaved) if rot else f64(q_pe)
        size = 2 * np.abs(f64(q_pe)).max(-1, keepdims=True)
        assert (np.abs(f64(q_pe_out) - want) <= 2.0 ** -8 * np.abs(want) + LOSS * size).all()
    else:
        assert (q_pe_out == 7).all()
    if ix:
        want, want_w = prep.query_values(f64(q_idx), f64(w), 0.125, cos, sin, idx_norm=f64(kn), eps=1e-5,
                                         idx_interleaved=not interleaved, idx_rope=idx_rope)
        nearest_ok(oracle.e4m3_decode(codes.cpu().numpy()), want, E4M3)
        np.testing.assert_allclose(f64(w_out), want_w, rtol=LOSS)
    else:
        assert (codes == 0x55).all() and (w_out == 7).all()


def test_query_prep_leaves_tokens_of_bad_positions():
    lay = smla.layout_init(64, 1, 512, 64, 128, 128, 1)
    prm = smla.make_params(8, 64, 16, 1.0)
    rope = smla.make_rope(torch.from_numpy(table(10, 64)).cuda(), interleaved=True)
    q_pe, q_idx = torch.ones(3, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 64, 128, dtype=torch.bfloat16, device="cuda")
    q_pe_out, codes, w_out = torch.full_like(q_pe, 7), torch.full((3, 64, 128), 9, dtype=torch.uint8, device="cuda"), torch.full((3, 64), 5.0, device="cuda")
    smla.smla_query_prep(lay, prm, rope, torch.tensor([1, 10, 9], device="cuda"), q_pe=q_pe, q_pe_out=q_pe_out, q_idx=q_idx,
                         w=torch.ones(3, 64, device="cuda"), q_idx_out=codes, w_out=w_out)
    assert smla.smla_get_last_error() == 4
    assert (q_pe_out[1] == 7).all() and (codes[1] == 9).all() and (w_out[1] == 5).all()
    for k in (0, 2):
        assert (w_out[k] != 5).all() and (codes[k] != 9).all() and (q_pe_out[k] != 7).any()


def test_prep_on_another_stream_and_in_a_graph():
    g = torch.Generator(device="cuda").manual_seed(5)
    lay = smla.layout_init(64, 1, 512, 64, 128, 128, 8)
    prm = smla.make_params(64, 64, 16, 1.0)
    rope = smla.make_rope(torch.from_numpy(table(100, 64)).cuda(), interleaved=True)
    n = 100
    kv, ik = wide(n, 576, 576, g), wide(n, 128, 128, g)
    q_pe, q_idx, w = torch.randn(n, 64, 64, generator=g, device="cuda").bfloat16(), torch.randn(n, 64, 128, generator=g, device="cuda").bfloat16(), torch.rand(n, 64, generator=g, device="cuda")
    pos, slots = torch.arange(n, device="cuda"), torch.randperm(512, device="cuda", generator=g)[:n].contiguous()

    def once(stream=None):
        pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")
        outs = torch.empty_like(q_pe), torch.empty(n, 64, 128, dtype=torch.uint8, device="cuda"), torch.empty(n, 64, device="cuda")
        torch.cuda.synchronize()

        def call():
            smla.kvpack_append(lay, pool, 0, kv[:, :512], kv[:, 512:], ik, rope, pos, slots, stream=stream)
            smla.smla_query_prep(lay, prm, rope, pos, q_pe=q_pe, q_pe_out=outs[0], q_idx=q_idx, w=w, q_idx_out=outs[1], w_out=outs[2], stream=stream)
        return call, (pool, *outs)
    call, want = once()
    call()
    side = torch.cuda.Stream()
    call, got = once(side)
    call()
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    call, got = once()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        got[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
