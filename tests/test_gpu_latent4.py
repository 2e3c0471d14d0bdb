"""4-bit latents on the GPU: written, read back, attended over, against float64 over the same cache."""
import numpy as np
import pytest
import torch

import paged_sparse_mla_gb300 as smla
import oracle
from oracle import latent4, prep
from oracle.store import _offsets
from tests import gpu_helpers as G
from tests.latent4_cases import P_BF16, Case4, bf16_bits
from tests.test_gpu_prep import E2M1, LOSS, nearest_ok, table, wide

pytestmark = pytest.mark.gpu

SHAPES = {"full": (64, 1, 512, 64, 128), "layers": (48, 3, 512, 64, 128), "tiny": (16, 1, 64, 16, 32), "mid": (7, 2, 256, 32, 64),
          "wide_index": (64, 1, 128, 64, 256), "no_rope": (16, 1, 512, 0, 128)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.ensure_built()


def ok():
    assert smla.smla_get_last_error() == 0


def layouts(shape, blocks, keys="e4m3", fmt="e2m1"):
    bs, layers, dl, dr, di = SHAPES[shape]
    tile = 16 if fmt == "e2m1" else min(128, dl)
    return (smla.layout_init(bs, layers, dl, dr, tile, di, blocks, keys, latent_format=fmt),
            oracle.PoolLayout(bs, layers, dl, dr, tile, di, blocks, keys, fmt))


def hard_values(n, dl, rng):
    """Latents of every size: ties between codes, zero groups, values past the scales' range and below it."""
    x = rng.standard_normal((n, dl)) * np.exp2(rng.integers(-24, 18, (n, 1)))
    x[0] = rng.integers(-24, 25, dl) * 0.25              # many lie half way between two codes
    if n > 3:
        x[1, :16] = 0
        x[2] = np.where(rng.random(dl) < 0.5, 1e5, -3e38)
        x[3] *= np.exp2(rng.integers(-20, 20, dl))
    return torch.from_numpy(x).bfloat16()


@pytest.mark.parametrize("keys", ["e4m3", "e2m1"])
@pytest.mark.parametrize("shape,n", [("full", 1), ("full", 300), ("layers", 77), ("tiny", 19), ("mid", 40), ("wide_index", 9), ("no_rope", 5)])
def test_store_writes_the_oracles_bytes(shape, n, keys):
    bs, layers, dl, dr, di = SHAPES[shape]
    blocks = -(-n // bs) + 2
    lay, ref = layouts(shape, blocks, keys)
    rng = np.random.default_rng(n + dl)
    lat, rope = hard_values(n, dl, rng), torch.from_numpy(rng.standard_normal((n, dr))).bfloat16()
    key = torch.from_numpy(rng.integers(0, 256, (n, lay.key_bytes), dtype=np.uint8))
    ks = torch.rand(n)
    slots = torch.from_numpy(rng.permutation(blocks * bs)[:n])
    if n > 4:
        slots[4] = -1
    pool = torch.from_numpy(rng.integers(0, 256, lay.pool_bytes, dtype=np.uint8))
    want = pool.numpy().copy()
    b16 = lambda t: t.view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    oracle.kvpack_store(ref, want, layers - 1, b16(lat), b16(rope), key.numpy(), ks.numpy(), slots.numpy())
    got = pool.cuda()
    smla.kvpack_store(lay, got, layers - 1, lat.cuda(), rope.cuda(), key.cuda(), ks.cuda(), slots.cuda())
    ok()
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("keys", ["e4m3", "e2m1"])
@pytest.mark.parametrize("shape,n,strided,interleaved,norm,bias,rot", [
    ("full", 1, False, True, True, True, True), ("full", 257, True, False, True, False, True), ("full", 33, True, True, False, False, False),
    ("layers", 50, True, True, True, True, True), ("tiny", 19, False, False, True, True, True), ("mid", 12, True, True, True, False, True),
    ("wide_index", 40, True, False, True, True, True),
])
def test_append_matches_the_oracle(shape, keys, n, strided, interleaved, norm, bias, rot):
    bs, layers, dl, dr, di = SHAPES[shape]
    g = torch.Generator(device="cuda").manual_seed(n + dl)
    blocks, layer = -(-n // bs) + 3, layers - 1
    lay, ref = layouts(shape, blocks, keys)
    pool = torch.randint(0, 256, (lay.pool_bytes,), dtype=torch.uint8, device="cuda", generator=g)
    before = pool.cpu().numpy().copy()
    if strided:
        lat, rk, ik = wide(n, dl, dl + dr + 16, g, 3.0), wide(n, dr, dr + 10, g), wide(n, di, di + 3, g, 2.0, 0.5)
    else:
        lat, rk, ik = wide(n, dl, dl, g, 0.01), wide(n, dr, dr, g), wide(n, di, di, g, 5.0)
    if n > 2:
        lat[1, :16] = 0
    ln = 1 + 0.1 * torch.randn(dl, generator=g, device="cuda") if norm else None
    kn = 1 + 0.1 * torch.randn(di, generator=g, device="cuda") if norm else None
    kb = 0.1 * torch.randn(di, generator=g, device="cuda") if bias else None
    tab = torch.from_numpy(table(5000, dr)).cuda()
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda")
    rope = smla.make_rope(tab, interleaved=interleaved, idx_interleaved=not interleaved) if rot else None
    slots = torch.randperm(blocks * bs, generator=g, device="cuda")[:n].contiguous()
    if n > 4:
        slots[3] = -1
    smla.kvpack_append(lay, pool, layer, lat, rk, ik, rope, pos if rot else None, slots, latent_norm=ln, idx_norm=kn, idx_bias=kb, eps=1e-5)
    ok()
    after = pool.cpu().numpy()
    f64 = lambda t: t.double().cpu().numpy() if t is not None else None  # noqa: E731
    cs = f64(tab)[pos.cpu().numpy()] if rot else None
    cos, sin = (cs[:, :dr // 2], cs[:, dr // 2:]) if rot else (None, None)
    codes, scales, r, key, kscale = prep.append_values(
        f64(lat), f64(rk), f64(ik), cos, sin, quant_tile=16, top=448.0 if keys == "e4m3" else 6.0, latent_norm=f64(ln), idx_norm=f64(kn),
        idx_bias=f64(kb), eps=1e-5, interleaved=interleaved, idx_interleaved=not interleaved)
    sl = slots.cpu().numpy()
    keep = np.flatnonzero(sl >= 0)
    y = (codes.reshape(n, dl // 16, 16) * scales[..., None])[keep]      # what is quantised
    rec = _offsets(ref, sl[keep], layer, "record")[:, None]
    got_s = after[rec + dl // 2 + np.arange(dl // 16)]
    amax = np.abs(y).max(-1)
    low, high = latent4.scale4_encode(amax / 6 * (1 - LOSS)), latent4.scale4_encode(amax / 6 * (1 + LOSS))
    assert ((got_s >= low) & (got_s <= high)).all()
    s = latent4.scale4_decode(got_s)[..., None]
    got_c = oracle.e2m1_decode(oracle.fp4.e2m1_unpack(after[rec + np.arange(dl // 2)])).reshape(y.shape)
    assert (got_c[(s == 0)[..., 0]] == 0).all()
    some = (s > 0)[..., 0]
    nearest_ok(got_c[some], np.clip((y / np.where(s > 0, s, 1))[some], -6, 6), E2M1)
    got_r = oracle.bf16_bits_to_f64(np.ascontiguousarray(after[rec + dl // 2 + dl // 16 + np.arange(2 * dr)]).view(np.uint16))
    assert (np.abs(got_r - r[keep]) <= 2.0 ** -8 * np.abs(r[keep]) + LOSS * 2 * np.abs(f64(rk)[keep]).max(-1, keepdims=True)).all()
    got_key, got_ks = oracle.read_index_key(ref, after, layer, sl[keep])
    np.testing.assert_allclose(got_ks, kscale[keep], rtol=LOSS)
    # what belongs to no appended token is as it was
    touched = np.zeros(lay.pool_bytes, bool)
    touched[(rec + np.arange(lay.rec_bytes)).reshape(-1)] = True
    touched[(_offsets(ref, sl[keep], layer, "key")[:, None] + np.arange(lay.key_bytes)).reshape(-1)] = True
    touched[(_offsets(ref, sl[keep], layer, "scale")[:, None] + np.arange(4)).reshape(-1)] = True
    assert np.array_equal(after[~touched], before[~touched])


def test_append_of_normless_latents_is_the_stores_bytes():
    """Without a norm the appended latent is the finished one: both calls write the same record."""
    lay, _ = layouts("full", 6)
    rng = np.random.default_rng(3)
    lat = hard_values(200, 512, rng).cuda()
    rope, key = torch.randn(200, 64, device="cuda").bfloat16(), torch.randn(200, 128, device="cuda").bfloat16()
    slots = torch.randperm(384, device="cuda")[:200].contiguous()
    a, b = (torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    smla.kvpack_append(lay, a, 0, lat, rope, None, None, None, slots)
    smla.kvpack_store(lay, b, 0, lat, rope, torch.zeros(200, 128, dtype=torch.uint8, device="cuda"), torch.zeros(200, device="cuda"), slots)
    ok()
    assert torch.equal(a, b)


# ---------------------------------- reading back ----------------------------------

@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("lens,starts,bs,dl,dr,layers", [
    ([1], None, 64, 512, 64, 1), ([5, 0, 130, 64], None, 64, 512, 64, 2), ([33, 700, 100], [0, 17, 99], 16, 512, 64, 1), ([40, 9], [40, 2], 7, 512, 64, 1),
    ([100, 31], [3, 0], 16, 128, 16, 1), ([20], None, 16, 512, 0, 1), ([50, 3], None, 5, 256, 32, 3),
])
@pytest.mark.parametrize("strided", [False, True])
def test_load_gives_the_cached_values(fmt, lens, starts, bs, dl, dr, layers, strided):
    c = Case4(lens, [0] * len(lens), 1, bs, dl, dr, layers, layers - 1, seed=sum(lens), fmt=fmt)
    st = [0] * len(lens) if starts is None else starts
    counts = [n - s for n, s in zip(lens, st)]
    n, pad = sum(counts), 3
    loc = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    buf = torch.full((n + pad, dl + dr + (5 if strided else 8)), 777.0, dtype=torch.bfloat16, device="cuda")
    lat, rope = (buf[:, :dl], buf[:, dl:dl + dr]) if strided else (buf[:, :dl].contiguous(), buf[:, dl:dl + dr].contiguous())
    smla.kvpack_load(c.lay, c.pool, c.layer, c.table, loc, lat, rope, starts=None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda"))
    ok()
    want = [np.concatenate([k[i][s:] for k, s in zip(c.keys, st)]) for i in (0, 1)]
    assert np.array_equal(rope[:n].double().cpu().numpy(), want[1])
    w = torch.from_numpy(want[0])
    assert torch.equal(lat[:n].cpu(), w.bfloat16())                # E2M1: exact; E4M3: the fp32 product rounded once
    if fmt == "e2m1":
        assert torch.equal(lat[:n].double().cpu(), w)
    assert (lat[n:] == 777).all() and (rope[n:] == 777).all()
    assert not strided or (buf[:, dl + dr:] == 777).all()
    only = torch.full((n + pad, dl), 777.0, dtype=torch.bfloat16, device="cuda")
    smla.kvpack_load(c.lay, c.pool, c.layer, c.table, loc, only, None, starts=None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda"))
    assert torch.equal(only[:n], lat[:n])


def test_load_of_bad_blocks_and_positions():
    c = Case4([100, 60], [0, 0], 1, 16, seed=1)
    c.table[0, 1] = c.lay.num_blocks
    c.table[1, 0] = -1
    loc = torch.tensor([0, 100, 165], dtype=torch.int32, device="cuda")
    lat = torch.full((165, 512), 777.0, dtype=torch.bfloat16, device="cuda")
    c.table = torch.cat([c.table, torch.full((2, 0), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    smla.kvpack_load(c.lay, c.pool, 0, c.table, loc, lat, starts=torch.tensor([-2, 0], dtype=torch.int32, device="cuda"))
    assert smla.smla_get_last_error() == 4
    assert (lat[:2] == 0).all() and (lat[18:34] == 0).all() and (lat[100:116] == 0).all()
    assert torch.equal(lat[2:18].double().cpu(), torch.from_numpy(c.keys[0][0][:16]))
    assert torch.equal(lat[116:160].double().cpu(), torch.from_numpy(c.keys[1][0][16:60]))


# ---------------------------------- the whole context ----------------------------------

@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lens,counts,heads,bs", [
    ([1], [1], 64, 64), ([63], [1], 64, 64), ([64], [1], 64, 64), ([65], [2], 64, 64), ([127, 128, 129, 1], [1, 1, 1, 1], 64, 64),
    ([1000], [1], 64, 64), ([777, 33, 400], [4, 4, 4], 64, 64), ([300, 5, 513, 70], [7, 5, 1, 70], 64, 16), ([260, 90], [33, 2], 16, 64),
    ([260, 90], [33, 2], 5, 48), ([130], [9], 1, 7), ([200, 140], [21, 3], 24, 32), ([300, 64], [3, 1], 128, 64), ([150], [5], 100, 16),
    ([2500], [2], 65, 128), ([400, 400, 400], [0, 3, 0], 64, 64), ([50, 80], [50, 80], 64, 64),
])
def test_dense_matches_float64(lens, counts, heads, bs, workspace):
    c = Case4(lens, counts, heads, bs, seed=sum(lens) + heads, pad_rows=2)
    c.check(c.dense(workspace))
    ok()


@pytest.mark.parametrize("lens,counts,heads,bs,dl,dr", [
    ([1], [1], 8, 16, 64, 16), ([100, 31, 33], [3, 1, 33], 8, 16, 64, 16), ([75], [4], 3, 7, 128, 32), ([140], [2], 16, 64, 256, 64),
    ([90], [2], 64, 64, 512, 0), ([90, 0], [2, 1], 9, 64, 512, 32),
])
def test_dense_of_other_shapes(lens, counts, heads, bs, dl, dr):
    c = Case4(lens, counts, heads, bs, dl, dr, seed=3)
    c.check(c.dense())
    ok()


def test_dense_long_contexts_split_over_the_sms():
    c = Case4([9001, 20000], [2, 1], 64, seed=6)
    c.check(c.dense(True))
    c.check(c.dense(False))
    ok()


def test_dense_uneven_sequences_give_the_same_bits_every_time():
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(1, 700, 90)]
    counts = [int(min(n, k)) for n, k in zip(lens, rng.integers(1, 6, 90))]
    for heads in (64, 16):
        c = Case4(lens, counts, heads, seed=5)
        want = c.dense()
        c.check(want)
        for _ in range(20):
            got = c.dense()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ok()


def test_dense_tokens_that_see_nothing():
    c = Case4([0, 3, 0, 200], [1, 5, 2, 1], 64, seed=7, pad_rows=3, extra_cols=4)
    for ws in (True, False):
        out, lse = c.dense(ws)
        c.check((out, lse))
        assert (out[0] == 0).all() and (lse[0] == -np.inf).all() and (out[1:3] == 0).all()
    ok()


def test_dense_layers_of_one_pool():
    for layer in (0, 2):
        c = Case4([150, 90], [2, 1], 64, 32, layers=3, layer=layer, seed=9)
        c.check(c.dense())
    ok()


@pytest.mark.parametrize("key_scale,q_scale", [(1e-4, 1.0), (1e-3, 30.0), (100.0, 0.01), (1.0, 1e-3), (1.0, 20.0), (1e4, 1e4), (1e4, 1e-4)])
def test_dense_magnitudes(key_scale, q_scale):
    """Scales down to the subnormal ones, keys near fp16's end, sharp softmaxes: the cached values stay exact."""
    c = Case4([333, 65], [3, 1], 64, seed=10, key_scale=key_scale, q_scale=q_scale)
    c.check(c.dense())
    ok()


def test_dense_bad_block_ids_read_as_zeros_and_latch():
    c = Case4([200, 100], [1, 2], 64, seed=12)
    c.table[0, 1] = c.lay.num_blocks
    c.table[1, 0] = -1
    keys = [tuple(x.copy() for x in k) for k in c.keys]
    for x in keys[0]:
        x[64:128] = 0
    for x in keys[1]:
        x[:64] = 0
    got = c.dense()
    assert smla.smla_get_last_error() == 4
    c.check(got, keys=keys)


@pytest.mark.parametrize("byte", [0xE3, 0xF8, 0xFF])
@pytest.mark.parametrize("at", [0, 99, 130])
def test_dense_scales_that_nothing_writes_are_latched(byte, at):
    """A scale byte above 10240's inside a context: past fp16's end, infinite or NaN.  Other sequences are not touched."""
    c = Case4([131, 90], [2, 3], 64, seed=13)
    blk = int(c.table[0, at // 64])
    c.pool.view(-1, c.lay.block_stride)[blk, (at % 64) * 416 + 256 + 7] = byte
    out, lse = c.dense()
    assert smla.smla_get_last_error() == 7
    clean = Case4([131, 90], [2, 3], 64, seed=13)
    o2, l2 = clean.dense()
    assert torch.equal(out[2:], o2[2:]) and torch.equal(lse[2:], l2[2:])
    ok()


# ---------------------------------- selected positions ----------------------------------

@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lens,counts,heads,bs,top_k,keep", [
    ([1], [1], 64, 64, 64, 1.0), ([65], [2], 64, 64, 64, 1.0), ([300, 5, 513, 70], [7, 5, 1, 70], 64, 16, 128, 1.0), ([500], [3], 5, 48, 200, 0.5),
    ([5000, 3000], [1, 2], 64, 64, 2048, 1.0), ([130], [9], 1, 7, 33, 1.0), ([900] * 8, [20] * 8, 64, 64, 256, 1.0), ([700, 900], [200, 130], 16, 64, 100, 1.0),
])
def test_selected_positions_match_float64(lens, counts, heads, bs, top_k, keep, workspace):
    c = Case4(lens, counts, heads, bs, seed=sum(lens) + heads, pad_rows=1)
    sel = c.select(top_k, keep)
    c.check(c.sparse(sel, workspace), sel, weight=P_BF16)
    ok()


@pytest.mark.parametrize("dl,dr", [(64, 16), (64, 64), (512, 0), (512, 32)])
def test_selected_positions_of_other_shapes(dl, dr):
    c = Case4([200, 60], [3, 1], 9, 16, dl, dr, layers=2, layer=1, seed=4)
    sel = c.select(100)
    c.check(c.sparse(sel), sel, weight=P_BF16)
    ok()


def test_rows_without_a_selection_and_holes_in_it():
    c = Case4([200, 300], [2, 3], 64, seed=5)
    sel = c.select(128)
    sel[1] = -1
    sel[3, ::3] = -1                                      # holes among the entries
    got = c.sparse(sel)
    c.check(got, sel, weight=P_BF16)
    assert (got[0][1] == 0).all() and (got[1][1] == -np.inf).all()
    ok()


def test_every_position_selected_is_the_dense_result():
    c = Case4([150, 64], [2, 1], 64, seed=6)
    sel = c.select(192)
    a, b = c.sparse(sel), c.dense()
    c.check(a, sel, weight=P_BF16)
    c.check(b)
    ok()


def test_selected_magnitudes():
    for key_scale, q_scale in ((1e-4, 1.0), (1e4, 1e-4), (1.0, 20.0)):
        c = Case4([400], [3], 64, seed=8, key_scale=key_scale, q_scale=q_scale)
        sel = c.select(256)
        c.check(c.sparse(sel), sel, weight=P_BF16)
    ok()


def test_host_tier_of_4_bit_records():
    """Evicted records read from pinned host memory give the bits of the pool's."""
    c = Case4([300, 200], [2, 2], 64, seed=9)
    sel = c.select(128)
    want = c.sparse(sel, workspace=False)
    per = c.lay.block_size * c.lay.rec_stride
    blocks = c.pool.view(-1, c.lay.block_stride)
    host_map = torch.full((c.lay.num_blocks,), -1, dtype=torch.int32)
    host_map[::2] = torch.arange((c.lay.num_blocks + 1) // 2, dtype=torch.int32)
    host = blocks[::2, :per].cpu().contiguous().view(-1).pin_memory()
    pool = c.pool.clone()
    pool.view(-1, c.lay.block_stride)[::2, :per] = 0xFF
    out, lse = c.buffers()
    smla.smla_attend_hisparse(c.lay, c.params(128), pool, 0, host, host_map.cuda(), c.q, c.q_pe, sel, c.table, c.qsl, out, lse)
    ok()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---------------------------------- together ----------------------------------

def fused_inputs(lay, lens, counts, bs, seed):
    """A batch of the full shape with its cached tokens stored, and a step's new ones."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")
    need = [-(-n // bs) for n in lens]
    perm = torch.randperm(lay.num_blocks, generator=g, device="cuda").int()
    bt = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    at, slots_old, slots_new = 0, [], []
    for i, n in enumerate(lens):
        bt[i, :need[i]] = perm[at:at + need[i]]
        at += need[i]
        j = torch.arange(n, device="cuda")
        s = bt[i, j // bs].long() * bs + j % bs
        slots_old.append(s[:n - counts[i]])
        slots_new.append(s[n - counts[i]:])
    ints = lambda n: torch.randint(-8, 9, (n, 128), generator=g, device="cuda").float().to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    old, new = torch.cat(slots_old), torch.cat(slots_new)
    if old.numel():
        smla.kvpack_store(lay, pool, 0, rnd(old.numel(), 512).bfloat16(), rnd(old.numel(), 64).bfloat16(), ints(old.numel()),
                          torch.ones(old.numel(), device="cuda"), old)
    t = new.numel()
    return dict(pool=pool, bt=bt, new=(rnd(t, 512).bfloat16(), rnd(t, 64).bfloat16(), ints(t), torch.ones(t, device="cuda"), new),
                q=rnd(t, 64, 512).bfloat16(), q_pe=rnd(t, 64, 64).bfloat16(), q_idx=ints(t * 64).view(t, 64, 128),
                w=torch.full((t, 64), 0.25, device="cuda"), seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                qsl=torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("static", [False, True])
def test_fused_step_is_its_parts(static):
    lens, counts, bs = [700, 300, 65], [4, 1, 65], 64
    lay = smla.layout_init(bs, 1, 512, 64, 16, 128, 24, latent_format="e2m1")
    prm = smla.make_params(64, 64, 128, 1 / 24)
    x = fused_inputs(lay, lens, counts, bs, 1)
    t, ctx = sum(counts), max(lens)
    a, b = x["pool"].clone(), x["pool"].clone()
    out, lse = torch.empty(t, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(t, 64, device="cuda")
    topk = torch.empty(t, 128, dtype=torch.int32, device="cuda")
    step = (x["q"], x["q_pe"], x["q_idx"], x["w"], x["bt"], x["seq_lens"], x["qsl"], max(counts), ctx, out, lse)
    if static:
        smla.smla_decode_static(lay, prm, a, 0, *x["new"], *step, topk_idx_out=topk)
    else:
        ws = torch.empty(smla.workspace_size(lay, prm, t, ctx), dtype=torch.uint8, device="cuda")
        smla.smla_decode(lay, prm, a, 0, *x["new"], *step, ws, topk_idx_out=topk)
    smla.kvpack_store(lay, b, 0, *x["new"])
    assert torch.equal(a, b)
    scores = torch.empty(t, (ctx + 3) // 4 * 4, device="cuda")
    smla.smla_index_scores(lay, prm, b, 0, x["q_idx"], x["w"], x["bt"], x["seq_lens"], x["qsl"], max(counts), ctx, scores)
    top2, out2, lse2 = torch.empty_like(topk), torch.empty_like(out), torch.empty_like(lse)
    smla.smla_topk(prm, scores, x["seq_lens"], x["qsl"], top2)
    smla.smla_attend(lay, prm, b, 0, x["q"], x["q_pe"], top2, x["bt"], x["qsl"], out2, lse2)
    ok()
    assert torch.equal(topk, top2)
    torch.testing.assert_close(out.float(), out2.float(), rtol=2.0 ** -7, atol=1e-3)   # the fused step splits rows: other sums
    torch.testing.assert_close(lse, lse2, rtol=1e-5, atol=1e-5)


# ---------------------------------- calls that other tests do not make ----------------------------------

def off_alignment(t):
    """A copy of t whose first element lies 2 bytes behind a 16-byte boundary."""
    buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)[1:1 + t.numel()].view(t.shape)
    buf.copy_(t)
    return buf


def test_queries_that_are_not_16_byte_aligned():
    """Their rows come by ordinary loads instead of tensor-map copies; the results are the same bits."""
    for lens, counts in (([700, 130, 1], [1, 1, 1]), ([300, 200], [9, 5])):
        c = Case4(lens, counts, 64, seed=31)
        want = c.dense()
        c.check(want)
        sel = c.select(256)
        want_sel = c.sparse(sel)
        c.q, c.q_pe = off_alignment(c.q), off_alignment(c.q_pe)
        got, got_sel = c.dense(), c.sparse(sel)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got_sel[0], want_sel[0]) and torch.equal(got_sel[1], want_sel[1])
    ok()
