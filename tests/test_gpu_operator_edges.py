"""Calls of kvpack_append, smla_query_prep and smla_attend_dense at their edges: many sequences, more query
tokens than positions, pages of one token, every head count's ends, two captured steps at once, caches
beyond 4 GiB, broadcast inputs, empty calls.  Values are checked against float64 with the bounds that
tests/test_gpu_dense.py and tests/test_gpu_prep.py derive, or for equality of bits."""
import numpy as np
import pytest
import torch

import paged_sparse_mla_gb300 as smla
from tests import gpu_helpers as G
from tests.test_gpu_dense import Case, ok
from tests.test_gpu_prep import table, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.ensure_built()


@pytest.mark.parametrize("workspace", [True, False])
def test_more_sequences_than_a_block_has_threads(workspace):
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(0, 90, 2000)]
    counts = [int(x) for x in rng.integers(0, 3, 2000)]
    c = Case(lens, counts, 16, 16, seed=31)
    c.check(c.run(workspace))
    ok()


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lens,counts,heads", [
    ([40, 0, 7], [300, 5, 9], 64),       # units that see nothing, then one that sees a little
    ([500, 130], [700, 131], 128),
])
def test_more_query_tokens_than_positions(lens, counts, heads, workspace):
    c = Case(lens, counts, heads, seed=32)
    c.check(c.run(workspace))
    ok()


@pytest.mark.parametrize("lens,counts,heads,bs", [
    ([300], [130], 1, 64), ([300, 129], [44, 1], 3, 1), ([200], [3], 127, 64), ([257, 31], [2, 2], 128, 1),
    ([700], [2], 63, 256), ([700], [5], 33, 3),
])
def test_head_counts_and_pages(lens, counts, heads, bs):
    c = Case(lens, counts, heads, bs, seed=33, extra_cols=3, pad_rows=2)
    c.check(c.run())
    ok()


@pytest.mark.parametrize("sigma", [-0.05, 0.0, 0.7])
def test_softmax_scales(sigma):
    c = Case([333, 64], [2, 1], 64, seed=34, sigma=sigma)
    c.check(c.run())
    ok()


def test_scales_of_every_size_side_by_side():
    """Neighbouring keys and the quant tiles of one key with scales from far below fp16's normal values to large."""
    rng = np.random.default_rng(44)
    size = np.array([1e-8, 1e-6, 1e-5, 1e-4, 1e-3, 0.03, 1.0, 10.0])[rng.integers(0, 8, (300, 4))].repeat(128, 1)
    c = Case([300], [3], 64, seed=44, key_scale=size)
    c.check(c.run())
    c = Case([300], [3], 64, 7, seed=44, key_scale=np.minimum(size, 1e-5))
    c.check(c.run())
    ok()


def test_scales_of_either_sign():
    """A negative scale (no store writes one) negates its 128 dims, and counts by its size for the range."""
    c = Case([150], [2], 64, seed=45)
    lat, rope = c.keys[0][0].copy(), c.keys[0][1]
    blocks = c.pool.view(-1, c.lay.block_stride)
    for pos, tile in ((0, 0), (64, 3), (149, 2)):
        rec = blocks[int(c.table[0, pos // 64]), :64 * 656].view(64, 656)
        sc = rec[pos % 64, 512 + 4 * tile:516 + 4 * tile]
        sc.copy_((-sc.clone().view(torch.float32)).view(torch.uint8))
        lat[pos, 128 * tile:128 * tile + 128] *= -1
    c.check(c.run(), keys=[(lat, rope)])
    ok()
    sc.copy_(torch.tensor([-200.0], device="cuda").view(torch.uint8))
    c.run()
    assert smla.smla_get_last_error() == 7


@pytest.mark.parametrize("value", [0x7F, 0xFF])
def test_nan_in_the_cache(value):
    """At a position that every token sees it is theirs; where only the last token sees it, the others' zero
    weights would carry it too: latched.  Past the sequence it is never read."""
    for lens, pos, latched in (([300], 100, False), ([300], 299, True), ([256], 255, True), ([300], 300, False)):
        c = Case(lens, [2], 64, seed=43)
        rec = c.pool.view(-1, c.lay.block_stride)[int(c.table[0, pos // 64]), :64 * 656].view(64, 656)
        rec[pos % 64, 7] = value
        out, _ = c.run()
        assert smla.smla_get_last_error() == (7 if latched else 0)
        nan = torch.isnan(out)
        if pos == 100:
            assert nan[..., 7].all()
        elif pos == 300:
            assert not nan.any()
        else:
            assert nan[1, :, 7].all()


def test_a_workspace_that_is_too_small_is_not_used():
    c = Case([900], [1], 64, seed=35)
    want, _ = c.run(workspace=False)
    out = torch.empty_like(want)
    ws = torch.full((4096,), 0x5A, dtype=torch.uint8, device="cuda")
    smla.smla_attend_dense(c.lay, c.prm, c.pool, 0, c.q, c.q_pe, c.table, c.seq_lens, c.qsl, out, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and (ws == 0x5A).all()
    ok()


def test_two_captured_steps_at_once():
    """Two graphs with a workspace each, replayed on two streams while both run, give an eager call's bits."""
    cases = [Case([3000, 200], [1, 4], 64, seed=36), Case([2000], [30], 128, 16, seed=37)]
    want, outs, graphs, streams, keep = [], [], [], [], []
    for c in cases:
        want.append(c.run()[0])
        outs.append(torch.zeros_like(want[-1]))
        keep.append(torch.zeros(smla.attend_dense_workspace_size(c.lay, c.prm, c.T), dtype=torch.uint8, device="cuda"))
        streams.append(torch.cuda.Stream())
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            smla.smla_attend_dense(c.lay, c.prm, c.pool, 0, c.q, c.q_pe, c.table, c.seq_lens, c.qsl, outs[-1], workspace=keep[-1])
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    ok()


def test_calls_in_turn_share_a_workspace():
    """A short call after a long one must not join parts that the long one left behind."""
    long, short = Case([6000, 500], [1, 1], 64, seed=38), Case([100], [3], 64, seed=39)
    ws = torch.zeros(smla.attend_dense_workspace_size(long.lay, long.prm, 2), dtype=torch.uint8, device="cuda")
    want = [c.run()[0] for c in (long, short)]
    outs = [torch.empty_like(w) for w in want]
    for _ in range(3):
        for c, o in zip((long, short), outs):
            smla.smla_attend_dense(c.lay, c.prm, c.pool, 0, c.q, c.q_pe, c.table, c.seq_lens, c.qsl, o, workspace=ws)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    ok()


def test_append_beyond_32_bits():
    """Tokens stored more than 4 GiB into the pool equal the same tokens stored at its start."""
    bs, far, n = 64, 110_000, 150                      # blocks of 50,432 bytes: 5.5 GB
    lay, small = smla.layout_init(bs, 1, 512, 64, 128, 128, far + 4), smla.layout_init(bs, 1, 512, 64, 128, 128, 4)
    g = torch.Generator(device="cuda").manual_seed(40)
    kv, ik, norm = wide(n, 576, 576, g), wide(n, 128, 128, g), torch.rand(512, generator=g, device="cuda")
    rope = smla.make_rope(torch.from_numpy(table(500, 64)).cuda(), interleaved=True)
    pos, slots = torch.arange(n, device="cuda"), torch.randperm(4 * bs, generator=g, device="cuda")[:n].contiguous()
    want = torch.zeros(small.pool_bytes, dtype=torch.uint8, device="cuda")
    pool = torch.empty(lay.pool_bytes, dtype=torch.uint8, device="cuda")
    tail = pool.view(-1, lay.block_stride)[far:]
    for shape in (512, 513):                           # 16-byte rows, and rows that are not
        x = torch.empty(n, shape + 64, dtype=torch.bfloat16, device="cuda")
        x[:, :512], x[:, shape:] = kv[:, :512], kv[:, 512:]
        want.zero_()
        tail.zero_()
        for lo, p, off in ((small, want, 0), (lay, pool, far * bs)):
            smla.kvpack_append(lo, p, 0, x[:, :512], x[:, shape:], ik, rope, pos, slots + off, latent_norm=norm)
        assert torch.equal(tail.flatten(), want)
    ok()


def test_broadcast_inputs():
    """Expanded tensors (strides of zero) give what their copies give."""
    g = torch.Generator(device="cuda").manual_seed(41)
    lay, prm = smla.layout_init(16, 1, 512, 64, 128, 128, 4), smla.make_params(16, 8, 16, 1.0)
    rope = smla.make_rope(torch.from_numpy(table(100, 64)).cuda(), interleaved=False)
    n, pos = 7, torch.arange(7, device="cuda")
    row = [wide(1, w, w, g) for w in (512, 64, 128)]
    pools = []
    for form in (lambda x: x.expand(n, -1), lambda x: x.expand(n, -1).contiguous()):
        pools.append(torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda"))
        smla.kvpack_append(lay, pools[-1], 0, *map(form, row), rope, pos, pos)
    assert torch.equal(*pools) and pools[0].any()
    pe, ix = torch.randn(n, 1, 64, generator=g, device="cuda").bfloat16(), torch.randn(1, 8, 128, generator=g, device="cuda").bfloat16()
    got = []
    for form in (lambda x: x, torch.Tensor.contiguous):
        got.append((torch.empty(n, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 8, 128, dtype=torch.uint8, device="cuda"),
                    torch.empty(n, 8, device="cuda")))
        smla.smla_query_prep(lay, prm, rope, pos, q_pe=form(pe.expand(n, 16, 64)), q_pe_out=got[-1][0], q_idx=form(ix.expand(n, 8, 128)),
                             w=torch.ones(n, 8, device="cuda"), q_idx_out=got[-1][1], w_out=got[-1][2])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    ok()


@pytest.mark.parametrize("heads,idx_heads,norm,interleaved", [(64, 64, True, False), (5, 7, True, True), (130, 0, False, True),
                                                              (0, 33, False, False), (1, 1, True, True)])
def test_many_queries_equal_a_few_at_a_time(heads, idx_heads, norm, interleaved):
    """A chunk's queries (three warps a token) have the bits of the same queries in small calls (twelve)."""
    g = torch.Generator(device="cuda").manual_seed(42)
    lay, prm = smla.layout_init(16, 1, 512, 64, 128, 128, 4), smla.make_params(max(heads, 1), max(idx_heads, 1), 16, 1.0)
    rope = smla.make_rope(torch.from_numpy(table(5000, 64)).cuda(), interleaved=interleaved, idx_interleaved=not interleaved)
    n = 1201
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda")
    pe, ix = torch.randn(n, heads, 64, generator=g, device="cuda").bfloat16(), torch.randn(n, idx_heads, 128, generator=g, device="cuda").bfloat16()
    w, kn = torch.randn(n, idx_heads, generator=g, device="cuda"), torch.rand(128, generator=g, device="cuda") if norm else None
    got = []
    for step in (n, 100):
        po = torch.full((n, heads, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        co, wo = torch.full((n, idx_heads, 128), 9, dtype=torch.uint8, device="cuda"), torch.full((n, idx_heads), 5.0, device="cuda")
        for a in range(0, n, step):
            b = slice(a, min(n, a + step))
            smla.smla_query_prep(lay, prm, rope, pos[b], q_pe=pe[b] if heads else None, q_pe_out=po[b] if heads else None,
                                 q_idx=ix[b] if idx_heads else None, w=w[b], q_idx_out=co[b], w_out=wo[b], idx_norm=kn)
        got.append((po, co, wo))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))
    ok()


def test_calls_without_tokens():
    lay, prm = smla.layout_init(64, 1, 512, 64, 128, 128, 2), smla.make_params(8, 4, 16, 1.0)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    pool = z(lay.pool_bytes, dt=torch.uint8)
    rope = smla.make_rope(torch.from_numpy(table(8, 64)).cuda(), interleaved=True)
    none = z(0, dt=torch.int64)
    smla.kvpack_append(lay, pool, 0, z(0, 512), z(0, 64), z(0, 128), rope, none, none)
    smla.smla_query_prep(lay, prm, rope, none, q_pe=z(0, 8, 64), q_pe_out=z(0, 8, 64), q_idx=z(0, 4, 128), w=z(0, 4, dt=torch.float32),
                         q_idx_out=z(0, 4, 128, dt=torch.uint8), w_out=z(0, 4, dt=torch.float32))
    one = z(1, 1, dt=torch.int32)
    smla.smla_attend_dense(lay, prm, pool, 0, z(0, 8, 512), z(0, 8, 64), one, one[0], z(2, dt=torch.int32), z(0, 8, 512))
    # rows, but no sequence has any of them: left as they were
    out = torch.full((3, 8, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = z(smla.attend_dense_workspace_size(lay, prm, 3), dt=torch.uint8)
    for w in (ws, None):
        smla.smla_attend_dense(lay, prm, pool, 0, z(3, 8, 512), z(3, 8, 64), one, one[0] + 20, z(2, dt=torch.int32), out, workspace=w)
    torch.cuda.synchronize()
    assert (out == 5).all() and not pool.any()
    # every slot unused
    slots = torch.full((5,), -1, device="cuda")
    smla.kvpack_append(lay, pool, 0, z(5, 512) + 1, z(5, 64) + 1, z(5, 128) + 1, rope, slots + 1, slots)
    torch.cuda.synchronize()
    assert not pool.any()
    ok()
