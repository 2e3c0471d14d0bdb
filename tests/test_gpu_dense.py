"""smla_attend_dense on the GPU against attention in float64 over the same cache.

Tolerance, per output element, from the roundings that the call documents.  The tensor-core path holds
the dequantised keys (scale and product: 2 x 2^-11 relative) and the probabilities (2^-11) in fp16.  Below
2^-14 fp16's step stays 2^-24: there a key is off by up to 2^-25, half a step, whatever its size.  So a
score is off by at most dS = sigma sum_d |q_d| (|K_jd| 2^-10 + 2^-25), which moves its probability by the
factor e^dS on either side of the normalisation, and
    |out - ref| <= 2^-8 |ref| + sum_j p_j |K_j| (2^-10 + 2^-11 + 2 dS_max) + 2^-25 + 1e-5 max_j |K_j|
with 2^-8 for the bf16 result, 2^-25 = sum_j p_j 2^-25 for the keys' steps near zero, and the last term
for the fp32 sums and the probabilities below 2^-14 (2^-25 each, of at most a few thousand).  lse moves by at most dS_max, plus 1e-5 (1 + |lse|) for its logarithm
and the fp32 sums.  The fp32 path of other shapes stays inside the same bounds.
"""
import numpy as np
import pytest
import torch

import paged_sparse_mla_gb300 as smla
import oracle
from tests import gpu_helpers as G

pytestmark = pytest.mark.gpu

FULL = dict(dl=512, dr=64, tile=128)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.ensure_built()


class Case:
    """A cache with random contents behind a shuffled block table; unused memory holds NaN patterns."""

    def __init__(self, lens, counts, heads, bs=64, dl=512, dr=64, tile=128, layers=1, layer=0, seed=0, key_scale=1.0,
                 q_scale=1.0, sigma=None, extra_cols=0, pad_rows=0):
        rng = np.random.default_rng(seed)
        self.lens, self.counts, self.heads, self.bs, self.layer = list(lens), list(counts), heads, bs, layer
        need = [-(-n // bs) for n in lens]
        blocks = sum(need) + 2
        self.lay = smla.layout_init(bs, layers, dl, dr, tile, 32, blocks)
        self.ref = oracle.PoolLayout(bs, layers, dl, dr, tile, 32, blocks)
        pool = np.full(self.lay.pool_bytes, 0xFF, dtype=np.uint8)   # NaN codes, scales and ropes everywhere else
        perm = rng.permutation(blocks)
        cols = max(1, max(need) + extra_cols)
        table = np.full((len(lens), cols), -1, dtype=np.int32)
        at = 0
        self.keys = []
        for b, n in enumerate(lens):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            j = np.arange(n)
            slots = table[b, j // bs].astype(np.int64) * bs + j % bs if n else np.zeros(0, np.int64)
            if n:
                to_bits = lambda x: torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
                lat = rng.standard_normal((n, dl)).astype(np.float32) * key_scale * (0.3 + rng.random((n, 1)).astype(np.float32))
                oracle.kvpack_store(self.ref, pool, layer, to_bits(lat), to_bits(rng.standard_normal((n, dr)).astype(np.float32)),
                                    np.zeros((n, 32), np.uint8), np.ones(n, np.float32), slots)
            self.keys.append(oracle.read_record(self.ref, pool, layer, slots) if n else (np.zeros((0, dl)), np.zeros((0, dr))))
        self.pool = torch.from_numpy(pool).cuda()
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.qsl = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        self.T = int(sum(counts)) + pad_rows
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.q = (torch.randn(self.T, heads, dl, generator=g, device="cuda") * q_scale).bfloat16()
        self.q_pe = (torch.randn(self.T, heads, dr, generator=g, device="cuda") * q_scale).bfloat16()
        self.sigma = 1.0 / np.sqrt(dl + dr) if sigma is None else sigma
        self.prm = smla.make_params(heads, 1, 1, self.sigma)

    def run(self, workspace=True, lse=True, stream=None, out=None):
        out = torch.full((self.T, self.heads, self.lay.d_latent), 777.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        le = torch.full((self.T, self.heads), 777.0, device="cuda") if lse else None
        n = smla.attend_dense_workspace_size(self.lay, self.prm, self.T)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if workspace and n else None
        torch.cuda.synchronize()
        smla.smla_attend_dense(self.lay, self.prm, self.pool, self.layer, self.q, self.q_pe, self.table, self.seq_lens, self.qsl, out, le,
                               workspace=ws, stream=stream)
        return out, le

    def want(self, keys=None):
        """(out, lse, out's bound, lse's bound) in float64."""
        outs, lses, bo, bl = [], [], [], []
        at = 0
        for b, (n, c) in enumerate(zip(self.lens, self.counts)):
            lat, rope = [torch.from_numpy(x).cuda() for x in (keys or self.keys)[b]]
            n = lat.shape[0]
            for i in range(c):
                q, qp = self.q[at + i].double(), self.q_pe[at + i].double()
                v = max(0, n - c + i + 1)
                if v == 0:
                    outs.append(torch.zeros(self.heads, lat.shape[1]).cuda().double())
                    lses.append(torch.full((self.heads,), -np.inf).cuda().double())
                    bo.append(torch.zeros_like(outs[-1]))
                    bl.append(torch.zeros_like(lses[-1]))
                    continue
                s = self.sigma * (q @ lat[:v].T + qp @ rope[:v].T)
                p = torch.softmax(s, -1)
                outs.append(p @ lat[:v])
                lses.append(torch.logsumexp(s, -1))
                ds = abs(self.sigma) * (2.0 ** -10 * (q.abs() @ lat[:v].abs().T).amax(-1) + 2.0 ** -25 * q.abs().sum(-1))
                bo.append(2.0 ** -8 * outs[-1].abs() + (p @ lat[:v].abs()) * (2.0 ** -10 + 2.0 ** -11 + 2 * ds[:, None]) + 2.0 ** -25 + 1e-5 * lat[:v].abs().max())
                bl.append(ds + 1e-5 * (1 + lses[-1].abs()))
            at += c
        return [torch.stack(x) for x in (outs, lses, bo, bl)]

    def check(self, got, keys=None):
        out, lse = got
        torch.cuda.synchronize()
        n = int(sum(self.counts))
        assert (out[n:] == 777).all() and (lse is None or (lse[n:] == 777).all())   # rows behind the last sequence
        if n == 0:
            return
        wo, wl, bo, bl = self.want(keys)
        e = (out[:n].double() - wo).abs()
        assert (e <= bo).all(), f"out off by {(e - bo).max():.3e} more than its bound"
        if lse is not None:
            fin = torch.isfinite(wl)
            assert (lse[:n][~fin] == -np.inf).all()
            e = (lse[:n].double() - wl).abs()[fin]
            assert (e <= bl[fin]).all(), f"lse off by {(e - bl[fin]).max():.3e} more than its bound"


def ok():
    assert smla.smla_get_last_error() == 0


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lens,counts,heads,bs", [
    ([1], [1], 64, 64),
    ([63], [1], 64, 64), ([64], [1], 64, 64), ([65], [2], 64, 64),
    ([127, 128, 129, 1], [1, 1, 1, 1], 64, 64),
    ([1000], [1], 64, 64), ([777, 33, 400], [4, 4, 4], 64, 64),
    ([300, 5, 513, 70], [7, 5, 1, 70], 64, 16),
    ([260, 90], [33, 2], 16, 64), ([260, 90], [33, 2], 5, 48), ([130], [9], 1, 7), ([200, 140], [21, 3], 24, 32),
    ([300, 64], [3, 1], 128, 64), ([150], [5], 100, 16), ([2500], [2], 65, 128),
    ([400, 400, 400], [0, 3, 0], 64, 64), ([50, 80], [50, 80], 64, 64),
])
def test_matches_float64(lens, counts, heads, bs, workspace):
    c = Case(lens, counts, heads, bs, seed=sum(lens) + heads)
    c.check(c.run(workspace))
    ok()


@pytest.mark.parametrize("lens,counts,heads,bs,dl,dr,tile", [
    ([1], [1], 8, 16, 64, 16, 64), ([100, 31, 33], [3, 1, 33], 8, 16, 64, 16, 64), ([75], [4], 3, 7, 128, 32, 128),
    ([140], [2], 16, 64, 256, 64, 64), ([90], [2], 64, 64, 512, 64, 64), ([90], [2], 64, 64, 512, 0, 128), ([90, 0], [2, 1], 9, 64, 512, 32, 128),
])
def test_other_shapes_match_float64(lens, counts, heads, bs, dl, dr, tile):
    c = Case(lens, counts, heads, bs, dl, dr, tile, seed=3)
    c.check(c.run())
    ok()


def test_many_sequences_of_uneven_length():
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(1, 700, 90)]
    counts = [int(min(n, k)) for n, k in zip(lens, rng.integers(1, 6, 90))]
    c = Case(lens, counts, 64, seed=5)
    a = c.run()
    c.check(a)
    ok()
    b = c.run()                                       # the same call again: the same bits
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_repeated_calls_give_the_same_bits():
    """Units of uneven rows and lengths, so that the two CTAs of a pair run apart: every hand-off between
    them has to hold whichever is ahead."""
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(1, 700, 90)]
    counts = [int(min(n, k)) for n, k in zip(lens, rng.integers(1, 6, 90))]
    for heads in (64, 16):
        c = Case(lens, counts, heads, seed=22)
        want = c.run()
        c.check(want)
        for _ in range(40):
            got = c.run()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ok()


def test_long_contexts_split_over_the_sms():
    c = Case([9001, 20000], [2, 1], 64, seed=6)
    split, whole = c.run(True), c.run(False)
    c.check(split)
    c.check(whole)
    ok()


def test_tokens_that_see_nothing():
    """Shards of a split context may hold none of a sequence's positions."""
    c = Case([0, 3, 0, 200], [1, 5, 2, 1], 64, seed=7)
    for ws in (True, False):
        out, lse = c.run(ws)
        c.check((out, lse))
        assert (out[0] == 0).all() and (lse[0] == -np.inf).all() and (out[1:3] == 0).all()
    ok()


def test_padded_batch_and_optional_lse():
    c = Case([70, 300], [2, 3], 64, seed=8, pad_rows=5, extra_cols=9)
    c.check(c.run())
    c.check(c.run(lse=False))
    c = Case([70], [0], 64, seed=8, pad_rows=3)
    c.check(c.run())
    ok()


def test_layers_of_one_pool():
    for layer in (0, 2):
        c = Case([150, 90], [2, 1], 64, 32, layers=3, layer=layer, seed=9)
        c.check(c.run())
    ok()


@pytest.mark.parametrize("key_scale,q_scale", [(1e-4, 1.0), (1e-6, 30.0), (100.0, 0.01), (1.0, 1e-3), (1.0, 20.0), (1e3, 1e4)])
def test_magnitudes_of_keys_and_queries(key_scale, q_scale):
    """Small latents (fp16's subnormals), large ones, and sharp softmaxes."""
    c = Case([333, 65], [3, 1], 64, seed=10, key_scale=key_scale, q_scale=q_scale)
    c.check(c.run())
    ok()


def test_growing_scores_move_the_running_maximum():
    """Scores that keep rising along the context: every tile moves the running maximum of every head."""
    c = Case([1500], [1], 64, seed=11, sigma=1.0)
    lat, rope = c.keys[0]
    j = np.arange(1500)
    c.q[:] = 0
    c.q_pe[:] = 0
    c.q_pe[..., 0] = 1
    slots = c.table[0].cpu().numpy()[j // 64].astype(np.int64) * 64 + j % 64
    rec = c.pool.view(-1, c.lay.block_stride)[:, :64 * 656].reshape(-1, 64, 656)
    ramp = torch.from_numpy(j / 8.0).bfloat16()
    b, o = torch.from_numpy(slots // 64).cuda(), torch.from_numpy(slots % 64).cuda()
    rec[b, o, 528:530] = ramp.view(torch.int16).cuda().view(torch.uint8).view(-1, 2)
    c.pool.view(-1, c.lay.block_stride)[:, :64 * 656] = rec.reshape(-1, 64 * 656)
    rope = rope.copy()
    rope[:, 0] = ramp.double().numpy()
    for ws in (True, False):
        c.check(c.run(ws), keys=[(lat, rope)])
    ok()


def test_bad_block_ids_read_as_zeros_and_latch():
    c = Case([200, 100], [1, 2], 64, seed=12)
    c.table[0, 1] = c.lay.num_blocks
    c.table[1, 0] = -1
    keys = [tuple(x.copy() for x in k) for k in c.keys]
    for x in keys[0]:
        x[64:128] = 0
    for x in keys[1]:
        x[:64] = 0
    got = c.run()
    assert smla.smla_get_last_error() == 4
    c.check(got, keys=keys)


def test_lengths_past_the_block_table_are_cut_and_latch():
    c = Case([256], [1], 64, seed=13)
    c.seq_lens[0] = 1000                              # the table's row holds 4 blocks of 64
    got = c.run()
    assert smla.smla_get_last_error() == 4
    c.check(got)


def test_values_beyond_fp16_latch_range():
    c = Case([100], [1], 64, seed=14)
    c.run()
    ok()
    rec = c.pool.view(-1, c.lay.block_stride)[int(c.table[0, 0]), :64 * 656].view(64, 656)
    rec[5, 512:516] = torch.tensor([200.0], device="cuda").view(torch.uint8)
    c.run()
    assert smla.smla_get_last_error() == 7
    c = Case([100], [1], 64, seed=14)
    rec = c.pool.view(-1, c.lay.block_stride)[int(c.table[0, 1]), :64 * 656].view(64, 656)
    rec[30, 528:530] = torch.tensor([70000.0], device="cuda").bfloat16().view(torch.uint8)
    c.run()
    assert smla.smla_get_last_error() == 7


def test_nan_query_stays_in_its_row():
    c = Case([150], [3], 64, seed=15)
    clean = c.run()[0]
    c.q[1, 7, 100] = float("nan")
    out = c.run()[0]
    bad = torch.isnan(out).any(-1)
    assert bad[1, 7] and bad.sum() == 1
    keep = ~bad
    assert torch.equal(out[keep], clean[keep])


def test_unaligned_queries_and_other_streams():
    c = Case([150, 700], [3, 1], 64, seed=16)
    want = c.run()
    buf = torch.empty(c.q.numel() + 1, dtype=torch.bfloat16, device="cuda")
    buf[1:] = c.q.flatten()
    q, c.q = c.q, buf[1:].view(c.q.shape)             # 2-byte aligned
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.q = q
    side = torch.cuda.Stream()
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_step_follows_new_lengths():
    """A captured call replays with lengths and tables changed in place, as a serving loop does."""
    c = Case([900, 500], [1, 1], 64, seed=17)
    out = torch.empty(2, 64, 512, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(smla.attend_dense_workspace_size(c.lay, c.prm, 2), dtype=torch.uint8, device="cuda")
    args = (c.lay, c.prm, c.pool, 0, c.q, c.q_pe, c.table, c.seq_lens, c.qsl, out)
    smla.smla_attend_dense(*args, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smla.smla_attend_dense(*args, workspace=ws)
    for lens in ([900, 500], [1, 499], [640, 64]):
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        c.lens = lens
        c.check((out, None), keys=[(a[:n], r[:n]) for (a, r), n in zip(c.keys, lens)])
    ok()


def test_offsets_beyond_32_bits():
    """Blocks more than 4 GiB into the pool."""
    bs, far = 64, 120_000                             # 120,000 blocks of 46 KB: 5.5 GB
    c = Case([200], [2], 64, bs, seed=18)
    lay = smla.layout_init(bs, 1, 512, 64, 128, 32, far + 8)
    pool = torch.empty(lay.pool_bytes, dtype=torch.uint8, device="cuda")
    small = c.pool.view(-1, c.lay.block_stride)
    pool.view(-1, lay.block_stride)[far:far + small.shape[0]] = small
    c.pool, c.lay = pool, lay
    c.table += far
    c.check(c.run())
    ok()


def test_equals_the_sparse_attention_over_every_position():
    c = Case([500, 129], [2, 1], 64, seed=19)
    out, lse = c.run()
    k = 512
    prm = smla.make_params(64, 1, k, c.sigma)
    sel = torch.arange(k, dtype=torch.int32, device="cuda").repeat(3, 1)
    for t, n in enumerate((499, 500, 129)):
        sel[t, n:] = -1
    so, sl = torch.empty_like(out), torch.empty_like(lse)
    smla.smla_attend(c.lay, prm, c.pool, 0, c.q, c.q_pe, sel, c.table, c.qsl, so, sl)
    ok()
    assert (so.float() - out.float()).abs().max() <= G.MAX_ERR and (sl - lse).abs().max() <= G.MAX_ERR


def test_shards_merge_to_the_whole():
    """Four context shards (round robin positions), each attended densely, merged by their lse."""
    n, shards = 331, 4
    c = Case([n], [1], 64, seed=20)
    want = c.run()
    lat, rope = c.keys[0]
    outs, lses = [], []
    recs = c.pool.view(-1, c.lay.block_stride)[:, :64 * 656].reshape(-1, 64, 656)
    j = torch.arange(n, device="cuda")
    rows = recs[c.table[0].long()[j // 64], j % 64]
    for r in range(shards):
        mine = rows[r::shards]
        lay = smla.layout_init(64, 1, 512, 64, 128, 32, 2)
        pool = torch.zeros(2, lay.block_stride, dtype=torch.uint8, device="cuda")
        for k in range(mine.shape[0]):
            pool[k // 64, (k % 64) * 656:(k % 64) * 656 + 656] = mine[k]
        o, le = torch.empty(1, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 64, device="cuda")
        smla.smla_attend_dense(lay, c.prm, pool.view(-1), 0, c.q, c.q_pe, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"),
                               torch.tensor([mine.shape[0]], dtype=torch.int32, device="cuda"), c.qsl, o, le)
        outs.append(o)
        lses.append(le)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    smla.smla_lse_merge(torch.stack(outs), torch.stack(lses), out, lse)
    ok()
    assert (out.float() - want[0].float()).abs().max() <= G.MAX_ERR and (lse - want[1]).abs().max() <= 1e-3


def test_append_query_dense_and_sparse_together():
    """A layer's step from its projections: append, query preparation, then the indexer's selection with
    the sparse attention, and the dense attention; with every position selected the two agree."""
    bs, n, heads = 64, 400, 64
    g = torch.Generator(device="cuda").manual_seed(21)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    lay = smla.layout_init(bs, 1, 512, 64, 128, 128, 8)
    pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")
    a = np.arange(4096)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    rope = smla.make_rope(torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda(), interleaved=True)
    table = torch.randperm(8, generator=g, device="cuda").int()[None, :7].contiguous()
    kv, ik = rnd(n, 576).bfloat16(), rnd(n, 128).bfloat16()
    j = torch.arange(n, device="cuda")
    slots = table[0].long()[j // bs] * bs + j % bs
    norm = 1 + 0.1 * rnd(512)
    t = 3                                             # the last tokens are this step's queries
    q = rnd(t, heads, 512).bfloat16()
    qp, qi, w = rnd(t, heads, 192).bfloat16(), rnd(t, 64, 128).bfloat16(), rnd(t, 64)
    q_pe, codes, w_out = torch.empty(t, heads, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(t, 64, 128, dtype=torch.uint8, device="cuda"), torch.empty(t, 64, device="cuda")
    seq, qsl = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, t], dtype=torch.int32, device="cuda")
    smla.kvpack_append(lay, pool, 0, kv[:n - t, :512], kv[:n - t, 512:], ik[:n - t], rope, j[:n - t], slots[:n - t].contiguous(),
                       latent_norm=norm, idx_norm=torch.ones(128, device="cuda"), idx_bias=torch.zeros(128, device="cuda"))
    smla.kvpack_append(lay, pool, 0, kv[n - t:, :512], kv[n - t:, 512:], ik[n - t:], rope, j[n - t:], slots[n - t:].contiguous(),
                       latent_norm=norm, idx_norm=torch.ones(128, device="cuda"), idx_bias=torch.zeros(128, device="cuda"))
    prm = smla.make_params(heads, 64, 2048, 1 / 24)
    smla.smla_query_prep(lay, prm, rope, j[n - t:], q_pe=qp[..., 128:], q_pe_out=q_pe, q_idx=qi, w=w, q_idx_out=codes, w_out=w_out)
    scores = torch.zeros(t, 448, device="cuda")
    smla.smla_index_scores(lay, prm, pool, 0, codes, w_out, table, seq, qsl, t, n, scores)
    sel = torch.empty(t, 2048, dtype=torch.int32, device="cuda")
    smla.smla_topk(prm, scores, seq, qsl, sel)
    so, sl = torch.empty(t, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(t, heads, device="cuda")
    smla.smla_attend(lay, prm, pool, 0, q, q_pe, sel, table, qsl, so, sl)
    do, dl = torch.empty_like(so), torch.empty_like(sl)
    ws = torch.empty(smla.attend_dense_workspace_size(lay, prm, t), dtype=torch.uint8, device="cuda")
    smla.smla_attend_dense(lay, prm, pool, 0, q, q_pe, table, seq, qsl, do, dl, workspace=ws)
    ok()
    assert (so.float() - do.float()).abs().max() <= G.MAX_ERR and (sl - dl).abs().max() <= G.MAX_ERR
    # and against float64 from the projections, within the cache's own E4M3 rounding (2^-4 of a value)
    x = kv.double()
    lat = x[:, :512] / (x[:, :512].square().mean(-1, keepdim=True) + 1e-6).sqrt() * norm.double()
    def turn(v, pos):
        ang = torch.from_numpy(a).cuda()[pos]
        z = torch.view_as_complex(v.unflatten(-1, (32, 2)).contiguous()) * torch.polar(torch.ones_like(ang), ang).view(ang.shape[0], *([1] * (v.dim() - 2)), 32)
        return torch.view_as_real(z).flatten(-2)
    kpe = turn(x[:, 512:], j)
    qpe = turn(qp[..., 128:].double(), j[n - t:])
    s = (torch.einsum("thd,nd->thn", q.double(), lat) + torch.einsum("thd,nd->thn", qpe, kpe)) / 24
    s.masked_fill_(j[None, None] > j[n - t:, None, None], -np.inf)
    want = torch.softmax(s, -1) @ lat
    rel = ((do.double() - want).norm() / want.norm()).item()
    assert rel <= 2.0 ** -4, rel
