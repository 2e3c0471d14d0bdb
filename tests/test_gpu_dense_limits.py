"""smla_attend_dense at the ends of what its fp16 operands hold: latent scales around the last one whose
largest code stays finite, tails of small weights, and scores of any size.  Values are checked with the
bounds that tests/test_gpu_dense.py derives."""
import numpy as np
import pytest
import torch

import paged_sparse_mla_gb300 as smla
from tests import gpu_helpers as G
from tests.test_gpu_dense import Case, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.ensure_built()


def record(c, pos):
    """The 656 bytes of position `pos` of the first sequence."""
    return c.pool.view(-1, c.lay.block_stride)[int(c.table[0, pos // c.bs]), :c.bs * 656].view(c.bs, 656)[pos % c.bs]


END = 146.1875  # half way between fp16's 146.125 (x 448 = 65,464) and 146.25 (x 448 = 65,520, which fp16 rounds to infinity)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("pos", [5, 70, 199])
@pytest.mark.parametrize("scale,latched", [(146.125, False), (146.18, False), (float(np.nextafter(np.float32(END), np.float32(0))), False),
                                           (END, True), (146.2, True), (65504 / 448, True), (146.25, True)])
def test_scales_up_to_the_last_finite_one(scale, latched, pos, sign):
    """A tile with code 448 of either sign is exact to fp16's roundings up to the last scale whose rounded value
    keeps it finite; from the first that does not, the call latches."""
    c = Case([200], [3], 64, seed=51, q_scale=1e-4)
    rec = record(c, pos)
    rec[384 + 9] = 0x7E                                   # +448 and -448 of the last tile
    rec[384 + 10] = 0xFE
    s = np.float32(sign * scale)
    rec[524:528] = torch.from_numpy(np.array([s])).cuda().view(torch.uint8)
    got = c.run()
    if latched:
        assert smla.smla_get_last_error() == 7
        return
    ok()
    lat, rope = c.keys[0][0].copy(), c.keys[0][1]
    lat[pos, 384:512] = rec[384:512].view(torch.float8_e4m3fn).double().cpu().numpy() * float(s)
    c.check(got, keys=[(lat, rope)])


class Sink:
    """A long cache made on the GPU: latents of codes around 160 and scales near 1 / 160 (values near one), ropes
    zero, and one position whose value is zero and whose score stands `gap` above all others': query rows hold a
    small random latent part and 1 in the first rope dim, which is gap / sigma at that position."""

    def __init__(self, n, gap, at, count, heads=8, seed=53, bs=64):
        g = torch.Generator(device="cuda").manual_seed(seed)
        blocks = -(-n // bs)
        self.heads, self.count, self.n, self.sigma = heads, count, n, 1 / 24
        self.lay = smla.layout_init(bs, 1, 512, 64, 128, 32, blocks)
        self.pool = torch.zeros(blocks, self.lay.block_stride, dtype=torch.uint8, device="cuda")
        rec = torch.as_strided(self.pool, (blocks, bs, 656), (self.lay.block_stride, 656, 1))
        codes = (160 + 40 * torch.randn(blocks, bs, 512, generator=g, device="cuda")).clamp_(-448, 448).to(torch.float8_e4m3fn)
        scales = (0.8 + 0.4 * torch.rand(blocks, bs, 4, generator=g, device="cuda")) / 160
        rope = torch.zeros(blocks, bs, 64, dtype=torch.bfloat16, device="cuda")
        codes.view(torch.uint8)[at // bs, at % bs] = 0
        rope[at // bs, at % bs, 0] = gap / self.sigma
        rec[..., :512], rec[..., 512:528], rec[..., 528:] = codes.view(torch.uint8), scales.view(torch.uint8), rope.view(torch.uint8)
        self.lat = (codes.double().unflatten(-1, (4, 128)) * scales.double()[..., None]).view(-1, 512)[:n]
        self.rope = rope.double().view(-1, 64)[:n]
        self.pool = self.pool.view(-1)
        self.table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None].contiguous()
        self.q = (0.01 * torch.randn(count, heads, 512, generator=g, device="cuda")).bfloat16()
        self.q_pe = torch.zeros(count, heads, 64, dtype=torch.bfloat16, device="cuda")
        self.q_pe[..., 0] = 1
        self.prm = smla.make_params(heads, 1, 1, self.sigma)

    def run(self, workspace):
        out = torch.empty(self.count, self.heads, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(self.count, self.heads, device="cuda")
        ws = torch.empty(smla.attend_dense_workspace_size(self.lay, self.prm, self.count), dtype=torch.uint8, device="cuda")
        smla.smla_attend_dense(self.lay, self.prm, self.pool, 0, self.q, self.q_pe, self.table,
                               torch.tensor([self.n], dtype=torch.int32, device="cuda"),
                               torch.tensor([0, self.count], dtype=torch.int32, device="cuda"), out, lse, workspace=ws if workspace else None)
        ok()
        return out, lse

    def check(self, got, tokens):
        """The bounds of tests/test_gpu_dense.py without their allowance for small probabilities, which here is
        n 2^-32 max |K|: a probability is held as a multiple of 2^-24 (off by 2^-25) where the largest is at least
        2^7 (2^15 at most, 2^8 below it at least), so n of them lose n 2^-25 / 2^7 of the sum's weight at most.  The fp32 sums
        (blocks of 128 products, then one addition a tile, 2^-24 each at most) stay below n / 128 2^-24 |out|."""
        out, lse = got
        for t in tokens:
            v = self.n - self.count + t + 1
            q, lat = self.q[t].double(), self.lat[:v]
            s = self.sigma * (q @ lat.T + self.q_pe[t].double() @ self.rope[:v].T)
            p = torch.softmax(s, -1)
            want, size = p @ lat, p @ lat.abs()
            ds = self.sigma * (2.0 ** -10 * (q.abs() @ lat.abs().T).amax(-1) + 2.0 ** -25 * q.abs().sum(-1))[:, None]
            bound = 2.0 ** -8 * want.abs() + size * (2.0 ** -10 + 2.0 ** -11 + 2 * ds + v / 128 * 2.0 ** -24) + 2.0 ** -25 + v * 2.0 ** -32 * lat.abs().max()
            e = (out[t].double() - want).abs()
            assert (e <= bound).all(), f"token {t}: off by {(e / bound).max():.1f} times the bound, {(e / want.abs()).max():.3f} of the value"
            wl = torch.logsumexp(s, -1)
            assert ((lse[t].double() - wl).abs() <= ds[:, 0] + 1e-5 * (1 + wl.abs())).all()


@pytest.mark.parametrize("at", [0, 131_000])
@pytest.mark.parametrize("gap", [12.0, 16.0, 17.5, 18.5])
def test_a_dominant_position_leaves_the_tail_its_weight(gap, at):
    """An attention sink: one position of zero value far above 262,143 others, whose sum still makes the output."""
    c = Sink(262_144, gap, at, 1)
    c.check(c.run(False), [0])
    c.check(c.run(True), [0])


@pytest.mark.parametrize("gap", [12.0, 17.5])
def test_a_dominant_position_before_a_chunk(gap):
    """The same for a chunk, whose units each see the whole prefix on one pair of SMs or two."""
    c = Sink(200_000, gap, 3, 1300)
    for workspace in (True, False):
        c.check(c.run(workspace), [0, 1, 500, 1024, 1299])


@pytest.mark.parametrize("q_scale", [1e4, 1e5, 1e6, 1e8, 1e20])
def test_scores_beyond_fp32s_integers(q_scale):
    """Scores so large that neighbouring fp32 values are whole powers of two apart in probability: weights come from
    differences of scores, so that the outputs stay averages of the values."""
    c = Case([333, 65], [3, 1], 64, seed=10, key_scale=1e3, q_scale=q_scale)
    for workspace in (True, False):
        out, lse = c.run(workspace)
        ok()
        c.check((out, lse))
        assert torch.isfinite(lse).all()
        for row, (lat, _) in zip((0, 3), c.keys):
            assert out[row].abs().max() <= 1.01 * np.abs(lat).max()
    # one position whose score is the largest by far more than the keys' roundings takes everything
    c.q[:], c.q_pe[:] = 0, 0
    c.q_pe[..., 0] = q_scale
    slots = [int(c.table[b, j // 64]) for b, j in ((0, 100), (1, 30))]
    blocks = c.pool.view(-1, c.lay.block_stride)
    for blk, j in zip(slots, (100, 30)):
        blocks[blk, (j % 64) * 656 + 528:(j % 64) * 656 + 530] = torch.tensor([1e4], device="cuda").bfloat16().view(torch.uint8)
    for workspace in (True, False):
        out, _ = c.run(workspace)
        ok()
        for t, (lat, j) in enumerate(((c.keys[0][0], 100),) * 3 + ((c.keys[1][0], 30),)):
            want = torch.from_numpy(lat[j]).cuda()
            assert ((out[t].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11) + 2.0 ** -25).all()


@pytest.mark.parametrize("bs", [3_300_000, 3_300_001])
def test_records_beyond_2_gib_of_one_page(bs):
    """A sequence in one page whose last records lie more than 2^31 bytes into it: all zeros but for its first 100
    and last 300 positions (a page size of either kind: multiples of 16, and others)."""
    g = torch.Generator(device="cuda").manual_seed(56)
    n, heads, sigma = bs - 7, 4, 1 / 24
    lay = smla.layout_init(bs, 1, 512, 64, 128, 32, 1)
    pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")
    rec = pool[:bs * 656].view(bs, 656)
    at = torch.cat([torch.arange(100), torch.arange(n - 300, n)]).cuda()
    assert int(at[-1]) * 656 > 2 ** 31
    codes = (100 * torch.randn(400, 512, generator=g, device="cuda")).clamp_(-448, 448).to(torch.float8_e4m3fn)
    scales = (0.8 + 0.4 * torch.rand(400, 4, generator=g, device="cuda")) / 100
    rope = torch.zeros(400, 64, dtype=torch.bfloat16, device="cuda")
    rope[:, 0] = 8 / sigma
    rec[at] = torch.cat([codes.view(torch.uint8), scales.view(torch.uint8), rope.view(torch.uint8)], 1)
    rec[n:] = 255                                             # NaN behind the sequence
    lat = (codes.double().unflatten(-1, (4, 128)) * scales.double()[..., None]).view(400, 512)
    q = (0.1 * torch.randn(2, heads, 512, generator=g, device="cuda")).bfloat16()
    q_pe = torch.zeros(2, heads, 64, dtype=torch.bfloat16, device="cuda")
    q_pe[..., 0] = 1
    prm = smla.make_params(heads, 1, 1, sigma)
    ws = torch.empty(smla.attend_dense_workspace_size(lay, prm, 2), dtype=torch.uint8, device="cuda")
    table, lens, qsl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0]], [n], [0, 2]))
    for workspace in (ws, None):
        out, lse = torch.empty(2, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, heads, device="cuda")
        smla.smla_attend_dense(lay, prm, pool, 0, q, q_pe, table, lens, qsl, out, lse, workspace=workspace)
        ok()
        for t in range(2):
            seen = 399 + t
            s = sigma * (q[t].double() @ lat[:seen].T) + sigma * float(rope[0, 0])
            total = s.exp().sum(-1, keepdim=True) + (n - 400)
            want, size = s.exp() @ lat[:seen] / total, s.exp() @ lat[:seen].abs() / total
            ds = sigma * (2.0 ** -10 * (q[t].double().abs() @ lat.abs().T).amax(-1) + 2.0 ** -25 * q[t].double().abs().sum(-1))[:, None]
            bound = 2.0 ** -8 * want.abs() + size * (2.0 ** -10 + 2.0 ** -11 + 2 * ds + n / 128 * 2.0 ** -24) + 2.0 ** -25 + 400 * 2.0 ** -32 * lat.abs().max()
            assert ((out[t].double() - want).abs() <= bound).all()
            wl = total.log()[:, 0]
            assert ((lse[t].double() - wl).abs() <= ds[:, 0] + n / 128 * 2.0 ** -24 + 1e-5 * (1 + wl.abs())).all()


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("count", [1, 9])
def test_the_longest_length_on_a_short_table(count, workspace):
    """Every token sees what the row holds, four blocks of 64."""
    c = Case([256], [count], 64, seed=57)
    c.seq_lens[0] = 2 ** 31 - 1
    out, lse = c.run(workspace)
    assert smla.smla_get_last_error() == 4
    q, q_pe, c.counts = c.q, c.q_pe, [1]
    for t in range(count):
        c.q, c.q_pe = q[t:t + 1], q_pe[t:t + 1]
        wo, wl, bo, bl = c.want()
        assert ((out[t:t + 1].double() - wo).abs() <= bo).all() and ((lse[t:t + 1].double() - wl).abs() <= bl).all()


def test_positions_up_to_the_last_that_is_visited():
    """A row of 513 pages of 2^22 tokens, all one page of zeros, and the longest length: 2^31 - 1024 positions count."""
    bs = 1 << 22
    lay = smla.layout_init(bs, 1, 512, 64, 128, 32, 1)
    pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, 513, dtype=torch.int32, device="cuda")
    prm = smla.make_params(2, 1, 1, 1 / 24)
    q, q_pe = torch.ones(1, 2, 512, dtype=torch.bfloat16, device="cuda"), torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(smla.attend_dense_workspace_size(lay, prm, 1), dtype=torch.uint8, device="cuda")
    lens, qsl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([2 ** 31 - 1], [0, 1]))
    out, lse = torch.full_like(q, 7), torch.empty(1, 2, device="cuda")
    smla.smla_attend_dense(lay, prm, pool, 0, q, q_pe, table, lens, qsl, out, lse, workspace=ws)
    assert smla.smla_get_last_error() == 4
    want = np.log(2.0 ** 31 - 1024)
    assert (out == 0).all() and ((lse - want).abs() <= 1e-5 * (1 + want)).all()


def test_steps_in_a_row_share_a_workspace():
    """Captured steps of other queries and lengths one after another on one workspace, as the layers of a model: each
    joins its own parts, not those that the step before left at the same place."""
    cases = [Case([5000 - 700 * i, 300], [1, 2], 64, seed=60 + i) for i in range(6)]
    want = [c.run()[0] for c in cases]
    ws = torch.empty(smla.attend_dense_workspace_size(cases[0].lay, cases[0].prm, 3), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, o in zip(cases, outs):
            smla.smla_attend_dense(c.lay, c.prm, c.pool, 0, c.q, c.q_pe, c.table, c.seq_lens, c.qsl, o, workspace=ws)
    for _ in range(30):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    ok()


def test_a_cache_of_small_latents():
    """Relative accuracy where every tile's largest value is about the smallest documented one, 2^-14: the keys'
    steps of 2^-25 are then 2^-11 of it.  Of smaller caches the sparse call over every position is exact to
    bf16's roundings: 2^-8 each of the key, its weight, the sum of weights and the result."""
    for scale, sparse in ((2.0 ** -14 / 0.3, False), (1e-9, True)):
        c = Case([300], [1], 64, seed=58, key_scale=scale)
        lat = torch.from_numpy(c.keys[0][0]).cuda()
        tops = lat.view(300, 4, 128).abs().amax(-1)
        assert sparse or float(tops.min()) >= 2.0 ** -14
        if sparse:
            prm = smla.make_params(64, 1, 512, c.sigma)
            sel = torch.arange(512, dtype=torch.int32, device="cuda")[None].clone()
            sel[:, 300:] = -1
            out, lse = torch.empty(1, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 64, device="cuda")
            smla.smla_attend(c.lay, prm, c.pool, 0, c.q, c.q_pe, sel, c.table, c.qsl, out, lse)
        else:
            out, lse = c.run()
        ok()
        s = c.sigma * (c.q[0].double() @ lat.T + c.q_pe[0].double() @ torch.from_numpy(c.keys[0][1]).cuda().T)
        p = torch.softmax(s, -1)
        ds = c.sigma * (2.0 ** -8 if sparse else 2.0 ** -10) * (c.q[0].double().abs() @ lat.abs().T).amax(-1)[:, None]
        ds = ds + (0 if sparse else c.sigma * 2.0 ** -25 * c.q[0].double().abs().sum(-1)[:, None])
        size = p @ tops.repeat_interleave(128, 1)             # every error is relative to the tiles' largest values
        want = p @ lat
        bound = 2.0 ** -8 * want.abs() + size * ((3 * 2.0 ** -8 if sparse else 2.0 ** -10 + 2 * 2.0 ** -11) + 2 * ds) + 1e-5 * tops.max()
        assert ((out[0].double() - want).abs() <= bound).all()
