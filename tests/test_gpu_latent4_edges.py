"""4-bit latents: the calls that the documentation allows and the plain cases do not make."""
import numpy as np
import pytest
import torch

import paged_sparse_mla_gb300 as smla
from tests import gpu_helpers as G
from tests.latent4_cases import P_BF16, Case4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.ensure_built()


def ok():
    assert smla.smla_get_last_error() == 0


def records(c):
    """The pool's records as a writable view [blocks, block_size, bytes] (one layer)."""
    return c.pool.as_strided((c.lay.num_blocks, c.bs, c.lay.rec_stride), (c.lay.block_stride, c.lay.rec_stride, 1))


def set_rope(c, b, values):
    """Rope value 0 of sequence b's positions, in the cache and in the keys that the expectation reads."""
    n = len(values)
    v = torch.as_tensor(values).bfloat16()
    j = np.arange(n)
    blk = c.table[b].cpu().numpy()[j // c.bs]
    view = records(c)
    view[torch.from_numpy(blk).long().cuda(), torch.from_numpy(j % c.bs).cuda(), 288:290] = v.view(torch.int16).cuda().view(torch.uint8).view(-1, 2)
    lat, rope = c.keys[b]
    rope = rope.copy()
    rope[:, 0] = v.double().numpy()
    c.keys[b] = (lat, rope)


# ---------------------------------- geometry ----------------------------------

@pytest.mark.parametrize("workspace", [True, False])
def test_more_sequences_than_a_block_has_threads(workspace):
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(1, 40, 1500)]
    counts = [int(x) for x in rng.integers(0, 2, 1500)]
    c = Case4(lens, counts, 8, 16, seed=1)
    c.check(c.dense(workspace))
    sel = c.select(20)
    c.check(c.sparse(sel, workspace), sel, weight=P_BF16)
    ok()


@pytest.mark.parametrize("counts", [[9] + [0] * 11, [1] * 11 + [1], [0] * 8 + [3, 0, 5, 0], [2, 1, 0, 1]])
@pytest.mark.parametrize("heads", [64, 24, 5])
def test_uneven_token_counts(counts, heads):
    lens = [130 + 7 * i for i in range(len(counts))]
    c = Case4(lens, counts, heads, seed=sum(counts) + heads, pad_rows=2)
    for ws in (True, False):
        c.check(c.dense(ws))
    ok()


def test_more_query_tokens_than_positions():
    c = Case4([3, 0, 1, 200], [5, 2, 1, 1], 16, seed=2)
    for ws in (True, False):
        c.check(c.dense(ws))
    ok()


@pytest.mark.parametrize("tokens", [159, 210])
def test_more_selections_than_sms(tokens):
    """Rows cut over the SMs (few more than SMs) and left whole (one SM's last round well filled)."""
    c = Case4([1300, 700], [tokens - 5, 5], 16, seed=tokens)
    sel = c.select(1024)
    c.check(c.sparse(sel), sel)
    assert all(torch.equal(x, y) for x, y in zip(c.sparse(sel), c.sparse(sel)))


@pytest.mark.parametrize("top_k", [1, 127, 129, 4096, 5000])
def test_selections_of_any_length(top_k):
    c = Case4([6000, 90, 1], [2, 1, 1], 64, seed=top_k)
    sel = c.select(top_k)
    for ws in (True, False):
        c.check(c.sparse(sel, ws), sel, weight=P_BF16)
    ok()


def test_the_same_position_twice_counts_twice():
    c = Case4([300], [2], 64, seed=3)
    sel = c.select(200)
    sel[:, 100:150] = sel[:, :50]
    c.check(c.sparse(sel), sel, weight=P_BF16)
    ok()


@pytest.mark.parametrize("masked", [1, 128, 130, 256, 511])
def test_masked_entries_before_the_first(masked):
    """The first tiles of a row hold no position: its maximum begins with the first that does."""
    c = Case4([900], [3], 64, seed=masked)
    sel = c.select(512)
    sel[:2, :masked] = -1
    for ws in (True, False):
        c.check(c.sparse(sel, ws), sel, weight=P_BF16)
    ok()


def test_selected_positions_without_a_page():
    c = Case4([100, 60], [1, 1], 64, 16, seed=4)
    sel = c.select(40)
    sel[0, 3] = c.table.shape[1] * 16          # past the block-table row: reads as zeros, latched
    sel[1, 0] = 2 ** 31 - 1
    got = c.sparse(sel)
    assert smla.smla_get_last_error() == 4
    keys = [tuple(np.concatenate([x, np.zeros((1, x.shape[1]))]) for x in k) for k in c.keys]
    plain = sel.clone()
    plain[0, 3], plain[1, 0] = 100, 60
    c.check(got, plain, keys, weight=P_BF16)


# ---------------------------------- values ----------------------------------

@pytest.mark.parametrize("sigma", [-0.05, 0.0, 1e-30, 3.0])
def test_softmax_scales(sigma):
    c = Case4([400, 77], [1, 1], 64, seed=5, sigma=sigma)
    c.check(c.dense())
    sel = c.select(300)
    c.check(c.sparse(sel), sel, weight=P_BF16)
    ok()


@pytest.mark.parametrize("n,step", [(1500, 1 / 8), (1500, -1 / 8), (2000, 1 / 64)])
def test_scores_that_rise_or_fall_along_the_context(n, step):
    """Every tile moves the running maximum of every row, or none does."""
    c = Case4([n, 700], [1, 1], 64, seed=6, sigma=1.0)
    c.q[:] = 0
    c.q_pe[:] = 0
    c.q_pe[..., 0] = 1
    c.q_pe[:, 7, 0] = -1                        # one head the other way
    for b, m in enumerate(c.lens):
        set_rope(c, b, np.arange(m) * step)
    for ws in (True, False):
        c.check(c.dense(ws))
    sel = c.select(640)
    for ws in (True, False):
        c.check(c.sparse(sel, ws), sel, weight=P_BF16)
    ok()


@pytest.mark.parametrize("at", [0, 600, 1499])
def test_one_position_far_above_the_others(at):
    """20 powers of e above 1,499 others: their weights are held to 2^-32 of the largest (fp16 probabilities, lifted by 2^7)."""
    c = Case4([1500], [1], 64, seed=7, sigma=1.0)
    c.q[:] = 0
    c.q_pe[:] = 0
    c.q_pe[..., 0] = 1
    ramp = np.zeros(1500)
    ramp[at] = 12.0
    set_rope(c, 0, ramp)
    c.check(c.dense())
    ok()


def test_scores_of_any_size():
    for q_scale in (1e8, 1e18):
        c = Case4([300], [1], 64, seed=8, q_scale=q_scale)
        out, lse = c.dense()
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    ok()


@pytest.mark.parametrize("value,latched", [(65280.0, False), (65536.0, True), (float("inf"), True), (float("nan"), True)])
def test_rope_values_at_fp16s_end(value, latched):
    c = Case4([200, 90], [1, 1], 64, seed=9, sigma=1e-6)
    set_rope(c, 0, np.where(np.arange(200) == 77, value, 0.5))
    sel = c.select(200)
    for run in (c.dense, lambda: c.sparse(sel)):
        out, lse = run()
        assert smla.smla_get_last_error() == (7 if latched else 0)
        assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()


def test_selected_scales_that_nothing_writes_are_latched():
    c = Case4([131, 90], [1, 1], 64, seed=13)
    blk = int(c.table[0, 1])
    clean = c.sparse(c.select(131))
    records(c)[blk, 3, 256 + 7] = 0xF9
    sel = torch.stack([torch.arange(131, dtype=torch.int32), torch.cat([torch.arange(90, dtype=torch.int32), torch.full((41,), -1, dtype=torch.int32)])]).cuda()
    out, lse = c.sparse(sel)
    assert smla.smla_get_last_error() == 7
    assert torch.equal(out[1], clean[0][1]) and torch.equal(lse[1], clean[1][1])


# ---------------------------------- workspaces, streams, graphs ----------------------------------

def test_workspaces_that_are_small_or_unaligned():
    c = Case4([3000, 2000], [1, 1], 64, seed=10)
    sel = c.select(1024)
    prm = c.params(1024)
    n = smla.attend_workspace_size(c.lay, prm, c.n)
    for ws in (torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")[4:], torch.full((1000,), 0xFF, dtype=torch.uint8, device="cuda")):
        out, lse = c.buffers()
        smla.smla_attend(c.lay, prm, c.pool, 0, c.q, c.q_pe, sel, c.table, c.qsl, out, lse, workspace=ws)
        c.check((out, lse), sel, weight=P_BF16)
    small = torch.full((4096,), 0xFF, dtype=torch.uint8, device="cuda")
    c.check(c.dense(ws=small))
    ok()


def test_two_captured_steps_at_once_and_lengths_that_change():
    """Two graphs on two streams, each with its own workspace; the lengths change between replays."""
    a, b = Case4([2000, 900], [1, 1], 64, seed=11, extra_cols=2), Case4([1500], [1], 64, seed=12)
    sel = b.select(700)
    want_b = b.sparse(sel)
    prm = b.params(700)
    ws_a = torch.empty(smla.attend_dense_workspace_size(a.lay, a.params(), a.T), dtype=torch.uint8, device="cuda")
    ws_b = torch.empty(smla.attend_workspace_size(b.lay, prm, b.T), dtype=torch.uint8, device="cuda")
    out_a, out_b = a.buffers(), b.buffers()
    graphs = []
    for run in (lambda: a.dense(out=out_a, ws=ws_a), lambda: smla.smla_attend(b.lay, prm, b.pool, 0, b.q, b.q_pe, sel, b.table, b.qsl, *out_b, workspace=ws_b)):
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens in ([2000, 900], [1, 900], [1999, 130]):
        a.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        full, a.lens = a.lens, lens
        keys = [(l[:n], r[:n]) for (l, r), n in zip(a.keys, lens)]
        a.check(out_a, keys=keys)
        a.lens = full
        assert torch.equal(out_b[0], want_b[0]) and torch.equal(out_b[1], want_b[1])
    ok()


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 3000, 40)]
    c = Case4(lens, [1] * 40, 64, seed=14)
    sel = c.select(1000)
    want, want_sel = c.dense(), c.sparse(sel)
    c.check(want)
    for _ in range(30):
        got, got_sel = c.dense(), c.sparse(sel)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got_sel[0], want_sel[0]) and torch.equal(got_sel[1], want_sel[1])
    ok()


def test_another_stream_without_lse():
    c = Case4([600], [1], 64, seed=15)
    s = torch.cuda.Stream()
    out, _ = c.buffers()
    s.wait_stream(torch.cuda.current_stream())
    smla.smla_attend_dense(c.lay, c.params(), c.pool, 0, c.q, c.q_pe, c.table, c.seq_lens, c.qsl, out, stream=s)
    s.synchronize()
    want = c.dense(workspace=False)
    assert torch.equal(out, want[0])
    ok()


# ---------------------------------- large offsets ----------------------------------

def test_records_beyond_2_gib_of_one_page():
    """One page of 5,300,000 tokens (2.2 GB of records): its last positions, read back, attended to and selected."""
    bs = 5_300_000
    lay = smla.layout_init(bs, 1, 512, 64, 16, 32, 1, latent_format="e2m1")
    pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")        # scales of zero: values of zero
    n = 300
    slots = torch.arange(bs - n, bs, device="cuda")
    lat, rope = torch.randn(n, 512, device="cuda").bfloat16(), torch.randn(n, 64, device="cuda").bfloat16()
    smla.kvpack_store(lay, pool, 0, lat, rope, torch.zeros(n, 32, dtype=torch.uint8, device="cuda"), torch.zeros(n, device="cuda"), slots)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    loc = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    got, pe = torch.empty(n, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 64, dtype=torch.bfloat16, device="cuda")
    smla.kvpack_load(lay, pool, 0, table, loc, got, pe, starts=torch.tensor([bs - n], dtype=torch.int32, device="cuda"))
    assert torch.equal(pe, rope)
    rel = ((got.double() - lat.double()).norm() / lat.double().norm()).item()
    assert 0.05 < rel < 0.12                                                    # four bits
    q, q_pe = torch.randn(1, 64, 512, device="cuda").bfloat16(), torch.randn(1, 64, 64, device="cuda").bfloat16()
    qsl, lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([bs], dtype=torch.int32, device="cuda")
    s = (q[0].double() @ got.double().T + q_pe[0].double() @ pe.double().T) / 24
    for top_k in (None, 512):
        out, lse = torch.empty_like(q), torch.empty(1, 64, device="cuda")
        if top_k is None:
            prm = smla.make_params(64, 1, 1, 1 / 24)
            ws = torch.empty(smla.attend_dense_workspace_size(lay, prm, 1), dtype=torch.uint8, device="cuda")
            smla.smla_attend_dense(lay, prm, pool, 0, q, q_pe, table, lens, qsl, out, lse, workspace=ws)
            others = bs - n                                                     # positions of score 0
        else:
            prm = smla.make_params(64, 1, top_k, 1 / 24)
            sel = torch.cat([slots.int(), torch.full((top_k - n,), -1, dtype=torch.int32, device="cuda")])[None].contiguous()
            smla.smla_attend(lay, prm, pool, 0, q, q_pe, sel, table, qsl, out, lse)
            others = 0
        e = torch.exp(s)
        total = e.sum(-1) + others
        want = (e @ got.double()) / total[:, None]
        torch.testing.assert_close(lse[0].double(), torch.log(total), rtol=1e-5, atol=1e-5)
        weight = (e @ got.double().abs()) / total[:, None]
        assert ((out[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -7 * weight + 1e-7).all()
    ok()


def test_layers_and_key_formats_share_a_pool():
    """Two layers of one pool, FP4 indexer keys: what one layer writes the other does not see."""
    lay = smla.layout_init(16, 2, 512, 64, 16, 128, 4, "e2m1", latent_format="e2m1")
    pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")
    n = 40
    slots = torch.randperm(64, device="cuda")[:n].contiguous()
    ks = torch.rand(n, device="cuda")
    args = lambda: (torch.randn(n, 512, device="cuda").bfloat16(), torch.randn(n, 64, device="cuda").bfloat16(),  # noqa: E731
                    torch.randint(0, 256, (n, 64), dtype=torch.uint8, device="cuda"), ks, slots)
    first = args()
    smla.kvpack_store(lay, pool, 0, *first)
    before = pool.clone()
    smla.kvpack_store(lay, pool, 1, *args())
    a, b = pool.view(4, 2, -1), before.view(4, 2, -1)
    assert torch.equal(a[:, 0], b[:, 0]) and not torch.equal(a[:, 1], b[:, 1])
    ok()


@pytest.mark.parametrize("selected", [False, True])
def test_queries_that_are_not_numbers_stay_by_themselves(selected):
    """Units of 64 and of 16 rows in turn: rows of NaN and infinite queries change no other row to the bit."""
    c = Case4([700, 300, 900, 40, 513], [4, 1, 4, 1, 2], 16, seed=77)
    sel = c.select(256) if selected else None
    run = (lambda: c.sparse(sel)) if selected else c.dense
    clean = run()
    c.check(clean, sel)
    bad = [(0, 3), (1, 15), (5, 0), (6, 9), (10, 2)]
    for i, (t, h) in enumerate(bad):
        c.q[t, h, 7 * i] = float("nan") if i % 2 else float("inf")
    got = run()
    torch.cuda.synchronize()
    keep = torch.ones(c.T, 16, dtype=torch.bool, device="cuda")
    for t, h in bad:
        keep[t, h] = False
    assert all(torch.equal(x[keep], y[keep]) for x, y in zip(clean, got))
    ok()
