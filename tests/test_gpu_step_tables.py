"""smla_step_tables on the GPU against its definition in plain Python; every output is a whole number and has to be equal."""
import numpy as np
import pytest
import torch

import paged_sparse_mla_gb300 as smla
from tests import gpu_helpers as G

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.ensure_built()


def dev(x, t=I32):
    return torch.tensor(np.asarray(x), dtype=t, device="cuda")


class Step:
    def __init__(self, lens, new, bs=16, held=None, rows=None, n_rows=None, stride=None, bt_stride=None, n_free=None, used=0, pad=0, seed=0,
                 num_blocks=None, tokens=None, identity=False, shared=False):
        rng = np.random.default_rng(seed)
        b = len(new)
        self.bs, self.b, self.shared = bs, b, shared
        n_rows = (b if identity else b + 3) if n_rows is None else n_rows
        self.rows = None if identity else (rng.permutation(n_rows)[:b] if rows is None else np.asarray(rows))
        r = np.arange(b) if identity else self.rows
        fit = (r >= 0) & (r < n_rows)
        self.lens = rng.integers(0, 50, n_rows)
        self.lens[r[fit]] = np.asarray(lens)[fit]
        self.held = -(-self.lens // bs)
        if held is not None:
            self.held[r[fit]] = np.asarray(held)[fit]
        self.new = np.asarray(new)
        most = max([1] + [-(-max(int(n) + max(int(q), 0), 0) // bs) for n, q in zip(lens, new)])
        self.stride = int(max(most, self.held.max())) + 1 if stride is None else stride
        self.bt_stride = self.stride if bt_stride is None else bt_stride
        free = n_rows * self.stride + 7 if n_free is None else n_free
        ids = rng.permutation(n_rows * self.stride + free)
        self.table = ids[:n_rows * self.stride].reshape(n_rows, self.stride)
        self.free = ids[n_rows * self.stride:]
        self.used, self.n_rows = used, n_rows
        self.tokens = int(sum(max(0, q) for q in new)) + pad if tokens is None else tokens
        self.num_blocks = len(ids) if num_blocks is None else num_blocks
        self.lay = smla.layout_init(bs, 1, 512, 64, 128, 128, self.num_blocks)

    def want(self):
        """(outputs by name, status)"""
        cap = min(self.stride, self.stride if self.shared else self.bt_stride) * self.bs
        table, held = self.table.copy(), self.held.copy()
        bt = np.full((self.b, self.bt_stride), -7)
        seq, qsl, pos, slots = [], [0], [], []
        used, bad, out = min(max(self.used, 0), len(self.free)), False, False
        bad |= used != self.used
        for i in range(self.b):
            row = i if self.rows is None else self.rows[i]
            if row < 0 or row >= self.n_rows:
                bad |= row >= self.n_rows
                seq.append(0)
                qsl.append(qsl[-1])
                continue
            n = min(max(self.lens[row], 0), cap)
            q = min(max(self.new[i], 0), cap - n)
            bad |= n != self.lens[row] or q != self.new[i]
            take = min(q, self.tokens - qsl[-1])
            bad |= take != q
            blocks = -(-(n + take) // self.bs)
            have = min(max(self.held[row], -(-n // self.bs)), self.stride)
            ids = list(table[row, :have])
            while len(ids) < blocks:
                if used < len(self.free):
                    ids.append(self.free[used])
                    used += 1
                    have += 1
                else:
                    ids.append(-1)
                    out = True
            held[row] = have
            table[row, :len(ids)] = ids
            bt[i, :blocks] = ids[:blocks]
            seq.append(n + take)
            for k in range(take):
                p = n + k
                pos.append(p)
                blk = ids[p // self.bs]
                good = 0 <= blk < self.num_blocks
                bad |= blk >= self.num_blocks
                slots.append(blk * self.bs + p % self.bs if good else -1)
            qsl.append(qsl[-1] + take)
        behind = self.tokens - len(pos)
        return (dict(seq_lens=seq, query_start_loc=qsl, positions=pos + [0] * behind, slots=slots + [-1] * behind, table=table, held=held, used=[used],
                     block_table=bt), 8 if out else 4 if bad else 0)

    def run(self, in_place=False, offset=0, stream=None):
        d = dict(table=dev(self.table), held=dev(self.held), used=dev([self.used], I64), seq_lens=dev([-7] * self.b), query_start_loc=dev([-7] * (self.b + 1)),
                 positions=dev([-7] * self.tokens, I64), slots=dev([-7] * self.tokens, I64), block_table=dev(np.full((self.b, self.bt_stride), -7)))
        if offset:   # tables that are not 16-byte aligned
            for k in ("table", "block_table"):
                buf = torch.empty(d[k].numel() + 4, dtype=I32, device="cuda")[offset:offset + d[k].numel()].view(d[k].shape)
                buf.copy_(d[k])
                d[k] = buf
        held_out, used_out = (d["held"], d["used"]) if in_place else (d["held"].clone(), dev([-7], I64))
        ws = torch.full((smla.step_tables_workspace_size(self.b),), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        self.call = lambda: smla.smla_step_tables(
            self.lay, dev_lens, dev_new, d["table"], d["held"], held_out, dev_free, d["used"], used_out, d["seq_lens"], d["query_start_loc"], d["positions"],
            d["slots"], rows=dev_rows, block_table=None if self.shared else d["block_table"], workspace=ws, stream=stream)
        dev_lens, dev_new, dev_free = dev(self.lens), dev(self.new), dev(self.free)
        dev_rows = None if self.rows is None else dev(self.rows)
        torch.cuda.synchronize()
        self.call()
        self.state = d
        return {**d, "held": held_out, "used": used_out}

    def check(self, **kw):
        got = self.run(**kw)
        want, status = self.want()
        assert smla.smla_get_last_error() == status
        for k, w in want.items():
            if k == "block_table" and self.shared:
                continue
            assert np.array_equal(got[k].cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), k
        return got


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,new,bs,pad", [
    ([0], [1], 16, 0), ([1], [1], 64, 0), ([15, 16, 17], [1, 1, 1], 16, 5), ([0, 0, 0], [0, 0, 0], 16, 0), ([0, 0], [0, 0], 7, 4),
    ([100, 5, 0, 64], [4, 700, 1, 0], 64, 3), ([33, 2], [64, 1], 1, 0), ([4000, 10], [1, 4], 3, 1),
])
def test_tables_of_small_steps(lens, new, bs, pad, in_place):
    Step(lens, new, bs, pad=pad, used=2).check(in_place=in_place)
    Step(lens, new, bs, pad=pad, identity=True).check(in_place=in_place)
    Step(lens, new, bs, pad=pad, identity=True, shared=True).check(in_place=in_place)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("batch,bs", [(1, 16), (33, 64), (257, 16), (1024, 64), (1025, 32), (4097, 16), (5000, 128)])
def test_tables_of_batches(batch, bs, offset):
    rng = np.random.default_rng(batch)
    lens = np.exp(rng.uniform(0, np.log(3000), batch)).astype(int)
    new = np.where(rng.random(batch) < 0.05, rng.integers(0, 300, batch), rng.integers(0, 5, batch))
    more = -(-(lens + rng.integers(0, 3 * bs, batch)) // bs)     # blocks that rejected tokens left
    Step(lens, new, bs, held=more, pad=int(rng.integers(0, 500)), seed=batch).check(offset=offset)


@pytest.mark.parametrize("offset", [0, 1])
def test_tables_large_enough_for_two_launches(offset):
    rng = np.random.default_rng(9)
    lens = rng.integers(10000, 20000, 600)
    new = np.where(rng.random(600) < 0.05, rng.integers(0, 300, 600), 1)
    Step(lens, new, 16, pad=33, seed=1).check(offset=offset)
    Step(lens[:530], new[:530], 16, pad=33, seed=2, n_free=100).check(offset=offset, in_place=True)


def test_a_long_row_and_many_new_blocks():
    Step([262143 * 4, 3], [5, 70000], 16).check()
    Step([0, 9], [300000, 1], 16, pad=7).check()


def test_entries_without_a_request():
    Step([40, 9, 70, 5], [3, 2, 100, 1], rows=[2, -1, 0, -5], n_rows=5).check()
    Step([40, 9, 70], [3, 2, 100], rows=[2, 5, 0], n_rows=5).check()           # row 5 of 5 is latched


def test_an_empty_free_list_is_latched_and_bounded():
    for n_free, used in ((0, 0), (3, 0), (5, 4), (2, 9), (4, -1)):
        Step([30, 16, 100], [5, 40, 70], n_free=n_free, used=used).check()


def test_tokens_that_do_not_fit_are_not_taken():
    Step([30, 16, 100], [5, 40, 70], tokens=20).check()
    Step([30, 16, 100], [5, 40, 70], tokens=0).check()
    Step([30, 60, 100], [5, 40, 70], stride=8, held=[2, 4, 7]).check()          # rows of 128 positions
    Step([30, 60, 100], [5, 40, 70], bt_stride=6, held=[2, 4, 7]).check()       # the batch's table is narrower: 96
    Step([-3, 60], [5, -40]).check()


def test_block_ids_outside_the_pool_give_no_slot():
    Step([30, 16, 100], [5, 40, 70], num_blocks=20, seed=3).check()


def test_repeated_and_captured_calls():
    """In place each replay takes further blocks; otherwise a repeated call gives the same tables."""
    s = Step([30, 16, 100], [5, 40, 70])
    a = {k: v.clone() for k, v in s.check().items()}
    s.call()
    torch.cuda.synchronize()
    for k, v in a.items():
        assert k in ("held", "used") or torch.equal(s.state[k], v), k
    s = Step([30, 16, 100], [5, 40, 70], seed=4)
    st = torch.cuda.Stream()
    got = s.run(in_place=True, stream=st)       # warm-up outside the capture: takes the step's blocks
    torch.cuda.synchronize()
    used, held = int(got["used"]), got["held"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        s.call()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert int(got["used"]) == used and torch.equal(got["held"], held)   # the rows hold the step's blocks already
    want, _ = s.want()
    for k in ("table", "slots", "block_table", "positions"):
        assert np.array_equal(got[k].cpu().numpy().reshape(-1), np.asarray(want[k]).reshape(-1)), k
    assert smla.smla_get_last_error() == 0


def test_steps_of_a_decode_loop_feed_the_other_calls():
    """Three sequences over forty steps of drafted tokens, some rejected: tables, appends and dense attention on the GPU, the
    lengths never leaving it, against the same tokens appended to a cache whose pages were dealt by the host."""
    torch.manual_seed(0)
    bs, b, k, steps = 16, 3, 4, 12
    for fmt, tile in (("e2m1", 16), ("e4m3", 128)):
        n_blocks, width = 64, 12
        lay = smla.layout_init(bs, 1, 512, 64, tile, 128, n_blocks, latent_format=fmt)
        prm = smla.make_params(16, 1, 1, 1 / 24)
        pool = torch.zeros(lay.pool_bytes, dtype=torch.uint8, device="cuda")
        lens, held, used = dev([0] * b), dev([0] * b), dev([0], I64)
        table = dev(np.full((b, width), -1))
        free = torch.randperm(n_blocks, device="cuda").int()
        new, ws = dev([k] * b), torch.empty(smla.step_tables_workspace_size(b), dtype=torch.uint8, device="cuda")
        seq, qsl = dev([0] * b), dev([0] * (b + 1))
        pos, slots = dev([0] * b * k, I64), dev([0] * b * k, I64)
        ws2 = torch.empty(smla.attend_dense_workspace_size(lay, prm, b * k), dtype=torch.uint8, device="cuda")
        kept = [[], [], []]
        for step in range(steps):
            smla.smla_step_tables(lay, lens, new, table, held, held, free, used, used, seq, qsl, pos, slots, workspace=ws)
            lat, rope = torch.randn(b * k, 512, device="cuda").bfloat16(), torch.randn(b * k, 64, device="cuda").bfloat16()
            smla.kvpack_append(lay, pool, 0, lat, rope, None, None, None, slots)
            q, q_pe = torch.randn(b * k, 16, 512, device="cuda").bfloat16(), torch.randn(b * k, 16, 64, device="cuda").bfloat16()
            out, lse = torch.empty_like(q), torch.empty(b * k, 16, device="cuda")
            smla.smla_attend_dense(lay, prm, pool, 0, q, q_pe, table, seq, qsl, out, lse, workspace=ws2)
            accepted = torch.randint(1, k + 1, (b,), device="cuda", dtype=I32)
            # the last drafted token of each sequence sees everything appended so far: softmax over the loaded rows
            loc = torch.cat([dev([0]), seq.cumsum(0).int()])
            rows = int(loc[-1])
            l2, r2 = torch.empty(rows, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, 64, dtype=torch.bfloat16, device="cuda")
            smla.kvpack_load(lay, pool, 0, table, loc, l2, r2)
            for i in range(b):
                kept[i] = kept[i][:int(lens[i])] + [rope[i * k + j].clone() for j in range(k)]
                assert torch.equal(r2[int(loc[i]):int(loc[i + 1])], torch.stack(kept[i]))
                lat64, rope64 = l2[int(loc[i]):int(loc[i + 1])].double(), r2[int(loc[i]):int(loc[i + 1])].double()
                s = (q[i * k + k - 1].double() @ lat64.T + q_pe[i * k + k - 1].double() @ rope64.T) / 24
                want = torch.softmax(s, -1) @ lat64
                # E4M3: the loaded rows are rounded to bf16 (2^-8 of each key, in scores and values), the result too
                assert (out[i * k + k - 1].double() - want).abs().max() <= (0.02 if fmt == "e2m1" else 0.06)
            lens = lens + accepted
        assert smla.smla_get_last_error() == 0
        t = table.cpu().numpy()
        mine = [x for i in range(b) for x in t[i, :int(held[i])]]
        assert len(set(mine)) == len(mine) == int(used) and min(mine) >= 0
