"""A random cache of E2M1 (or E4M3) latents behind a shuffled block table, and attention over it in float64.

Bounds, per output element.  E2M1 latents are exact in fp16 and bf16, queries too (scaled by a power of two), so that a
score is off by its fp32 sum alone: 36 partial sums, each within 2^-22 of what it adds up, dS <= 2^-16 sigma sum_d |q_d K_jd|
(the tensor cores' alignment may cut a bit more than an fp32 rounding would), and the exponential's argument in fp32, 2^-21 of
the score's size.  The weights are rounded to fp16 (2^-11; dense) or bf16 (2^-8; selected), the result to bf16 (2^-8):
    |out - ref| <= 2^-8 |ref| + sum_j p_j |K_j| (w + 2 dS_max) + 1e-5 max_j |K_j|
with the last term for the fp32 sums and the weights near fp16's end, and |lse - ref| <= dS_max + 1e-6 (1 + |lse|) (its
fp32 sum and logarithm).
"""
import numpy as np
import torch

import paged_sparse_mla_gb300 as smla
import oracle

P_FP16, P_BF16 = 2.0 ** -11, 2.0 ** -8


def bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().view(torch.int16).numpy().view(np.uint16)


class Case4:
    def __init__(self, lens, counts, heads, bs=64, dl=512, dr=64, layers=1, layer=0, seed=0, key_scale=1.0, q_scale=1.0, sigma=None,
                 extra_cols=0, pad_rows=0, fmt="e2m1"):
        rng = np.random.default_rng(seed)
        self.lens, self.counts, self.heads, self.bs, self.layer = list(lens), list(counts), heads, bs, layer
        need = [-(-n // bs) for n in lens]
        blocks = sum(need) + 2
        tile = 16 if fmt == "e2m1" else 128
        self.lay = smla.layout_init(bs, layers, dl, dr, tile, 32, blocks, latent_format=fmt)
        self.ref = oracle.PoolLayout(bs, layers, dl, dr, tile, 32, blocks, "e4m3", fmt)
        pool = np.full(self.lay.pool_bytes, 0xFF, dtype=np.uint8)   # NaN scales and ropes everywhere else
        perm = rng.permutation(blocks)
        table = np.full((len(lens), max(1, max(need) + extra_cols)), -1, dtype=np.int32)
        at = 0
        self.keys = []
        for b, n in enumerate(lens):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            j = np.arange(n)
            slots = table[b, j // bs].astype(np.int64) * bs + j % bs if n else np.zeros(0, np.int64)
            if n:
                lat = rng.standard_normal((n, dl)) * key_scale * (0.3 + rng.random((n, 1)))
                oracle.kvpack_store(self.ref, pool, layer, bf16_bits(lat), bf16_bits(rng.standard_normal((n, dr))), np.zeros((n, 32), np.uint8),
                                    np.ones(n, np.float32), slots)
            self.keys.append(oracle.read_record(self.ref, pool, layer, slots) if n else (np.zeros((0, dl)), np.zeros((0, dr))))
        self.pool = torch.from_numpy(pool).cuda()
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.qsl = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        self.n = int(sum(counts))
        self.T = self.n + pad_rows
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.q = (torch.randn(self.T, heads, dl, generator=g, device="cuda") * q_scale).bfloat16()
        self.q_pe = (torch.randn(self.T, heads, dr, generator=g, device="cuda") * q_scale).bfloat16()
        self.sigma = 1.0 / np.sqrt(dl + dr) if sigma is None else sigma
        self.rng = rng

    def params(self, top_k=1):
        return smla.make_params(self.heads, 1, top_k, self.sigma)

    def buffers(self):
        return (torch.full((self.T, self.heads, self.lay.d_latent), 777.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((self.T, self.heads), 777.0, device="cuda"))

    def dense(self, workspace=True, stream=None, out=None, ws=None):
        out, lse = self.buffers() if out is None else out
        prm = self.params()
        n = smla.attend_dense_workspace_size(self.lay, prm, self.T)
        if ws is None and workspace and n:
            ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.current_stream().synchronize() if stream is not None else None
        smla.smla_attend_dense(self.lay, prm, self.pool, self.layer, self.q, self.q_pe, self.table, self.seq_lens, self.qsl, out, lse,
                               workspace=ws, stream=stream)
        return out, lse

    def sees(self, t):
        """(sequence, visible positions) of query token t."""
        b = int(np.searchsorted(np.cumsum(self.counts), t, side="right"))
        i = t - int(sum(self.counts[:b]))
        return b, max(0, self.lens[b] - self.counts[b] + i + 1)

    def select(self, top_k, keep=1.0):
        """Random ascending visible positions per token, -1 behind them (`keep`: the share of top_k that is used at most)."""
        sel = np.full((self.T, top_k), -1, dtype=np.int32)
        for t in range(self.n):
            _, v = self.sees(t)
            k = min(v, int(round(top_k * keep)))
            sel[t, :k] = np.sort(self.rng.permutation(v)[:k])
        return torch.from_numpy(sel).cuda()

    def sparse(self, sel, workspace=True):
        out, lse = self.buffers()
        prm = self.params(sel.shape[1])
        n = smla.attend_workspace_size(self.lay, prm, self.n)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if workspace and n else None
        smla.smla_attend(self.lay, prm, self.pool, self.layer, self.q[:self.n], self.q_pe[:self.n], sel[:self.n].contiguous(), self.table, self.qsl, out, lse,
                         workspace=ws)
        return out, lse

    def want(self, sel=None, keys=None, weight=P_FP16):
        """(out, lse, out's bound, lse's bound) in float64."""
        got = [[], [], [], []]
        cache = [[torch.from_numpy(x).cuda() for x in k] for k in (keys or self.keys)]
        for t in range(self.n):
            b, v = self.sees(t)
            lat, rope = cache[b]
            if sel is None:
                lat, rope = lat[:v], rope[:v]
            else:
                pick = sel[t][sel[t] >= 0].long()
                lat, rope = lat[pick], rope[pick]
            if lat.shape[0] == 0:
                o = torch.zeros(self.heads, lat.shape[1], dtype=torch.float64, device="cuda")
                s = torch.full((self.heads,), -np.inf, dtype=torch.float64, device="cuda")
                parts = (o, s, torch.zeros_like(o), torch.zeros_like(s))
            else:
                q, qp = self.q[t].double(), self.q_pe[t].double()
                s = self.sigma * (q @ lat.T + qp @ rope.T)
                p = torch.softmax(s, -1)
                ds = abs(self.sigma) * 2.0 ** -16 * (q.abs() @ lat.abs().T + qp.abs() @ rope.abs().T).amax(-1) + 2.0 ** -21 * s.abs().amax(-1)
                o, lse = p @ lat, torch.logsumexp(s, -1)
                parts = (o, lse, 2.0 ** -8 * o.abs() + (p @ lat.abs()) * (weight + 2 * ds[:, None]) + 1e-5 * lat.abs().max(),
                         ds + 1e-6 * (1 + lse.abs()))
            for to, x in zip(got, parts):
                to.append(x)
        return [torch.stack(x) for x in got]

    def check(self, got, sel=None, keys=None, weight=P_FP16):
        out, lse = got
        torch.cuda.synchronize()
        n = self.n
        assert (out[n:] == 777).all() and (lse[n:] == 777).all()   # rows behind the last sequence
        if n == 0:
            return
        wo, wl, bo, bl = self.want(sel, keys, weight)
        e = (out[:n].double() - wo).abs()
        assert (e <= bo).all(), f"out off by {(e - bo).max():.3e} more than its bound"
        fin = torch.isfinite(wl)
        assert (lse[:n][~fin] == -np.inf).all()
        e = (lse[:n].double() - wl).abs()[fin]
        assert (e <= bl[fin]).all(), f"lse off by {(e - bl[fin]).max():.3e} more than its bound"
