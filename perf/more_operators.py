"""A cache with latents in 4 bits, and the tables of a step: cases, inputs, plain forms and values in 64 bits.

Five operators around the paged cache of latent attention:

* ``tables``  block tables, positions and slots of a step from the requests' lengths, new blocks from a free list;
* ``append``  norm, rotation, quantisation to 4 bits and scatter of new tokens, which are then read back;
* ``load``    a range of each sequence's cached positions as bf16 rows, for up-projection;
* ``attend``  latent attention over the whole visible context;
* ``select``  latent attention over each token's selected positions.

A record holds 512 E2M1 codes (two to a byte, the even one in the low bits), a scale for every 16 of them (5 bits of exponent,
3 of mantissa: the first byte of an fp16 value without its sign) and 64 bf16 rope values.  ``run`` computes the operators
in plain torch operations in fp32, or, where ``own`` is true, through the library.
"""
import math
import random

import torch

own = False

D_LATENT, D_ROPE, GROUP, D_INDEX = 512, 64, 16, 128   # the full shape of this repository's workloads
CODES, SCALES = D_LATENT // 2, D_LATENT // GROUP
REC = CODES + SCALES + 2 * D_ROPE                     # bytes of one cached record
E2M1_MAX, SCALE_MAX, E4M3_MAX = 6.0, 10240.0, 448.0
EPS = 1e-6


def listed():
    return [
        # one request's next token: latency
        {"name": "tables-1", "op": "tables", "batch": 1, "ctx_lo": 1000, "ctx_hi": 1000, "new_lo": 1, "new_hi": 1, "block": 64, "pad": 0},
        # the repository's agentic step: 64 sequences, three drafted tokens each, some of the last step's drafts rejected
        {"name": "tables-mtp4-b64", "op": "tables", "batch": 64, "ctx_lo": 16384, "ctx_hi": 262144, "new_lo": 4, "new_hi": 4, "block": 64, "pad": 0},
        # many requests on small pages, prefill chunks beside decode tokens, arrays padded for a captured graph
        {"name": "tables-mixed-b1024", "op": "tables", "batch": 1024, "ctx_lo": 100, "ctx_hi": 32768, "new_lo": 1, "new_hi": 512, "block": 16, "pad": 333},
        # a decode step of 64 sequences with three drafted tokens each, the arrays padded
        {"name": "append-256", "op": "append", "batch": 64, "queries": 4, "ragged": False, "ctx_lo": 4, "ctx_hi": 4096, "block": 64, "interleaved": True, "idx_bias": True, "pad": 9},
        # prefill chunks of a few requests
        {"name": "append-8192", "op": "append", "batch": 5, "queries": 2777, "ragged": True, "ctx_lo": 2777, "ctx_hi": 9000, "block": 64, "interleaved": False, "idx_bias": False, "pad": 0},
        # a short cached prefix of each of a few requests
        {"name": "load-ragged", "op": "load", "batch": 7, "ctx_lo": 33, "ctx_hi": 700, "start": 17, "block": 16},
        # the whole prefix of the repository's prefill workload
        {"name": "load-131072", "op": "load", "batch": 1, "ctx_lo": 131072, "ctx_hi": 131072, "start": 0, "block": 64},
        # the repository's decode batch: 32 sequences, one token each
        {"name": "attend-decode-b32", "op": "attend", "batch": 32, "queries": 1, "ragged": False, "ctx_lo": 8192, "ctx_hi": 32768, "heads": 64, "block": 64},
        # a prefill chunk on a cached prefix
        {"name": "attend-chunk-2048", "op": "attend", "batch": 1, "queries": 2048, "ragged": False, "ctx_lo": 18432, "ctx_hi": 18432, "heads": 64, "block": 64},
        # a mixed batch: chunks of uneven length beside decode tokens, few heads (a model split by heads), small pages
        {"name": "attend-ragged-h16", "op": "attend", "batch": 9, "queries": 177, "ragged": True, "ctx_lo": 333, "ctx_hi": 5003, "heads": 16, "block": 16},
        # one decode token on a long context
        {"name": "select-1", "op": "select", "batch": 1, "queries": 1, "ctx_lo": 65536, "ctx_hi": 65536, "heads": 64, "top_k": 2048, "block": 64},
        # the agentic step: 256 tokens, 2,048 positions each
        {"name": "select-mtp4-b64", "op": "select", "batch": 64, "queries": 4, "ctx_lo": 1500, "ctx_hi": 65536, "heads": 64, "top_k": 2048, "block": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "load", "attend", "select"])
    block = rng.choice([16, 32, 64, 128])
    if op == "tables":
        batch, hi = _log(rng, 1, 1024), _log(rng, 1, 32768)
        return {"op": op, "batch": batch, "ctx_lo": hi // rng.choice([1, 3, 50]), "ctx_hi": hi, "new_lo": rng.choice([0, 1, 1, 4]),
                "new_hi": _log(rng, 1, 512), "block": block, "pad": rng.choice([0, 1, 100])}
    if op == "append":
        batch, q = _log(rng, 1, 64), _log(rng, 1, 512)
        while batch * q > 8192:
            q = (q + 1) // 2
        hi = _log(rng, q, 8192)
        return {"op": op, "batch": batch, "queries": q, "ragged": rng.random() < 0.5, "ctx_lo": max(q, hi // rng.choice([1, 5])), "ctx_hi": hi, "block": block,
                "interleaved": rng.random() < 0.5, "idx_bias": rng.random() < 0.5, "pad": rng.randint(0, 20)}
    if op == "load":
        batch, hi = _log(rng, 1, 32), _log(rng, 1, 131072)
        while batch * hi > 131072:
            hi = (hi + 1) // 2
        return {"op": op, "batch": batch, "ctx_lo": max(1, hi // rng.choice([1, 2, 9])), "ctx_hi": hi, "start": rng.choice([0, 0, 1, 100]), "block": block}
    if op == "select":
        batch, q, hi = _log(rng, 1, 64), rng.choice([1, 2, 4]), _log(rng, 1, 65536)
        hi = max(hi, q)
        return {"op": op, "batch": batch, "queries": q, "ctx_lo": max(q, hi // rng.choice([1, 2, 7])), "ctx_hi": hi, "heads": rng.choice([5, 8, 16, 32, 64]),
                "top_k": rng.choice([64, 500, 2048]), "block": block}
    batch, queries, hi = _log(rng, 1, 64), _log(rng, 1, 1024), _log(rng, 1, 32768)
    heads = rng.choice([5, 8, 16, 32, 64, 64, 128])
    while queries > 1 and batch * queries * heads * max(hi, queries) > 2048 * 64 * 9216:
        queries = (queries + 1) // 2
    hi = max(hi, queries)
    return {"op": op, "batch": batch, "queries": queries, "ragged": rng.random() < 0.5, "ctx_lo": max(queries, hi // rng.choice([1, 2, 7])),
            "ctx_hi": hi, "heads": heads, "block": block}


def _spread(case):
    """The sequences' lengths: spread evenly, in an order fixed by the case."""
    b, lo, hi = case["batch"], case["ctx_lo"], case["ctx_hi"]
    lens = [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]
    random.Random(b * 1000003 + hi * 31 + lo).shuffle(lens)
    return lens


def _geometry(case):
    """Of each sequence: positions at the step's end and query tokens (for ``load``: rows) among them, the last ones."""
    lens = _spread(case)
    r = random.Random(case["batch"] * 7919 + case["ctx_hi"])
    if case["op"] == "load":
        return lens, [n - min(case["start"], n - 1) for n in lens]
    q = case["queries"]
    return lens, [q if not case.get("ragged") or i == 0 else r.randint(1, q) for i in range(len(lens))]


def _new_tokens(case):
    """Of each entry of a step: cached tokens, new ones, and how many tokens beyond the cached ones its blocks held already."""
    r = random.Random(case["batch"] * 31 + case["ctx_hi"] + case["new_hi"])
    lens = _spread(case)
    new = [r.randint(case["new_lo"], max(case["new_lo"], case["new_hi"])) if i % 8 == 0 else case["new_lo"] for i in range(len(lens))]
    new[0] += not any(new)
    return lens, new, [r.randint(0, 3) for _ in lens]


def _strides(block):
    """(bytes of one block of one layer, offset of its keys, offset of its key scales): every region starts on 256 bytes."""
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    keys = up(block * REC)
    scales = up(keys + block * D_INDEX)
    return up(scales + 4 * block), keys, scales


def _cache(s, case, lens, g, fill):
    """The pool and the block table of sequences of these lengths; `fill`: cached records are written (their unused rest holds NaN)."""
    bs = case["block"]
    need = [-(-n // bs) for n in lens]
    blocks, stride = sum(need), _strides(bs)[0]
    perm = torch.randperm(blocks, generator=g, device="cuda").int()
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    pool = torch.zeros(blocks, stride, dtype=torch.uint8, device="cuda")
    rec = torch.as_strided(pool, (blocks, bs, REC), (stride, REC, 1))
    step = max(1, (1 << 18) // bs)
    for k in range(0, blocks if fill else 0, step):
        n = min(step, blocks - k)
        rec[k:k + n, :, :CODES] = torch.randint(0, 256, (n, bs, CODES), generator=g, device="cuda", dtype=torch.uint8)
        scales = (0.1 + 0.5 * torch.rand(n, bs, SCALES, generator=g, device="cuda")).half()
        rec[k:k + n, :, CODES:CODES + SCALES] = (scales.view(torch.int16) >> 7).to(torch.uint8)
        rec[k:k + n, :, CODES + SCALES:] = torch.randn(n, bs, D_ROPE, generator=g, device="cuda").bfloat16().view(torch.uint8)
    at = 0
    for i, n in enumerate(lens):
        table[i, :need[i]] = perm[at:at + need[i]]
        if fill and n % bs:
            rec[table[i, need[i] - 1].long(), n % bs:] = 255
        at += need[i]
    s.update(pool=pool.view(-1), block_table=table, blocks=blocks)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *z: torch.randn(z, generator=g, device="cuda")  # noqa: E731
    ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    op, bs = case["op"], case["block"]
    s = {"op": op, "case": case}
    if op == "tables":
        lens, new, more = _new_tokens(case)
        b = len(lens)
        n_rows, most = b + b // 4 + 1, max(-(-(n + max(q, m)) // bs) for n, q, m in zip(lens, new, more))
        stride = -(-most // 4) * 4
        rows = torch.randperm(n_rows, generator=g, device="cuda")[:b]
        by_row = lambda v: torch.zeros(n_rows, dtype=torch.int32, device="cuda").index_copy_(0, rows, ints(v))  # noqa: E731
        held = by_row([-(-(n + m) // bs) for n, m in zip(lens, more)])
        ids = torch.randperm(n_rows * stride * 2, generator=g, device="cuda").int()
        n_free = n_rows * stride
        total = sum(new) + case["pad"]
        s.update(rows=rows.int(), lens=by_row(lens), new=ints(new), held=held, held_out=held.clone(), table=ids[:n_free].view(n_rows, stride).clone(),
                 free=ids[n_free:].contiguous(), used=ints([5], torch.int64), used_out=ints([0], torch.int64), tokens=total, blocks=2 * n_free,
                 seq_lens=ints([0] * b), qsl=ints([0] * (b + 1)), positions=torch.zeros(total, dtype=torch.int64, device="cuda"),
                 slots=torch.zeros(total, dtype=torch.int64, device="cuda"), block_table=torch.zeros(b, stride, dtype=torch.int32, device="cuda"))
    else:
        lens, counts = _geometry(case)
        _cache(s, case, lens, g, op != "append")
        t = sum(counts)
        s.update(seq_lens=ints(lens), row_loc=ints([0] + counts).cumsum(0).int(), starts=ints([n - c for n, c in zip(lens, counts)]), rows=t,
                 max_ctx=max(lens), max_q=max(counts))
    if op in ("append", "load"):
        n = t + case.get("pad", 0)
        s.update(latent_out=torch.empty(t, D_LATENT, dtype=torch.bfloat16, device="cuda"), rope_out=torch.empty(t, D_ROPE, dtype=torch.bfloat16, device="cuda"))
    if op == "append":
        f = 10000.0 ** (-torch.arange(0, D_ROPE, 2, device="cuda", dtype=torch.float64) / D_ROPE)
        angle = torch.arange(s["max_ctx"], device="cuda", dtype=torch.float64)[:, None] * f
        seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), ints(counts))
        pos = s["starts"][seq].long() + torch.arange(t, device="cuda") - s["row_loc"][seq].long()
        slots = s["block_table"][seq, pos // bs].long() * bs + pos % bs
        fill = lambda v, x: torch.cat([v, torch.full((case["pad"],), x, dtype=torch.int64, device="cuda")])  # noqa: E731
        s.update(table=torch.cat([angle.cos(), angle.sin()], dim=1).float(), positions=fill(pos, 0), slots=fill(slots, -1),
                 kv=(rnd(n, D_LATENT + D_ROPE) * (0.5 + rnd(n, 1).abs())).bfloat16(),  # the projection's output: latent and rope key side by side
                 idx_k=(rnd(n, D_INDEX) * 2 + 0.3).bfloat16(), norm=1 + 0.1 * rnd(D_LATENT), idx_norm=1 + 0.1 * rnd(D_INDEX),
                 idx_bias=0.1 * rnd(D_INDEX) if case["idx_bias"] else None)
    if op in ("attend", "select"):
        h = case["heads"]
        s.update(q=rnd(t, h, D_LATENT).bfloat16(), q_pe=rnd(t, h, D_ROPE).bfloat16(), scale=1.0 / math.sqrt(D_LATENT + D_ROPE),
                 out=torch.empty(t, h, D_LATENT, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(t, h, device="cuda"))
    if op == "select":  # ascending positions of what each token sees, -1 behind them
        k = case["top_k"]
        seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), ints(counts))
        sees = (s["starts"][seq] + torch.arange(t, device="cuda") - s["row_loc"][seq] + 1)[:, None]
        picks = []
        for i in range(0, t, 32):
            key = torch.rand(min(32, t - i), max(k, s["max_ctx"]), generator=g, device="cuda")
            key[torch.arange(key.shape[1], device="cuda")[None] >= sees[i:i + 32]] = -1
            top, at = key.topk(k, dim=1)
            at = torch.where(top < 0, torch.full_like(at, 1 << 40), at).sort(dim=1).values
            picks.append(torch.where(at == 1 << 40, torch.full_like(at, -1), at).int())
        s["topk"] = torch.cat(picks)
    if own:  # the handles that a program keeps: layout, parameters, rotation table, workspace
        import paged_sparse_mla_gb300 as smla
        s["smla"] = smla
        s["layout"] = smla.layout_init(bs, 1, D_LATENT, D_ROPE, GROUP, D_INDEX, s["blocks"], latent_format="e2m1")
        need = 0
        if op == "tables":
            need = smla.step_tables_workspace_size(case["batch"])
        elif op == "append":
            s["rope"] = smla.make_rope(s["table"], interleaved=case["interleaved"], idx_interleaved=False, idx_rope=True)
        elif op in ("attend", "select"):
            s["params"] = smla.make_params(case["heads"], 64, case.get("top_k", 2048), s["scale"])
            size = smla.attend_dense_workspace_size if op == "attend" else smla.attend_workspace_size
            need = size(s["layout"], s["params"], t)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return s


def _key_views(s):
    """The cached indexer keys' codes and scales."""
    bs, blocks = s["case"]["block"], s["blocks"]
    stride, keys, scales = _strides(bs)
    return {"key_codes": s["pool"].view(torch.float8_e4m3fn).as_strided((blocks, bs, D_INDEX), (stride, D_INDEX, 1), keys),
            "key_scales": s["pool"].view(torch.float32).as_strided((blocks, bs), (stride // 4, 1), scales // 4)}


def _rotate(x, cs, interleaved):
    """x [..., d] rotated by the angles whose cosines and sines are cs [..., d]."""
    half = D_ROPE // 2
    c, d = cs[..., :half], cs[..., half:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * d, a * d + b * c], dim=-1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * d, a * d + b * c], dim=-1)


def _to_4_bits(y):
    """The values that y's groups of 16 keep: E2M1 codes times the group's scale, both rounded to even."""
    y = y.unflatten(-1, (SCALES, GROUP))
    s = y.abs().amax(-1, keepdim=True) / E2M1_MAX
    step = torch.exp2(torch.frexp(s).exponent.clamp(min=-13).float() - 4)  # of a scale with three bits behind its first, from 2^-14 on
    s = ((s / step).round() * step).clamp(max=SCALE_MAX)
    v = torch.where(s > 0, y.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    v = ((v / step).round() * step).clamp(max=E2M1_MAX)
    return (torch.copysign(v, y) * s).flatten(-2)


def _from_4_bits(rec, dtype):
    """(latent, rope) of records [..., REC]."""
    byte = rec[..., :CODES]
    code = torch.stack([byte & 15, byte >> 4], dim=-1).flatten(-2)
    m, e = (code & 1).to(dtype), ((code >> 1) & 3).to(dtype)
    v = torch.where(e > 0, (1 + 0.5 * m) * torch.exp2(e - 1), 0.5 * m)
    v = torch.where(code > 7, -v, v).unflatten(-1, (SCALES, GROUP))
    scale = (rec[..., CODES:CODES + SCALES].to(torch.int16) << 7).view(torch.half).to(dtype)
    return (v * scale[..., None]).flatten(-2), rec[..., CODES + SCALES:].contiguous().view(torch.bfloat16).to(dtype)


def _records(s, dtype, seq, j):
    """Latent and rope parts of positions j of sequences seq, zero where there is none."""
    bs = s["case"]["block"]
    stride = _strides(bs)[0]
    there = (j >= 0) & (j < s["seq_lens"][seq])
    jc = torch.where(there, j, torch.zeros_like(j)).long()
    rec = s["pool"].as_strided((s["blocks"], bs, REC), (stride, REC, 1))[s["block_table"][seq, jc // bs].long(), jc % bs]
    lat, rope = _from_4_bits(rec, dtype)
    zero = torch.zeros((), dtype=dtype, device=lat.device)
    return torch.where(there[..., None], lat, zero), torch.where(there[..., None], rope, zero)


def _tables_plain(s):
    bs, rows, new, free = s["case"]["block"], s["rows"].long(), s["new"], s["free"]
    b, stride = s["block_table"].shape
    dev = rows.device
    start, held = s["lens"][rows], s["held"][rows]
    end = start + new
    blocks = (end + bs - 1) // bs
    need = (blocks - held).clamp(min=0)
    first = s["used"] + need.cumsum(0) - need  # of the free list, for each entry
    j = torch.arange(stride, device=dev, dtype=torch.int32)[None]
    fresh = (j >= held[:, None]) & (j < blocks[:, None])
    ids = torch.where(fresh, free[(first[:, None] + j - held[:, None]).clamp(0, free.numel() - 1)], s["table"][rows])
    table, held_out = s["table"].clone(), s["held_out"].clone()
    table[rows] = ids
    held_out[rows] = torch.maximum(held, blocks)
    qsl = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), new.cumsum(0)])
    t = torch.arange(s["tokens"], device=dev)
    real = t < qsl[-1]
    e = torch.searchsorted(qsl[1:], t, right=True).clamp(max=b - 1)
    pos = torch.where(real, start[e] + t - qsl[e], 0)
    slots = torch.where(real, ids[e, (pos // bs).clamp(max=stride - 1)].long() * bs + pos % bs, -1)
    return {"seq_lens": end, "query_start_loc": qsl.int(), "positions": pos, "slots": slots, "table": table, "held": held_out,
            "block_table": torch.where(j < blocks[:, None], ids, torch.zeros_like(ids)), "used": s["used"] + need.sum()}


def _append_plain(s):
    cs, n = s["table"][s["positions"]], s["rows"]
    x, r, k = s["kv"][:, :D_LATENT].float(), s["kv"][:, D_LATENT:].float(), s["idx_k"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["norm"]
    if s["idx_bias"] is not None:
        k = k - k.mean(-1, keepdim=True)
    z = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["idx_norm"]
    if s["idx_bias"] is not None:
        z = z + s["idx_bias"]
    z = torch.cat([_rotate(z[:, :D_ROPE], cs, False), z[:, D_ROPE:]], dim=1)
    amax = z.abs().amax(-1, keepdim=True)
    bs, v = s["case"]["block"], _key_views(s)
    blk, off = s["slots"][:n] // bs, s["slots"][:n] % bs
    v["key_codes"].view(torch.uint8)[blk, off] = (z * (E4M3_MAX / amax)).to(torch.float8_e4m3fn).view(torch.uint8)[:n]
    v["key_scales"][blk, off] = (amax / E4M3_MAX)[:n, 0]
    return {"latent": _to_4_bits(y)[:n].bfloat16(), "rope": _rotate(r, cs, s["case"]["interleaved"]).bfloat16()[:n], **v}


def _load_plain(s):
    r = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["row_loc"][1:].long(), r, right=True)
    lat, rope = _records(s, torch.float32, seq, s["starts"][seq] + r - s["row_loc"][seq])
    return {"latent": lat.bfloat16(), "rope": rope.bfloat16()}


def _attend_plain(s):
    b, h, nq, ctx = s["case"]["batch"], s["case"]["heads"], s["max_q"], s["max_ctx"]
    dev = s["q"].device
    start, count = s["row_loc"][:-1], s["row_loc"].diff()
    i = torch.arange(nq, device=dev)[None]
    here = i < count[:, None]                                         # [b, nq] rows that are query tokens
    row = torch.where(here, start[:, None] + i, start[:, None]).long()
    pos = s["starts"][:, None] + i                                     # the last position that each sees
    seq = torch.arange(b, device=dev)[:, None]
    j = torch.arange(ctx, device=dev)[None].expand(b, ctx)
    lat, rope = _records(s, torch.float32, seq, j)
    x = torch.bmm(s["q"][row].float().view(b, nq * h, D_LATENT), lat.transpose(1, 2))
    x += torch.bmm(s["q_pe"][row].float().view(b, nq * h, D_ROPE), rope.transpose(1, 2))
    x = x.mul_(s["scale"]).view(b, nq, h, ctx)
    x.masked_fill_((j[:, None] > pos[:, :, None])[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    x.div_(total)
    out = torch.bmm(x.view(b, nq * h, ctx), lat).view(b, nq, h, D_LATENT)
    return {"out": out[here].bfloat16(), "lse": (top + total.log())[..., 0][here]}


def _select_plain(s):
    t = s["rows"]
    seq = torch.searchsorted(s["row_loc"][1:].long(), torch.arange(t, device="cuda"), right=True)[:, None]
    lat, rope = _records(s, torch.float32, seq, s["topk"])
    x = torch.bmm(s["q"].float(), lat.transpose(1, 2)) + torch.bmm(s["q_pe"].float(), rope.transpose(1, 2))
    x = x.mul_(s["scale"]).masked_fill_((s["topk"] < 0)[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return {"out": torch.bmm(x.div_(total), lat).bfloat16(), "lse": (top + total.log())[..., 0]}


def run(s):
    if not own:
        return {"tables": _tables_plain, "append": _append_plain, "load": _load_plain, "attend": _attend_plain, "select": _select_plain}[s["op"]](s)
    smla = s["smla"]
    if s["op"] == "tables":
        smla.smla_step_tables(s["layout"], s["lens"], s["new"], s["table"], s["held"], s["held_out"], s["free"], s["used"], s["used_out"], s["seq_lens"],
                              s["qsl"], s["positions"], s["slots"], rows=s["rows"], block_table=s["block_table"], workspace=s["workspace"])
        return {"seq_lens": s["seq_lens"], "query_start_loc": s["qsl"], "positions": s["positions"], "slots": s["slots"], "table": s["table"],
                "held": s["held_out"], "block_table": s["block_table"], "used": s["used_out"]}
    if s["op"] == "append":
        smla.kvpack_append(s["layout"], s["pool"], 0, s["kv"][:, :D_LATENT], s["kv"][:, D_LATENT:], s["idx_k"], s["rope"], s["positions"], s["slots"],
                           latent_norm=s["norm"], idx_norm=s["idx_norm"], idx_bias=s["idx_bias"], eps=EPS)
    if s["op"] in ("append", "load"):
        smla.kvpack_load(s["layout"], s["pool"], 0, s["block_table"], s["row_loc"], s["latent_out"], s["rope_out"], starts=s["starts"])
        return {"latent": s["latent_out"], "rope": s["rope_out"], **(_key_views(s) if s["op"] == "append" else {})}
    if s["op"] == "attend":
        smla.smla_attend_dense(s["layout"], s["params"], s["pool"], 0, s["q"], s["q_pe"], s["block_table"], s["seq_lens"], s["row_loc"], s["out"], s["lse"],
                               workspace=s["workspace"])
    else:
        smla.smla_attend(s["layout"], s["params"], s["pool"], 0, s["q"], s["q_pe"], s["topk"], s["block_table"], s["row_loc"], s["out"], s["lse"],
                         workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    if case["op"] == "tables":
        lens, new, more = _new_tokens(case)
        blocks = sum(-(-(n + q) // case["block"]) for n, q in zip(lens, new))
        # the held ids read and written, the new ones from the free list, positions and slots, and an entry's scalars
        return {"bytes": 8 * blocks + 16 * (sum(new) + case["pad"]) + 28 * len(lens), "flops": 0}
    lens, counts = _geometry(case)
    t = sum(counts)
    if case["op"] == "append":  # bf16 latent, rope and key, position, slot and a row of the table; record, key and scale; the rows read back
        return {"bytes": t * (2 * (D_LATENT + D_ROPE + D_INDEX) + 16 + 4 * D_ROPE + REC + D_INDEX + 4 + 2 * (D_LATENT + D_ROPE)),
                "flops": t * 12 * (D_LATENT + D_INDEX)}
    if case["op"] == "load":
        return {"bytes": t * (REC + 2 * (D_LATENT + D_ROPE)), "flops": t * D_LATENT}
    if case["op"] == "select":
        sees = [min(case["top_k"], n - c + i + 1) for n, c in zip(lens, counts) for i in range(c)]
        # tokens of a sequence may pick the same positions: at most every record once
        records = sum(min(n, c * case["top_k"]) for n, c in zip(lens, counts))
        io, seen = t * case["top_k"] * 4, sum(sees)
    else:
        records, io = sum(lens), 0
        seen = sum(c * (2 * n - c + 1) // 2 for n, c in zip(lens, counts))  # (query token, visible position) pairs
    return {"bytes": records * REC + t * case["heads"] * ((2 * D_LATENT + D_ROPE) * 2 + 4) + io, "flops": seen * case["heads"] * 2 * (2 * D_LATENT + D_ROPE)}


def _values64(rec):
    """Latent and rope of records [n, REC] by looking their codes up."""
    f64 = torch.float64
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=f64, device=rec.device)
    e2m1 = torch.cat([e2m1, -e2m1])
    i = torch.arange(256, dtype=f64, device=rec.device)
    e, m = (i / 8).floor(), i % 8
    ue5m3 = torch.where(e == 0, m * 2.0 ** -17, (8 + m) * torch.exp2(e - 18))
    lat = torch.empty(rec.shape[0], D_LATENT, dtype=f64, device=rec.device)
    lat[:, 0::2], lat[:, 1::2] = e2m1[(rec[:, :CODES] % 16).long()], e2m1[(rec[:, :CODES] // 16).long()]
    scale = ue5m3[rec[:, CODES:CODES + SCALES].long()]
    return lat * scale.repeat_interleave(GROUP, dim=1), rec[:, CODES + SCALES:].contiguous().view(torch.bfloat16).to(f64)


def _turn64(x, cos, sin, interleaved):
    """Each pair of the last axis as a complex number, times e^(i angle)."""
    i = torch.arange(D_ROPE // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + D_ROPE // 2)
    z = torch.complex(x[..., a], x[..., b]) * torch.complex(cos, sin)
    y = torch.empty_like(x)
    y[..., a], y[..., b] = z.real, z.imag
    return y


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    f64, bs = torch.float64, case["block"]
    lens, counts = _geometry(case)
    if case["op"] == "append":  # the key before quantisation, its codes in units of the unrounded scale
        t = s["rows"]
        cs = s["table"].to(f64)[s["positions"][:t]]
        cos, sin = cs[:, :D_ROPE // 2], cs[:, D_ROPE // 2:]
        k = s["idx_k"][:t].to(f64)
        if s["idx_bias"] is None:
            z = k / (k.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["idx_norm"].to(f64)
        else:
            z = (k - k.mean(-1, keepdim=True)) / (k.var(-1, unbiased=False, keepdim=True) + EPS).sqrt() * s["idx_norm"].to(f64) + s["idx_bias"].to(f64)
        z[:, :D_ROPE] = _turn64(z[:, :D_ROPE].clone(), cos, sin, False)
        zs = z.abs().amax(-1) / E4M3_MAX
        # a latent next to the border of two codes (a tenth of the value apart) may fall to either side in 32 bits: no value for it
        out = {"latent": None, "rope": _turn64(s["kv"][:t, D_LATENT:].to(f64), cos, sin, case["interleaved"])}
        for name, v in (("key_codes", z / zs[:, None]), ("key_scales", zs)):
            full = torch.zeros((s["blocks"] * bs,) + v.shape[1:], dtype=f64, device="cuda")
            full[s["slots"][:t]] = v
            out[name] = full.unflatten(0, (s["blocks"], bs))
        return out
    stride = _strides(bs)[0]
    rec = s["pool"].as_strided((s["blocks"], bs, REC), (stride, REC, 1))
    got, at = {"latent": [], "rope": [], "out": [], "lse": []}, 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        lat, rope = _values64(rec[s["block_table"][b, :-(-n // bs)].long()].reshape(-1, REC)[:n])
        if case["op"] == "load":
            got["latent"].append(lat[n - c:])
            got["rope"].append(rope[n - c:])
            continue
        key, h = torch.cat([lat, rope], 1), case["heads"]
        step = max(1, (1 << 28) // (n * h))
        for i in range(0, c, step):
            e = min(c, i + step)
            q = torch.cat([s["q"][at + i:at + e], s["q_pe"][at + i:at + e]], 2).to(f64)
            x = (q.reshape(-1, D_LATENT + D_ROPE) @ key.T).view(e - i, h, n) * s["scale"]
            if case["op"] == "attend":
                sees = torch.arange(n, device="cuda")[None] <= n - c + torch.arange(i, e, device="cuda")[:, None]
            else:
                pick = s["topk"][at + i:at + e].long()
                sees = torch.zeros(e - i, n + 1, dtype=torch.bool, device="cuda").scatter_(1, torch.where(pick < 0, n, pick), True)[:, :n]
            x = x.masked_fill(~sees[:, None], -math.inf)
            got["lse"].append(torch.logsumexp(x, -1))
            got["out"].append((torch.softmax(x, -1).view(-1, n) @ lat).view(e - i, h, D_LATENT))
        at += c
    return {k: torch.cat(v) for k, v in got.items() if v}
