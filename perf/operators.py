"""The cache-writing, query-preparing and dense-attention operators: cases, inputs, plain forms and values in 64 bits.

Three operators around the packed, paged FP8 cache of latent attention:

* ``append``  norm, rotation, quantisation and scatter of new tokens into the cache;
* ``query``   rotation of the attention's q_pe, and norm, rotation and E4M3 quantisation of the indexer's queries;
* ``attend``  latent attention (absorbed form) of decode tokens or a chunk over the whole visible context.

``run`` computes them in plain torch operations in fp32, or, where ``own`` is true, through the library.
"""
import math
import random

import torch

own = False

D_LATENT, D_ROPE, TILE, D_INDEX = 512, 64, 128, 128   # the full shape of this repository's workloads
REC = D_LATENT + 4 * (D_LATENT // TILE) + 2 * D_ROPE  # bytes of one cached record
E4M3_MAX = 448.0
EPS = 1e-6
W_SCALE = 1.0 / math.sqrt(64 * 128)


def listed():
    return [
        # the first token of a short prompt on its own: latency
        {"name": "attend-first-token", "op": "attend", "batch": 1, "queries": 1, "ragged": False, "ctx_lo": 1, "ctx_hi": 1, "heads": 64, "block": 64},
        # the repository's decode batch: 32 sequences, one token each
        {"name": "attend-decode-b32", "op": "attend", "batch": 32, "queries": 1, "ragged": False, "ctx_lo": 8192, "ctx_hi": 32768, "heads": 64, "block": 64},
        # decode with three drafted tokens, 64 sequences, as the repository's agentic batch
        {"name": "attend-mtp4-b64", "op": "attend", "batch": 64, "queries": 4, "ragged": False, "ctx_lo": 4096, "ctx_hi": 32768, "heads": 64, "block": 64},
        # a prefill chunk on a cached prefix
        {"name": "attend-chunk-2048", "op": "attend", "batch": 1, "queries": 2048, "ragged": False, "ctx_lo": 18432, "ctx_hi": 18432, "heads": 64, "block": 64},
        # a mixed batch: chunks of uneven length beside decode tokens, 128 heads, small pages
        {"name": "attend-ragged-h128", "op": "attend", "batch": 5, "queries": 333, "ragged": True, "ctx_lo": 777, "ctx_hi": 5003, "heads": 128, "block": 16},
        # one long conversation, few heads (a model split by heads over several devices), one drafted token
        {"name": "attend-long-h16", "op": "attend", "batch": 1, "queries": 2, "ragged": False, "ctx_lo": 262143, "ctx_hi": 262143, "heads": 16, "block": 64},
        # one decode token
        {"name": "append-1", "op": "append", "tokens": 1, "block": 64, "interleaved": True, "idx_bias": True, "skip": 0},
        # a decode step of 64 sequences with three drafted tokens each, some slots unused
        {"name": "append-256", "op": "append", "tokens": 256, "block": 64, "interleaved": True, "idx_bias": True, "skip": 9},
        # a prefill chunk
        {"name": "append-8192", "op": "append", "tokens": 8192, "block": 64, "interleaved": False, "idx_bias": False, "skip": 0},
        # one decode token
        {"name": "query-1", "op": "query", "tokens": 1, "heads": 64, "idx_heads": 64, "interleaved": True, "norm": False},
        # the same decode step
        {"name": "query-256", "op": "query", "tokens": 256, "heads": 64, "idx_heads": 64, "interleaved": True, "norm": False},
        # the same chunk, with a norm of each head
        {"name": "query-8192", "op": "query", "tokens": 8192, "heads": 64, "idx_heads": 64, "interleaved": False, "norm": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "query"])
    if op == "append":
        n = _log(rng, 1, 8192)
        return {"op": op, "tokens": n, "block": rng.choice([16, 32, 64, 128]), "interleaved": rng.random() < 0.5,
                "idx_bias": rng.random() < 0.5, "skip": rng.randint(0, n // 4)}
    if op == "query":
        return {"op": op, "tokens": _log(rng, 1, 8192), "heads": rng.choice([8, 16, 24, 64]), "idx_heads": rng.choice([4, 32, 64]),
                "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.5}
    batch, queries, hi = _log(rng, 1, 64), _log(rng, 1, 1024), _log(rng, 1, 32768)
    heads = rng.choice([5, 8, 16, 32, 64, 64, 128])
    while queries > 1 and batch * queries * heads * max(hi, queries) > 2048 * 64 * 9216:
        queries = (queries + 1) // 2
    hi = max(hi, queries)
    return {"op": op, "batch": batch, "queries": queries, "ragged": rng.random() < 0.5, "ctx_lo": max(queries, hi // rng.choice([1, 2, 7])),
            "ctx_hi": hi, "heads": heads, "block": rng.choice([16, 32, 64, 128])}


def _lengths(case):
    """(cached tokens, query tokens) of each sequence: spread evenly, in an order fixed by the case."""
    b, lo, hi, q = case["batch"], case["ctx_lo"], case["ctx_hi"], case["queries"]
    lens = [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]
    r = random.Random(b * 1000003 + hi * 31 + q)
    r.shuffle(lens)
    counts = [q if not case["ragged"] or i == 0 else r.randint(1, q) for i in range(b)]
    return lens, counts


def _rec_stride(block):
    """(bytes of one block of one layer, offset of its keys, offset of its key scales): every region starts on 256 bytes."""
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    keys = up(block * REC)
    scales = up(keys + block * D_INDEX)
    return up(scales + 4 * block), keys, scales


def _rope_table(n, device):
    f = 10000.0 ** (-torch.arange(0, D_ROPE, 2, device=device, dtype=torch.float64) / D_ROPE)
    a = torch.arange(n, device=device, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    s = {"op": case["op"], "case": case}
    if case["op"] == "attend":
        lens, counts = _lengths(case)
        bs, b, h = case["block"], case["batch"], case["heads"]
        need = [-(-n // bs) for n in lens]
        blocks = sum(need)
        stride = _rec_stride(bs)[0]
        perm = torch.randperm(blocks, generator=g, device="cuda").int()
        table = torch.zeros(b, max(need), dtype=torch.int32, device="cuda")
        pool = torch.zeros(blocks, stride, dtype=torch.uint8, device="cuda")
        rec = torch.as_strided(pool, (blocks, bs, REC), (stride, REC, 1))
        step = max(1, (1 << 18) // bs)
        for k in range(0, blocks, step):
            n = min(step, blocks - k)
            codes = (rnd(n, bs, D_LATENT) * 160).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            scales = (0.8 + 0.4 * torch.rand(n, bs, 4, generator=g, device="cuda")) / 160
            rec[k:k + n, :, :D_LATENT] = codes.view(torch.uint8)
            rec[k:k + n, :, D_LATENT:D_LATENT + 16] = scales.view(torch.uint8)
            rec[k:k + n, :, D_LATENT + 16:] = rnd(n, bs, D_ROPE).bfloat16().view(torch.uint8)
        at = 0
        for i in range(b):
            table[i, :need[i]] = perm[at:at + need[i]]
            if lens[i] % bs:  # the unused end of a sequence's last page holds whatever was there: NaN codes, scales and ropes
                rec[table[i, need[i] - 1].long(), lens[i] % bs:] = 255
            at += need[i]
        t = sum(counts)
        s.update(pool=pool.view(-1), block_table=table, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 query_start_loc=torch.tensor([0] + counts, device="cuda").cumsum(0).int(), blocks=blocks, max_ctx=max(lens), max_q=max(counts),
                 q=rnd(t, h, D_LATENT).bfloat16(), q_pe=rnd(t, h, D_ROPE).bfloat16(), scale=1.0 / math.sqrt(D_LATENT + D_ROPE),
                 out=torch.empty(t, h, D_LATENT, dtype=torch.bfloat16, device="cuda"))
    else:
        n = case["tokens"]
        s.update(table=_rope_table(65536, "cuda"), positions=torch.randint(0, 65536, (n,), generator=g, device="cuda"))
        if case["op"] == "append":
            bs = case["block"]
            blocks = -(-n // bs) + 2
            kv = (rnd(n, D_LATENT + D_ROPE) * (0.5 + rnd(n, 1).abs())).bfloat16()  # the projection's output: latent and rope key side by side
            slots = torch.randperm(blocks * bs, generator=g, device="cuda")[:n].contiguous()
            slots[torch.randperm(n, generator=g, device="cuda")[:case["skip"]]] = -1
            s.update(pool=torch.zeros(blocks * _rec_stride(bs)[0], dtype=torch.uint8, device="cuda"), blocks=blocks, kv=kv, slots=slots,
                     idx_k=(rnd(n, D_INDEX) * 2 + 0.3).bfloat16(), norm=1 + 0.1 * rnd(D_LATENT), idx_norm=1 + 0.1 * rnd(D_INDEX),
                     idx_bias=0.1 * rnd(D_INDEX) if case["idx_bias"] else None)
        else:
            h, hi = case["heads"], case["idx_heads"]
            s.update(q=rnd(n, h, 128 + D_ROPE).bfloat16(),  # the projection's output: [.., 128:] is each head's q_pe
                     q_idx=(rnd(n, hi, D_INDEX) * (0.5 + rnd(n, hi, 1).abs())).bfloat16(), w=rnd(n, hi),
                     norm=1 + 0.1 * rnd(D_INDEX) if case["norm"] else None,
                     q_pe_out=torch.empty(n, h, D_ROPE, dtype=torch.bfloat16, device="cuda"),
                     codes=torch.empty(n, hi, D_INDEX, dtype=torch.uint8, device="cuda"), w_out=torch.empty(n, hi, device="cuda"))
    if own:  # the handles that a program keeps: layout, parameters, rotation table, workspace
        import paged_sparse_mla_gb300 as smla
        s["smla"] = smla
        if case["op"] == "attend":
            s["layout"] = smla.layout_init(case["block"], 1, D_LATENT, D_ROPE, TILE, D_INDEX, s["blocks"])
            s["params"] = smla.make_params(case["heads"], 64, 2048, s["scale"])
            s["workspace"] = torch.empty(smla.attend_dense_workspace_size(s["layout"], s["params"], s["q"].shape[0]), dtype=torch.uint8, device="cuda")
        elif case["op"] == "append":
            s["layout"] = smla.layout_init(case["block"], 1, D_LATENT, D_ROPE, TILE, D_INDEX, s["blocks"])
            s["rope"] = smla.make_rope(s["table"], interleaved=case["interleaved"], idx_interleaved=False, idx_rope=True)
        else:
            s["layout"] = smla.layout_init(64, 1, D_LATENT, D_ROPE, TILE, D_INDEX, 1)
            s["params"] = smla.make_params(case["heads"], case["idx_heads"], 2048, 1.0)
            s["rope"] = smla.make_rope(s["table"], interleaved=case["interleaved"], idx_interleaved=False, idx_rope=True)
    return s


def _pool_views(pool, bs, blocks):
    """The cache's parts as tensors: latent codes, their scales, rope keys, indexer-key codes, their scales."""
    stride, keys, scales = _rec_stride(bs)
    f8, f32, b16 = pool.view(torch.float8_e4m3fn), pool.view(torch.float32), pool.view(torch.bfloat16)
    return {"codes": f8.as_strided((blocks, bs, D_LATENT), (stride, REC, 1), 0),
            "scales": f32.as_strided((blocks, bs, 4), (stride // 4, REC // 4, 1), D_LATENT // 4),
            "rope": b16.as_strided((blocks, bs, D_ROPE), (stride // 2, REC // 2, 1), (D_LATENT + 16) // 2),
            "key_codes": f8.as_strided((blocks, bs, D_INDEX), (stride, D_INDEX, 1), keys),
            "key_scales": f32.as_strided((blocks, bs), (stride // 4, 1), scales // 4)}


def _rotate(x, cs, interleaved):
    """x [..., d] rotated by the angles whose cosines and sines are cs [..., d]."""
    half = D_ROPE // 2
    c, s = cs[..., :half], cs[..., half:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1)


def _quantise(x):
    """(E4M3 codes, scale) of the last axis; an all-but-zero vector has scale 1."""
    amax = x.abs().amax(-1, keepdim=True)
    tiny = amax < 2.0 ** -100
    scale = torch.where(tiny, torch.ones_like(amax), amax / E4M3_MAX)
    return (x * torch.where(tiny, torch.ones_like(amax), E4M3_MAX / amax)).to(torch.float8_e4m3fn), scale[..., 0]


def _append_plain(s):
    case = s["case"]
    cs = s["table"][s["positions"]]
    x, r, k = s["kv"][:, :D_LATENT].float(), s["kv"][:, D_LATENT:].float(), s["idx_k"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["norm"]
    codes, scales = _quantise(y.view(-1, 4, TILE))
    if s["idx_bias"] is not None:
        k = k - k.mean(-1, keepdim=True)
    z = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["idx_norm"]
    if s["idx_bias"] is not None:
        z = z + s["idx_bias"]
    z = torch.cat([_rotate(z[:, :D_ROPE], cs, False), z[:, D_ROPE:]], dim=1)
    key, key_scale = _quantise(z)
    keep = s["slots"] >= 0
    blk, off = s["slots"][keep] // case["block"], s["slots"][keep] % case["block"]
    v = _pool_views(s["pool"], case["block"], s["blocks"])
    v["codes"].view(torch.uint8)[blk, off] = codes.view(torch.uint8).view(-1, D_LATENT)[keep]
    v["scales"][blk, off] = scales[keep]
    v["rope"][blk, off] = _rotate(r, cs, case["interleaved"]).bfloat16()[keep]
    v["key_codes"].view(torch.uint8)[blk, off] = key.view(torch.uint8)[keep]
    v["key_scales"][blk, off] = key_scale[keep]
    return v


def _query_plain(s):
    cs = s["table"][s["positions"]][:, None]
    x = s["q_idx"].float()
    if s["norm"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["norm"]
    x = torch.cat([_rotate(x[..., :D_ROPE], cs, False), x[..., D_ROPE:]], dim=-1)
    codes, scale = _quantise(x)
    return {"q_pe": _rotate(s["q"][..., 128:].float(), cs, s["case"]["interleaved"]).bfloat16(), "codes": codes, "w": s["w"] * W_SCALE * scale}


def _records(s, dtype, seq, j):
    """Latent and rope parts of positions j of sequences seq, zero past a sequence's length."""
    bs = s["case"]["block"]
    stride = _rec_stride(bs)[0]
    there = j < s["seq_lens"][seq]
    jc = torch.where(there, j, torch.zeros_like(j)).long()
    rec = s["pool"].as_strided((s["blocks"], bs, REC), (stride, REC, 1))[s["block_table"][seq, jc // bs].long(), jc % bs]
    lat = rec[..., :D_LATENT].view(torch.float8_e4m3fn).to(dtype).unflatten(-1, (4, TILE))
    lat = (lat * rec[..., D_LATENT:D_LATENT + 16].contiguous().view(torch.float32).to(dtype)[..., None]).flatten(-2)
    rope = rec[..., D_LATENT + 16:].contiguous().view(torch.bfloat16).to(dtype)
    zero = torch.zeros((), dtype=dtype, device=lat.device)
    return torch.where(there[..., None], lat, zero), torch.where(there[..., None], rope, zero)


def _attend_plain(s):
    b, h, nq, ctx = s["case"]["batch"], s["case"]["heads"], s["max_q"], s["max_ctx"]
    dev = s["q"].device
    start, count = s["query_start_loc"][:-1], s["query_start_loc"].diff()
    i = torch.arange(nq, device=dev)[None]
    here = i < count[:, None]                                         # [b, nq] rows that are query tokens
    row = torch.where(here, start[:, None] + i, start[:, None]).long()
    pos = s["seq_lens"][:, None] - count[:, None] + i                  # the last position that each sees
    seq = torch.arange(b, device=dev)[:, None]
    j = torch.arange(ctx, device=dev)[None].expand(b, ctx)
    lat, rope = _records(s, torch.float32, seq, j)
    x = torch.bmm(s["q"][row].float().view(b, nq * h, D_LATENT), lat.transpose(1, 2))
    x += torch.bmm(s["q_pe"][row].float().view(b, nq * h, D_ROPE), rope.transpose(1, 2))
    x = x.mul_(s["scale"]).view(b, nq, h, ctx)
    x.masked_fill_((j[:, None] > pos[:, :, None])[:, :, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    out = torch.bmm(x.view(b, nq * h, ctx), lat).view(b, nq, h, D_LATENT)
    return {"out": out[here].bfloat16()}


def run(s):
    if not own:
        return {"attend": _attend_plain, "append": _append_plain, "query": _query_plain}[s["op"]](s)
    smla = s["smla"]
    if s["op"] == "attend":
        smla.smla_attend_dense(s["layout"], s["params"], s["pool"], 0, s["q"], s["q_pe"], s["block_table"], s["seq_lens"], s["query_start_loc"],
                               s["out"], workspace=s["workspace"])
        return {"out": s["out"]}
    if s["op"] == "append":
        smla.kvpack_append(s["layout"], s["pool"], 0, s["kv"][:, :D_LATENT], s["kv"][:, D_LATENT:], s["idx_k"], s["rope"], s["positions"], s["slots"],
                           latent_norm=s["norm"], idx_norm=s["idx_norm"], idx_bias=s["idx_bias"], eps=EPS)
        return _pool_views(s["pool"], s["case"]["block"], s["blocks"])
    smla.smla_query_prep(s["layout"], s["params"], s["rope"], s["positions"], q_pe=s["q"][..., 128:], q_pe_out=s["q_pe_out"], q_idx=s["q_idx"], w=s["w"],
                         w_scale=W_SCALE, q_idx_out=s["codes"], w_out=s["w_out"], idx_norm=s["norm"], eps=EPS)
    return {"q_pe": s["q_pe_out"], "codes": s["codes"].view(torch.float8_e4m3fn), "w": s["w_out"]}


def work(case):
    if case["op"] == "append":
        n = case["tokens"] - case["skip"]  # bf16 latent, rope and key, position, slot and a row of the table; record, key and scale
        return {"bytes": n * (2 * (D_LATENT + D_ROPE + D_INDEX) + 16 + 4 * D_ROPE + REC + D_INDEX + 4), "flops": n * 12 * (D_LATENT + D_INDEX)}
    if case["op"] == "query":
        n, h, hi = case["tokens"], case["heads"], case["idx_heads"]
        return {"bytes": n * (4 * h * D_ROPE + 3 * hi * D_INDEX + 8 * hi + 8 + 4 * D_ROPE), "flops": n * 10 * (h * D_ROPE + hi * D_INDEX)}
    lens, counts = _lengths(case)
    seen = sum(c * (2 * n - c + 1) // 2 for n, c in zip(lens, counts))  # (query token, visible position) pairs
    return {"bytes": sum(lens) * REC + sum(counts) * case["heads"] * (2 * D_LATENT + D_ROPE) * 2,
            "flops": seen * case["heads"] * 2 * (2 * D_LATENT + D_ROPE)}


def _turn64(x, angle_cos, angle_sin, pairs):
    """Each pair (x_a, x_b) of the last axis as a complex number, times e^(i angle)."""
    z = torch.complex(x[..., pairs[0]], x[..., pairs[1]]) * torch.complex(angle_cos, angle_sin)
    y = torch.empty_like(x)
    y[..., pairs[0]], y[..., pairs[1]] = z.real, z.imag
    return y


def _pairs(interleaved):
    i = torch.arange(D_ROPE // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + D_ROPE // 2)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "attend":
        lens, counts = _lengths(case)
        h, at, outs = case["heads"], 0, []
        for b in range(case["batch"]):
            n, c = lens[b], counts[b]
            lat, rope = _records(s, f64, torch.full((n,), b, device="cuda"), torch.arange(n, device="cuda"))
            key = torch.cat([lat, rope], 1)
            step = max(1, (1 << 28) // (n * h))
            for i in range(0, c, step):
                e = min(c, i + step)
                q = torch.cat([s["q"][at + i:at + e], s["q_pe"][at + i:at + e]], 2).to(f64)
                x = (q.reshape(-1, D_LATENT + D_ROPE) @ key.T).view(e - i, h, n) * s["scale"]
                last = n - c + torch.arange(i, e, device="cuda")
                x = x.masked_fill(torch.arange(n, device="cuda")[None, None] > last[:, None, None], -math.inf)
                outs.append((torch.softmax(x, -1).view(-1, n) @ lat).view(e - i, h, D_LATENT))
            at += c
        return {"out": torch.cat(outs)}
    cs = s["table"].to(f64)[s["positions"]]
    cos, sin = cs[:, :D_ROPE // 2], cs[:, D_ROPE // 2:]
    if case["op"] == "query":
        x = s["q_idx"].to(f64)
        if s["norm"] is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["norm"].to(f64)
        x[..., :D_ROPE] = _turn64(x[..., :D_ROPE].clone(), cos[:, None], sin[:, None], _pairs(False))
        scale = x.abs().amax(-1) / E4M3_MAX
        return {"q_pe": _turn64(s["q"][..., 128:].to(f64), cos[:, None], sin[:, None], _pairs(case["interleaved"])),
                "codes": x / scale[..., None], "w": s["w"].to(f64) * W_SCALE * scale}
    x, k = s["kv"][:, :D_LATENT].to(f64), s["idx_k"].to(f64)
    y = (x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["norm"].to(f64)).view(-1, 4, TILE)
    if s["idx_bias"] is None:
        z = k / (k.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["idx_norm"].to(f64)
    else:
        z = (k - k.mean(-1, keepdim=True)) / (k.var(-1, unbiased=False, keepdim=True) + EPS).sqrt() * s["idx_norm"].to(f64) + s["idx_bias"].to(f64)
    z[:, :D_ROPE] = _turn64(z[:, :D_ROPE].clone(), cos, sin, _pairs(False))
    ys, zs = y.abs().amax(-1) / E4M3_MAX, z.abs().amax(-1) / E4M3_MAX
    got = {"codes": (y / ys[..., None]).view(-1, D_LATENT), "scales": ys, "rope": _turn64(s["kv"][:, D_LATENT:].to(f64), cos, sin, _pairs(case["interleaved"])),
           "key_codes": z / zs[:, None], "key_scales": zs}
    keep = s["slots"] >= 0
    out = {}
    for name, v in got.items():
        full = torch.zeros((s["blocks"] * case["block"],) + v.shape[1:], dtype=f64, device="cuda")
        full[s["slots"][keep]] = v[keep]
        out[name] = full.unflatten(0, (s["blocks"], case["block"]))
    return out
