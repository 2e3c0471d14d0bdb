"""What kvpack_append, smla_query_prep and smla_attend_dense refuse, on CPU.

The binding's checks run on CPU tensors: well-formed calls stop only at "CUDA tensors only", anything a
kernel could overrun or misread is refused before.  The C entry points answer bad arguments with a status
before any device work; the addresses given to them here are never dereferenced.
"""
import ctypes

import pytest
import torch

import paged_sparse_mla_gb300 as smla
from paged_sparse_mla_gb300 import build_lib

BF, F, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return smla.lib()


def layout(bs=16, dl=512, dr=64, tile=128, di=128, blocks=4, layers=2, **kw):
    return smla.layout_init(bs, layers, dl, dr, tile, di, blocks, **kw)


def params(heads=8, idx=4):
    return smla.make_params(heads, idx, 8, 0.1)


# ---------------------------------- the binding ----------------------------------

def append_args(lay, n=3):
    return dict(layout=lay, pool=torch.zeros(lay.pool_bytes, dtype=U8), layer=0, latent=torch.zeros(n, 512, dtype=BF),
                rope_key=torch.zeros(n, 64, dtype=BF), idx_k=torch.zeros(n, 128, dtype=BF),
                rope=smla.make_rope(torch.zeros(10, 64), True), positions=torch.zeros(n, dtype=I64),
                slot_mapping=torch.zeros(n, dtype=I64), latent_norm=torch.ones(512), idx_norm=torch.ones(128),
                idx_bias=torch.zeros(128))


def query_args(lay, prm, n=3):
    return dict(layout=lay, params=prm, rope=smla.make_rope(torch.zeros(10, 64), True), positions=torch.zeros(n, dtype=I64),
                q_pe=torch.zeros(n, 8, 64, dtype=BF), q_pe_out=torch.zeros(n, 8, 64, dtype=BF),
                q_idx=torch.zeros(n, 4, 128, dtype=BF), w=torch.zeros(n, 4), q_idx_out=torch.zeros(n, 4, 128, dtype=U8),
                w_out=torch.zeros(n, 4), idx_norm=torch.ones(128))


def dense_args(lay, prm, n=3):
    return dict(layout=lay, params=prm, pool=torch.zeros(lay.pool_bytes, dtype=U8), layer=0, q=torch.zeros(n, 8, 512, dtype=BF),
                q_pe=torch.zeros(n, 8, 64, dtype=BF), block_table=torch.zeros(2, 2, dtype=I32),
                seq_lens=torch.zeros(2, dtype=I32), query_start_loc=torch.zeros(3, dtype=I32),
                out=torch.zeros(n, 8, 512, dtype=BF), lse=torch.zeros(n, 8),
                workspace=torch.zeros(smla.attend_dense_workspace_size(lay, prm, n), dtype=U8))


MAKE = {"append": (smla.kvpack_append, lambda: append_args(layout())),
        "query": (smla.smla_query_prep, lambda: query_args(layout(), params())),
        "dense": (smla.smla_attend_dense, lambda: dense_args(layout(), params()))}


@pytest.mark.parametrize("which,without", [
    ("append", ()), ("append", ("latent_norm", "idx_bias")), ("append", ("idx_k", "idx_norm", "idx_bias")), ("append", ("rope", "positions")),
    ("query", ()), ("query", ("q_idx", "w", "q_idx_out", "w_out", "idx_norm")), ("query", ("q_pe", "q_pe_out")),
    ("dense", ()), ("dense", ("lse", "workspace")),
])
def test_well_formed_calls_reach_the_device_check(lib, which, without):
    call, make = MAKE[which]
    a = make()
    for k in without:
        a[k] = None
    with pytest.raises(ValueError, match="CUDA tensors only"):
        call(**a)


def short(t):
    return t.reshape(-1)[:-1]


@pytest.mark.parametrize("which,arg,change", [
    *[("append", a, short) for a in ("pool", "latent_norm", "idx_norm", "idx_bias", "positions")],
    *[("append", a, lambda t: t[:-1]) for a in ("latent", "rope_key", "idx_k")],             # a row too few
    *[("append", a, lambda t: t[:, :-8]) for a in ("latent", "rope_key", "idx_k")],          # too narrow
    *[("append", a, lambda t: t.repeat_interleave(2, 1)[:, ::2]) for a in ("latent", "rope_key", "idx_k")],  # elements apart
    *[("query", a, short) for a in ("positions", "q_pe_out", "w", "q_idx_out", "w_out", "idx_norm")],
    *[("query", a, lambda t: t[:-1]) for a in ("q_idx",)],
    *[("query", a, lambda t: t[:, :-1]) for a in ("q_pe", "q_idx")],                         # a head too few
    *[("query", a, lambda t: t.repeat_interleave(2, 2)[..., ::2]) for a in ("q_pe", "q_idx")],
    *[("query", a, lambda t: None) for a in ("q_pe_out", "w", "q_idx_out", "w_out", "positions")],
    *[("dense", a, short) for a in ("pool", "q_pe", "query_start_loc", "out", "lse")],
    ("dense", "q", lambda t: t[:, :-1]), ("dense", "block_table", lambda t: t[:1]), ("dense", "block_table", lambda t: t[0]),
    ("dense", "q", lambda t: t.transpose(0, 1)), ("dense", "out", lambda t: t.repeat_interleave(2, 2)[..., ::2]),
    ("dense", "block_table", lambda t: t.repeat(1, 2)[:, :2]),
])
def test_buffers_that_do_not_fit_are_refused(lib, which, arg, change):
    call, make = MAKE[which]
    a = make()
    a[arg] = change(a[arg])
    with pytest.raises(ValueError, match="|".join((arg, "needed with", "contiguous"))) as e:
        call(**a)
    assert "CUDA tensors only" not in str(e.value)


@pytest.mark.parametrize("which,arg", [
    *[("append", a) for a in ("pool", "latent", "rope_key", "idx_k", "positions", "slot_mapping", "latent_norm", "idx_norm", "idx_bias")],
    *[("query", a) for a in ("positions", "q_pe", "q_pe_out", "q_idx", "w", "q_idx_out", "w_out", "idx_norm")],
    *[("dense", a) for a in ("pool", "q", "q_pe", "block_table", "seq_lens", "query_start_loc", "out", "lse", "workspace")],
])
def test_other_element_types_are_refused(lib, which, arg):
    call, make = MAKE[which]
    a = make()
    a[arg] = a[arg].to(torch.float64)
    with pytest.raises(TypeError, match=arg):
        call(**a)


def test_rotation_tables(lib):
    with pytest.raises(TypeError):
        smla.make_rope(torch.zeros(4, 64, dtype=torch.float64), True)
    with pytest.raises(ValueError):
        smla.make_rope(torch.zeros(64), True)
    with pytest.raises(ValueError):
        smla.make_rope(torch.zeros(4, 128)[:, :64], True)
    a = append_args(layout())
    a["rope"] = smla.make_rope(torch.zeros(10, 32), True)          # another width than d_rope
    with pytest.raises(ValueError, match="d_rope"):
        smla.kvpack_append(**a)
    b = query_args(layout(), params())
    b["q_pe"] = b["q_idx"] = None
    with pytest.raises(ValueError, match="needs q_pe or q_idx"):
        smla.smla_query_prep(**b)


# ---------------------------------- the C entry points ----------------------------------

P16 = 4096            # an aligned address that nothing reads
REF = ctypes.byref


def c_append(lib, lay, **over):
    a = dict(layout=REF(lay), pool=P16, layer=0, latent=P16, ls=512, rope_key=P16, rs=64, idx_k=P16, ks=128, latent_norm=P16,
             idx_norm=P16, idx_bias=P16, eps=1e-6, rope=None, positions=None, slots=P16, n=1, stream=None)
    a.update(over)
    return lib.kvpack_append(*a.values())


def c_query(lib, lay, prm, **over):
    a = dict(layout=REF(lay), params=REF(prm), rope=None, positions=None, q_pe=P16, pt=512, ph=64, q_pe_out=P16, q_idx=P16,
             it=512, ih=128, idx_norm=P16, eps=1e-6, w=P16, w_scale=1.0, q_idx_out=P16, w_out=P16, n=1, stream=None)
    a.update(over)
    return lib.smla_query_prep(*a.values())


def c_dense(lib, lay, prm, **over):
    a = dict(layout=REF(lay), params=REF(prm), pool=P16, layer=0, q=P16, q_pe=P16, table=P16, stride=4, lens=P16, qsl=P16, batch=1,
             n=1, out=P16, lse=P16, ws=None, ws_bytes=0, stream=None)
    a.update(over)
    return lib.smla_attend_dense(*a.values())


def rope(table=P16, rows=10, inter=1, idx_inter=1, idx=1):
    return REF(smla.Rope(table, rows, inter, idx_inter, idx))


NAN = float("nan")


@pytest.mark.parametrize("over", [
    dict(layout=None), dict(pool=None), dict(pool=P16 + 8), dict(layer=-1), dict(layer=2), dict(n=-1), dict(latent=None),
    dict(rope_key=None), dict(slots=None), dict(ls=-1), dict(rs=-64), dict(ks=-128), dict(idx_norm=None), dict(eps=-1.0), dict(eps=NAN),
    dict(rope=rope(), positions=None), dict(rope=rope(table=None), positions=P16), dict(rope=rope(rows=-1), positions=P16),
])
def test_append_refuses(lib, over):
    assert c_append(lib, layout(), **over) == INVALID


@pytest.mark.parametrize("over", [
    dict(layout=None), dict(params=None), dict(n=-1), dict(q_pe_out=None), dict(pt=-1), dict(ph=-1), dict(it=-1), dict(ih=-1),
    dict(w=None), dict(q_idx_out=None), dict(w_out=None), dict(eps=-1.0), dict(eps=NAN), dict(rope=rope(), positions=None),
    dict(rope=rope(table=None), positions=P16), dict(rope=rope(rows=-1), positions=P16),
])
def test_query_prep_refuses(lib, over):
    assert c_query(lib, layout(), params(), **over) == INVALID


@pytest.mark.parametrize("over", [
    dict(layout=None), dict(params=None), dict(pool=None), dict(pool=P16 + 8), dict(layer=2), dict(layer=-1), dict(q=None),
    dict(q_pe=None), dict(table=None), dict(stride=0), dict(lens=None), dict(qsl=None), dict(batch=0), dict(n=-1), dict(out=None),
    dict(out=P16 + 8), dict(ws_bytes=64), dict(ws=P16 + 8, ws_bytes=1 << 30),
])
def test_attend_dense_refuses(lib, over):
    assert c_dense(lib, layout(), params(), **over) == INVALID


def test_layouts_not_made_by_layout_init(lib):
    lay, prm = layout(), params()
    lay.rec_stride += 16
    assert c_append(lib, lay) == c_query(lib, lay, prm) == c_dense(lib, lay, prm) == INVALID
    assert lib.smla_attend_dense_workspace_size(REF(lay), REF(prm), 4) == 0


def test_shapes_that_are_not_built(lib):
    prm = params()
    assert c_dense(lib, layout(), params(heads=129)) == UNSUPPORTED
    assert c_dense(lib, layout(dr=128), prm) == UNSUPPORTED
    assert c_dense(lib, layout(dl=1024), prm) == UNSUPPORTED
    assert c_append(lib, layout(dr=128)) == UNSUPPORTED
    assert c_append(lib, layout(dl=1024)) == UNSUPPORTED
    assert c_append(lib, layout(di=96)) == UNSUPPORTED
    assert c_query(lib, layout(di=96), prm) == UNSUPPORTED
    assert c_query(lib, layout(dr=128), prm) == UNSUPPORTED
    wide = layout(dr=64, di=32)                                     # the indexer cannot rotate 64 of 32 dims
    assert c_append(lib, wide, rope=rope(), positions=P16) != 0
    assert c_query(lib, wide, prm, rope=rope(), positions=P16) != 0


def test_nothing_to_do(lib):
    lay, prm = layout(), params()
    assert c_append(lib, lay, n=0, latent=None, slots=None) == 0
    assert c_query(lib, lay, prm, n=0, q_pe=None, q_idx=None) == 0
    assert c_query(lib, lay, prm, q_pe=None, q_idx=None) == 0
    assert c_dense(lib, lay, prm, n=0, q=None, out=None) == 0


def test_workspace_sizes(lib):
    full, small, prm = layout(), layout(dl=64, dr=16, tile=64, di=32), params()
    size = smla.attend_dense_workspace_size(full, prm, 1)
    assert 0 < size < 1 << 27 and size % 16 == 0
    assert smla.attend_dense_workspace_size(full, prm, 1 << 20) == size
    assert smla.attend_dense_workspace_size(full, prm, 0) == 0
    assert smla.attend_dense_workspace_size(small, prm, 8) == 0     # other shapes do not split
    assert lib.smla_attend_dense_workspace_size(None, REF(prm), 4) == 0
    assert lib.smla_attend_dense_workspace_size(REF(full), None, 4) == 0
