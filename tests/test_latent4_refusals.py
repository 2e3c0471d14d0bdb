"""What 4-bit latent layouts, kvpack_load and smla_step_tables refuse, on CPU (see test_operator_refusals.py)."""
import ctypes

import pytest
import torch

import oracle
import paged_sparse_mla_gb300 as smla
from paged_sparse_mla_gb300 import build_lib

BF, F, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
INVALID, UNSUPPORTED = 1, 2
P16 = 4096            # an aligned address that nothing reads
REF = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return smla.lib()


def layout(bs=16, dl=512, dr=64, di=128, blocks=4, layers=2, keys="e4m3", fmt="e2m1"):
    return smla.layout_init(bs, layers, dl, dr, 16 if fmt == "e2m1" else 128, di, blocks, keys, latent_format=fmt)


@pytest.mark.parametrize("keys", ["e4m3", "e2m1"])
@pytest.mark.parametrize("args", [(64, 1, 512, 64, 128, 1000), (16, 1, 64, 16, 32, 32), (64, 3, 256, 0, 128, 7), (7, 2, 128, 32, 64, 5)])
def test_layout_is_the_oracles(lib, args, keys):
    bs, layers, dl, dr, di, blocks = args
    lay = smla.layout_init(bs, layers, dl, dr, 16, di, blocks, keys, latent_format="e2m1")
    ref = oracle.PoolLayout(bs, layers, dl, dr, 16, di, blocks, keys, "e2m1")
    assert smla.latent_format(lay) == "e2m1" and lay.rec_bytes == ref.rec_bytes and lay.rec_stride == ref.rec_stride
    assert (lay.idx_key_off, lay.idx_scale_off, lay.block_stride, lay.pool_bytes) == (ref.idx_key_off, ref.idx_scale_off, ref.block_stride, ref.pool_bytes)
    # E4M3 latents in tiles of 16 are another layout of the same shape fields
    other = smla.layout_init(bs, layers, dl, dr, 16 if dl == 512 else max(16, dl // 4), di, blocks, keys)
    assert smla.latent_format(other) == "e4m3" and other.rec_bytes > lay.rec_bytes


def test_layout_refusals(lib):
    L = REF(smla.Layout())
    assert lib.smla_layout_init_latents(L, 64, 1, 512, 64, 16, 128, 0, 1, 10) == 0
    assert lib.smla_layout_init_latents(L, 64, 1, 512, 64, 128, 128, 0, 1, 10) == INVALID     # E2M1 latents have groups of 16
    assert lib.smla_layout_init_latents(L, 64, 1, 512, 64, 16, 128, 0, 2, 10) == INVALID      # no such format
    assert lib.smla_layout_init_latents(L, 64, 1, 500, 64, 16, 128, 0, 1, 10) == INVALID
    assert lib.smla_layout_init_latents(None, 64, 1, 512, 64, 16, 128, 0, 1, 10) == INVALID
    assert lib.smla_layout_latent_format(None) == -1
    with pytest.raises(ValueError):
        smla.layout_init(64, 1, 512, 64, 16, 128, 10, latent_format="fp4")
    with pytest.raises(ValueError):
        smla.layout_init(64, 1, 512, 64, 16, 128, 10, key_format="fp4", latent_format="e2m1")


@pytest.mark.parametrize("field,delta", [("rec_bytes", 16), ("rec_bytes", 352), ("rec_stride", 16), ("idx_key_off", 256), ("n_scales", -4),
                                         ("quant_tile", 112), ("block_stride", 256)])
def test_changed_layouts_are_refused(lib, field, delta):
    lay = layout()
    setattr(lay, field, getattr(lay, field) + delta)
    prm = smla.make_params(8, 4, 8, 0.1)
    assert lib.smla_layout_latent_format(REF(lay)) == -1
    with pytest.raises(ValueError):
        smla.latent_format(lay)
    assert lib.kvpack_store(REF(lay), P16, 0, P16, P16, P16, P16, P16, 1, None) == INVALID
    assert lib.smla_attend(REF(lay), REF(prm), P16, 0, P16, P16, P16, P16, 4, P16, 1, 1, P16, P16, None, 0, None) == INVALID
    assert c_load(lib, lay) == c_tables(lib, lay) == INVALID


def test_unaligned_pools_of_4_bit_latents(lib):
    lay, prm = layout(), smla.make_params(64, 64, 64, 0.1)
    p = P16 + 8
    assert lib.kvpack_store(REF(lay), p, 0, P16, P16, P16, P16, P16, 1, None) == INVALID
    assert lib.smla_attend(REF(lay), REF(prm), p, 0, P16, P16, P16, P16, 4, P16, 1, 1, P16, P16, None, 0, None) == INVALID
    assert lib.smla_attend_hisparse(REF(lay), REF(prm), p, 0, P16, P16, 1, P16, P16, P16, P16, 4, P16, 1, 1, P16, P16, None) == INVALID
    step = (p, 0, P16, P16, P16, P16, P16, P16, P16, P16, P16, P16, 16, P16, P16, 1, 1, 1, 100, P16, P16, None)
    assert lib.smla_decode(REF(lay), REF(prm), *step, P16, 1 << 30, None) == INVALID
    assert lib.smla_decode_static(REF(lay), REF(prm), *step, None) == INVALID


# ---------------------------------- kvpack_load ----------------------------------

def c_load(lib, lay, **over):
    a = dict(layout=REF(lay), pool=P16, layer=0, table=P16, stride=4, starts=None, loc=P16, batch=1, n=1, lat=P16, ls=512, rope=P16, rs=64, stream=None)
    a.update(over)
    return lib.kvpack_load(*a.values())


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("over", [
    dict(layout=None), dict(pool=None), dict(pool=P16 + 8), dict(layer=-1), dict(layer=2), dict(table=None), dict(stride=0), dict(loc=None), dict(batch=0),
    dict(n=-1), dict(lat=None), dict(ls=511), dict(ls=-512), dict(rs=63),
])
def test_load_refuses(lib, over, fmt):
    assert c_load(lib, layout(fmt=fmt), **over) == INVALID


def test_load_of_nothing(lib):
    assert c_load(lib, layout(), n=0, lat=None) == 0


def load_args(n=5, b=2):
    lay = layout()
    return dict(layout=lay, pool=torch.zeros(lay.pool_bytes, dtype=U8), layer=0, block_table=torch.zeros(b, 3, dtype=I32), row_loc=torch.zeros(b + 1, dtype=I32),
                latent_out=torch.zeros(n, 512, dtype=BF), rope_out=torch.zeros(n, 64, dtype=BF), starts=torch.zeros(b, dtype=I32))


# ---------------------------------- smla_step_tables ----------------------------------

def c_tables(lib, lay, **over):
    a = dict(layout=REF(lay), rows=P16, lens=P16, new=P16, batch=2, table=P16, n_rows=3, ts=4, held=P16, held_out=P16, free=P16, n_free=5, used=P16,
             used_out=P16, n=4, seq=P16, qsl=P16, pos=P16, slots=P16, bt=1 << 20, bts=4, ws=P16, wsb=48, stream=None)
    a.update(over)
    return lib.smla_step_tables(*a.values())


@pytest.mark.parametrize("over", [
    dict(layout=None), dict(lens=None), dict(new=None), dict(batch=0), dict(table=None), dict(n_rows=0), dict(ts=0), dict(held=None), dict(held_out=None),
    dict(free=None), dict(n_free=-1), dict(used=None), dict(used_out=None), dict(n=-1), dict(seq=None), dict(qsl=None), dict(pos=None), dict(slots=None),
    dict(bt=None),                              # a selection of rows needs a table of its own
    dict(rows=None, batch=4, wsb=96),           # more entries than rows
    dict(bts=0), dict(bt=P16), dict(bt=P16 + 40), dict(bt=P16 - 28),   # over the persistent table
    dict(ws=None), dict(ws=P16 + 8), dict(wsb=47),
])
def test_step_tables_refuses(lib, over):
    assert c_tables(lib, layout(), **over) == INVALID


LENS, NEW, SEQ, QSL, HELD = 1 << 12, 1 << 13, 1 << 14, 1 << 15, 1 << 16   # apart, as every result is from the lengths


@pytest.mark.parametrize("over,refused", [
    (dict(), False), (dict(seq=LENS), True), (dict(seq=NEW), True), (dict(qsl=LENS), True), (dict(qsl=NEW - 8), True), (dict(seq=NEW - 8), False),
    (dict(held_out=LENS - 8), True), (dict(held_out=NEW), True), (dict(seq=LENS + 12), False), (dict(seq=LENS + 8), True),
])
def test_step_tables_results_over_the_lengths(lib, over, refused):
    args = dict(lens=LENS, new=NEW, seq=SEQ, qsl=QSL, held=HELD, held_out=HELD, table=1 << 18)
    args.update(over)
    if torch.cuda.is_available() and not refused:
        pytest.skip("a call with made-up addresses")
    assert (c_tables(lib, layout(), **args) == INVALID) == refused


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_unaligned_outputs_of_attention_over_4_bit_latents(lib, fmt):
    lay, prm = layout(fmt=fmt), smla.make_params(64, 64, 64, 0.1)
    if torch.cuda.is_available() and fmt == "e4m3":
        pytest.skip("a call with made-up addresses")
    out = P16 + 8
    step = (P16, 0, P16, P16, P16, P16, P16, P16, P16, P16, P16, P16, 16, P16, P16, 1, 1, 1, 100, out, P16, None)
    got = [lib.smla_attend(REF(lay), REF(prm), P16, 0, P16, P16, P16, P16, 4, P16, 1, 1, out, P16, None, 0, None),
           lib.smla_attend_hisparse(REF(lay), REF(prm), P16, 0, P16, P16, 1, P16, P16, P16, P16, 4, P16, 1, 1, out, P16, None),
           lib.smla_decode(REF(lay), REF(prm), *step, P16, 1 << 30, None)]
    assert [g == INVALID for g in got] == [fmt == "e2m1"] * 3


def test_step_tables_workspace(lib):
    assert smla.step_tables_workspace_size(10) == 240 and smla.step_tables_workspace_size(0) == 0


def tables_args(b=3, rows=5, n=4):
    z = lambda *s, t=I32: torch.zeros(s, dtype=t)  # noqa: E731
    return dict(layout=layout(), lens=z(rows), new_lens=z(b), table=z(rows, 4), held=z(rows), held_out=z(rows), free_blocks=z(7), free_used=z(1, t=I64),
                free_used_out=z(1, t=I64), seq_lens=z(b), query_start_loc=z(b + 1), positions=z(n, t=I64), slot_mapping=z(n, t=I64), rows=z(b),
                block_table=z(b, 4), workspace=z(24 * b, t=U8))


MAKE = {"load": (smla.kvpack_load, load_args), "tables": (smla.smla_step_tables, tables_args)}


@pytest.mark.parametrize("which,without", [("load", ()), ("load", ("rope_out",)), ("load", ("starts",)), ("tables", ()), ("tables", ("rows", "block_table"))])
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
    *[("load", a, short) for a in ("pool", "starts")], ("load", "row_loc", lambda t: t[:1]), ("load", "block_table", lambda t: t[:1]),
    ("load", "block_table", lambda t: t[0]), ("load", "rope_out", lambda t: t[:-1]), ("load", "latent_out", lambda t: t[:, :-8]),
    ("load", "latent_out", lambda t: t.repeat_interleave(2, 1)[:, ::2]), ("load", "block_table", lambda t: t.repeat(1, 2)[:, :3]),
    *[("tables", a, short) for a in ("lens", "held", "held_out", "free_used", "free_used_out", "seq_lens", "query_start_loc", "rows", "workspace")],
    ("tables", "slot_mapping", short), ("tables", "table", lambda t: t[0]), ("tables", "block_table", lambda t: t[:-1]),
    ("tables", "table", lambda t: t.repeat(1, 2)[:, :4]), ("tables", "free_blocks", lambda t: t.repeat_interleave(2)[::2]),
])
def test_buffers_that_do_not_fit_are_refused(lib, which, arg, change):
    call, make = MAKE[which]
    a = make()
    a[arg] = change(a[arg])
    with pytest.raises(ValueError, match="|".join((arg, "contiguous"))) as e:
        call(**a)
    assert "CUDA tensors only" not in str(e.value)


@pytest.mark.parametrize("which,arg", [
    *[("load", a) for a in ("pool", "block_table", "row_loc", "starts", "latent_out", "rope_out")],
    *[("tables", a) for a in ("lens", "new_lens", "table", "held", "held_out", "free_blocks", "free_used", "free_used_out", "seq_lens", "query_start_loc",
                              "positions", "slot_mapping", "rows", "block_table", "workspace")],
])
def test_other_element_types_are_refused(lib, which, arg):
    call, make = MAKE[which]
    a = make()
    a[arg] = a[arg].to(torch.float64)
    with pytest.raises(TypeError, match=arg):
        call(**a)
