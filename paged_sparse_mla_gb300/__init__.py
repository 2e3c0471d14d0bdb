"""Python binding of libsmla, the GB300 paged top-k sparse-MLA library.

Argument marshalling only: every function takes torch CUDA tensors on the
current device, checks their dtypes and that each holds at least the elements
the kernels read or write through it (a short buffer raises here instead of
being overrun on the GPU), and calls the same-named C entry point of
``include/smla.h`` through ctypes.  All computation happens in the library's
CUDA kernels; there is no CPU path.  If ``_build/libsmla.so`` is missing the
import of ``lib()`` raises -- build it with ``paged_sparse_mla_gb300.build_lib.build()``.
"""

import ctypes
import os

import torch

from . import build_lib

__all__ = [
    "SmlaError", "Layout", "Params", "lib", "layout_init", "workspace_size", "kvpack_store",
    "smla_index_scores", "smla_topk", "smla_attend", "smla_decode", "smla_get_last_error",
    "status_string", "version", "EXPORTED_SYMBOLS", "smla_decode_static", "smla_prefill_chunk",
    "smla_dcp_topk_merge", "smla_lse_merge", "smla_attend_hisparse", "smla_selftest_wait",
    "attend_workspace_size", "topk_workspace_size", "Rope", "make_rope", "kvpack_append", "smla_query_prep",
    "smla_attend_dense", "attend_dense_workspace_size", "kvpack_load", "smla_step_tables", "step_tables_workspace_size",
    "latent_format",
]

EXPORTED_SYMBOLS = (
    "smla_layout_init", "smla_workspace_size", "kvpack_store", "smla_index_scores", "smla_topk",
    "smla_attend", "smla_decode", "smla_get_last_error", "smla_status_string", "smla_version",
    "smla_decode_static", "smla_prefill_chunk", "smla_dcp_topk_merge", "smla_lse_merge", "smla_attend_hisparse",
    "smla_selftest_wait", "smla_attend_workspace_size", "smla_topk_workspace_size", "smla_layout_init_keys",
    "kvpack_append", "smla_query_prep", "smla_attend_dense", "smla_attend_dense_workspace_size",
    "smla_layout_init_latents", "smla_layout_latent_format", "kvpack_load", "smla_step_tables",
    "smla_step_tables_workspace_size",
)

KEY_FORMATS = {"e4m3": 0, "e2m1": 1}  # smla_key_format_t
LATENT_FORMATS = {"e4m3": 0, "e2m1": 1}  # smla_latent_format_t

STATUS = {0: "SMLA_OK", 1: "SMLA_ERR_INVALID_ARG", 2: "SMLA_ERR_UNSUPPORTED", 3: "SMLA_ERR_CUDA",
          4: "SMLA_ERR_BAD_INDEX", 5: "SMLA_ERR_TIMEOUT", 6: "SMLA_ERR_SCRATCH_LIMIT",
          7: "SMLA_ERR_RANGE", 8: "SMLA_ERR_NO_BLOCKS"}


class SmlaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


class Layout(ctypes.Structure):
    """Mirror of smla_layout_t."""
    _fields_ = [
        ("block_size", ctypes.c_int32), ("n_layers", ctypes.c_int32), ("d_latent", ctypes.c_int32),
        ("d_rope", ctypes.c_int32), ("quant_tile", ctypes.c_int32), ("d_index", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64), ("n_scales", ctypes.c_int32), ("rec_bytes", ctypes.c_int32),
        ("rec_stride", ctypes.c_int32), ("idx_key_format", ctypes.c_int32), ("rec_off", ctypes.c_int64),
        ("idx_key_off", ctypes.c_int64), ("idx_scale_off", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
        ("block_stride", ctypes.c_int64),
    ]

    @property
    def pool_bytes(self) -> int:
        return self.num_blocks * self.block_stride

    @property
    def key_bytes(self) -> int:
        """Bytes of one cached indexer key: d_index E4M3 codes, or d_index / 2 bytes of packed E2M1."""
        return self.d_index // 2 if self.idx_key_format == KEY_FORMATS["e2m1"] else self.d_index


class Params(ctypes.Structure):
    """Mirror of smla_params_t."""
    _fields_ = [("n_heads", ctypes.c_int32), ("n_idx_heads", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float)]


class Rope(ctypes.Structure):
    """Mirror of smla_rope_t (made by make_rope, which keeps the table alive in ``table``)."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("n_positions", ctypes.c_int64), ("interleaved", ctypes.c_int32),
                ("idx_interleaved", ctypes.c_int32), ("idx_rope", ctypes.c_int32)]


_LIB = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64


def lib() -> ctypes.CDLL:
    """Load libsmla.so (built in-tree).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(build_lib.LIB):
            raise RuntimeError(f"libsmla.so not built ({build_lib.LIB}); run paged_sparse_mla_gb300.build_lib.build()")
        L = ctypes.CDLL(build_lib.LIB)
        LP, PP, RP = ctypes.POINTER(Layout), ctypes.POINTER(Params), ctypes.POINTER(Rope)
        _F = ctypes.c_float
        sig = {
            "smla_layout_init": (_I, [LP, _I, _I, _I, _I, _I, _I, _I64]),
            "smla_layout_init_keys": (_I, [LP, _I, _I, _I, _I, _I, _I, _I, _I64]),
            "smla_workspace_size": (ctypes.c_size_t, [LP, PP, _I, _I]),
            "kvpack_store": (_I, [LP, _P, _I, _P, _P, _P, _P, _P, _I, _P]),
            "smla_index_scores": (_I, [LP, PP, _P, _I, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _I64, _P]),
            "smla_topk": (_I, [PP, _P, _I64, _P, _P, _I, _I, _P, _P, ctypes.c_size_t, _P]),
            "smla_topk_workspace_size": (ctypes.c_size_t, [PP, _I]),
            "smla_attend": (_I, [LP, PP, _P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _P, _P, _P, ctypes.c_size_t, _P]),
            "smla_attend_workspace_size": (ctypes.c_size_t, [LP, PP, _I]),
            "smla_decode": (_I, [LP, PP, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I,
                                 _I, _I, _P, _P, _P, _P, ctypes.c_size_t, _P]),
            "smla_decode_static": (_I, [LP, PP, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I,
                                        _I, _I, _I, _P, _P, _P, _P]),
            "smla_prefill_chunk": (_I, [LP, PP, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I,
                                        _I, _I, _I, _P, _P, _P, _P, ctypes.c_size_t, _P]),
            "smla_dcp_topk_merge": (_I, [_P, _I64, _I64, _P, _I, _I, _I, _P, _P, _P]),
            "smla_attend_hisparse": (_I, [LP, PP, _P, _I, _P, _P, _I64, _P, _P, _P, _P, _I, _P, _I, _I, _P, _P, _P]),
            "smla_lse_merge": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P]),
            "kvpack_append": (_I, [LP, _P, _I, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _F, RP, _P, _P, _I, _P]),
            "smla_query_prep": (_I, [LP, PP, RP, _P, _P, _I64, _I64, _P, _P, _I64, _I64, _P, _F, _P, _F, _P, _P, _I,
                                     _P]),
            "smla_attend_dense": (_I, [LP, PP, _P, _I, _P, _P, _P, _I, _P, _P, _I, _I, _P, _P, _P, ctypes.c_size_t,
                                       _P]),
            "smla_attend_dense_workspace_size": (ctypes.c_size_t, [LP, PP, _I]),
            "smla_layout_init_latents": (_I, [LP, _I, _I, _I, _I, _I, _I, _I, _I, _I64]),
            "smla_layout_latent_format": (_I, [LP]),
            "kvpack_load": (_I, [LP, _P, _I, _P, _I, _P, _P, _I, _I, _P, _I64, _P, _I64, _P]),
            "smla_step_tables": (_I, [LP, _P, _P, _P, _I, _P, _I64, _I, _P, _P, _P, _I64, _P, _P, _I, _P, _P, _P, _P, _P,
                                      _I, _P, ctypes.c_size_t, _P]),
            "smla_step_tables_workspace_size": (ctypes.c_size_t, [_I]),
            "smla_selftest_wait": (_I, [_I64, _P]),
            "smla_get_last_error": (_I, [_P]),
            "smla_status_string": (ctypes.c_char_p, [_I]),
            "smla_version": (_I, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _check(code: int, where: str) -> None:
    if code != 0:
        raise SmlaError(code, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libsmla takes CUDA tensors only")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError("libsmla takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _expect(t, dtype, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")


def _need(t, dtype, name, numel=0, dims=None):
    """A tensor argument's dtype, rank and minimum element count (the kernels read or write that many
    elements through its pointer).  None passes: the argument is optional or checked by the library."""
    if t is None:
        return
    _expect(t, dtype, name)
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got shape {tuple(t.shape)}")
    if t.numel() < numel:
        raise ValueError(f"{name}: needs at least {numel} elements, got shape {tuple(t.shape)}")


def _need_geometry(block_table, seq_lens, query_start_loc, batch):
    """block_table [>= batch, bt_stride], seq_lens [>= batch] and query_start_loc [>= batch + 1], int32."""
    _need(block_table, torch.int32, "block_table", dims=2)
    if block_table.shape[0] < batch:
        raise ValueError(f"block_table: needs a row per sequence ({batch}), got shape {tuple(block_table.shape)}")
    _need(seq_lens, torch.int32, "seq_lens", batch)
    _need(query_start_loc, torch.int32, "query_start_loc", batch + 1)


def _need_step(layout, params, pool, q, q_pe, q_idx, w, out, lse, topk_idx_out):
    """The per-query-token arrays of a fused step with T = q.shape[0] query tokens."""
    T, H, HI = q.shape[0], params.n_heads, params.n_idx_heads
    _need(pool, torch.uint8, "pool", layout.pool_bytes)
    _need(q, torch.bfloat16, "q", T * H * layout.d_latent)
    _need(q_pe, torch.bfloat16, "q_pe", T * H * layout.d_rope)
    _need(q_idx, torch.uint8, "q_idx", T * HI * layout.d_index)
    _need(w, torch.float32, "w", T * HI)
    _need(out, torch.bfloat16, "out", T * H * layout.d_latent)
    _need(lse, torch.float32, "lse", T * H)
    _need(topk_idx_out, torch.int32, "topk_idx_out", T * params.top_k)


def _need_new_tokens(layout, n, latent, rope, idx_k, idx_scale, slot_mapping, what="new"):
    """The n new tokens a step stores: latent, rope, indexer key and scale, slot per token."""
    _need(slot_mapping, torch.int64, "slot_mapping", n)
    _need(latent, torch.bfloat16, f"{what}_latent", n * layout.d_latent)
    _need(rope, torch.bfloat16, f"{what}_rope", n * layout.d_rope)
    _need(idx_k, torch.uint8, f"{what}_idx_k", n * layout.key_bytes)
    _need(idx_scale, torch.float32, f"{what}_idx_scale", n)


def version() -> int:
    return lib().smla_version()


def status_string(code: int) -> str:
    return lib().smla_status_string(code).decode()


def layout_init(block_size, n_layers, d_latent, d_rope, quant_tile, d_index, num_blocks, key_format="e4m3",
                latent_format="e4m3") -> Layout:
    """smla_layout_init (E4M3 indexer keys), with key_format="e2m1" smla_layout_init_keys (packed FP4 keys), or with
    latent_format="e2m1" smla_layout_init_latents (latents in 4 bits; quant_tile is 16)."""
    lay = Layout()
    if latent_format not in LATENT_FORMATS:
        raise ValueError(f"unknown latent format {latent_format!r}")
    if latent_format != "e4m3":
        if key_format not in KEY_FORMATS:
            raise ValueError(f"unknown indexer key format {key_format!r}")
        _check(lib().smla_layout_init_latents(ctypes.byref(lay), block_size, n_layers, d_latent, d_rope, quant_tile, d_index,
                                              KEY_FORMATS[key_format], LATENT_FORMATS[latent_format], num_blocks),
               "smla_layout_init_latents")
    elif key_format == "e4m3":
        _check(lib().smla_layout_init(ctypes.byref(lay), block_size, n_layers, d_latent, d_rope, quant_tile, d_index,
                                      num_blocks), "smla_layout_init")
    else:
        if key_format not in KEY_FORMATS:
            raise ValueError(f"unknown indexer key format {key_format!r}")
        _check(lib().smla_layout_init_keys(ctypes.byref(lay), block_size, n_layers, d_latent, d_rope, quant_tile,
                                           d_index, KEY_FORMATS[key_format], num_blocks), "smla_layout_init_keys")
    return lay


def latent_format(layout: Layout) -> str:
    """"e4m3" or "e2m1": the format of a layout's cached latents."""
    code = lib().smla_layout_latent_format(ctypes.byref(layout))
    if code < 0:
        raise ValueError("not a layout that layout_init made")
    return "e2m1" if code == LATENT_FORMATS["e2m1"] else "e4m3"


def make_params(n_heads, n_idx_heads, top_k, softmax_scale) -> Params:
    return Params(n_heads, n_idx_heads, top_k, softmax_scale)


def workspace_size(layout: Layout, params: Params, n_tokens: int, max_ctx: int) -> int:
    return int(lib().smla_workspace_size(ctypes.byref(layout), ctypes.byref(params), n_tokens, max_ctx))


def kvpack_store(layout, pool, layer, latent, rope, idx_k, idx_scale, slot_mapping, stream=None):
    _expect(slot_mapping, torch.int64, "slot_mapping")
    n = slot_mapping.numel()
    _need(pool, torch.uint8, "pool", layout.pool_bytes)
    _need(latent, torch.bfloat16, "latent", n * layout.d_latent)
    _need(rope, torch.bfloat16, "rope", n * layout.d_rope)
    _need(idx_k, torch.uint8, "idx_k", n * layout.key_bytes)
    _need(idx_scale, torch.float32, "idx_scale", n)
    _check(lib().kvpack_store(ctypes.byref(layout), _ptr(pool), layer, _ptr(latent), _ptr(rope), _ptr(idx_k),
                              _ptr(idx_scale), _ptr(slot_mapping), n, _stream(stream)), "kvpack_store")


def smla_index_scores(layout, params, pool, layer, q_idx, w, block_table, seq_lens, query_start_loc, max_q,
                      max_ctx, scores, stream=None):
    n_tokens = q_idx.shape[0]
    _need(pool, torch.uint8, "pool", layout.pool_bytes)
    _need(q_idx, torch.uint8, "q_idx", n_tokens * params.n_idx_heads * layout.d_index)
    _need(w, torch.float32, "w", n_tokens * params.n_idx_heads)
    _need_geometry(block_table, seq_lens, query_start_loc, seq_lens.numel())
    _need(scores, torch.float32, "scores", dims=2)
    if scores.shape[0] < n_tokens:
        raise ValueError(f"scores: needs a row per query token ({n_tokens}), got shape {tuple(scores.shape)}")
    _check(lib().smla_index_scores(ctypes.byref(layout), ctypes.byref(params), _ptr(pool), layer, _ptr(q_idx),
                                   _ptr(w), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
                                   _ptr(query_start_loc), seq_lens.numel(), n_tokens, max_q, max_ctx, _ptr(scores),
                                   scores.stride(0), _stream(stream)), "smla_index_scores")


def topk_workspace_size(params, n_tokens) -> int:
    return int(lib().smla_topk_workspace_size(ctypes.byref(params), n_tokens))


def smla_topk(params, scores, seq_lens, query_start_loc, topk_idx, stream=None, workspace=None):
    """Exact top-k per row.  `workspace` (uint8 device tensor of at least topk_workspace_size(...)
    bytes, optional) lets a small batch of long rows split each row over CTAs."""
    _need(topk_idx, torch.int32, "topk_idx", dims=2)
    rows = topk_idx.shape[0]
    if topk_idx.shape[1] != params.top_k:
        raise ValueError(f"topk_idx: rows of top_k = {params.top_k} entries expected, got shape {tuple(topk_idx.shape)}")
    _need(scores, torch.float32, "scores", dims=2)
    if scores.shape[0] < rows:
        raise ValueError(f"scores: needs a row per top-k row ({rows}), got shape {tuple(scores.shape)}")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(query_start_loc, torch.int32, "query_start_loc", seq_lens.numel() + 1)
    _need(workspace, torch.uint8, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().smla_topk(ctypes.byref(params), _ptr(scores), scores.stride(0), _ptr(seq_lens),
                           _ptr(query_start_loc), seq_lens.numel(), topk_idx.shape[0], _ptr(topk_idx),
                           _ptr(workspace), ws_bytes, _stream(stream)), "smla_topk")


def attend_workspace_size(layout, params, n_tokens) -> int:
    return int(lib().smla_attend_workspace_size(ctypes.byref(layout), ctypes.byref(params), n_tokens))


def _need_attend(layout, params, pool, q, q_pe, topk_idx, block_table, query_start_loc, out, lse):
    """Arrays of smla_attend with T = q.shape[0] query tokens and B = query_start_loc.numel() - 1 sequences."""
    T, H = q.shape[0], params.n_heads
    _need(pool, torch.uint8, "pool", layout.pool_bytes)
    _need(q, torch.bfloat16, "q", T * H * layout.d_latent)
    _need(q_pe, torch.bfloat16, "q_pe", T * H * layout.d_rope)
    _need(topk_idx, torch.int32, "topk_idx", T * params.top_k)
    _need(query_start_loc, torch.int32, "query_start_loc", 1)
    batch = query_start_loc.numel() - 1
    _need(block_table, torch.int32, "block_table", dims=2)
    if block_table.shape[0] < batch:
        raise ValueError(f"block_table: needs a row per sequence ({batch}), got shape {tuple(block_table.shape)}")
    _need(out, torch.bfloat16, "out", T * H * layout.d_latent)
    _need(lse, torch.float32, "lse", T * H)


def smla_attend(layout, params, pool, layer, q, q_pe, topk_idx, block_table, query_start_loc, out, lse,
                stream=None, workspace=None):
    """Latent attention over the selected positions.  `workspace` (uint8 device tensor of at least
    attend_workspace_size(...) bytes, optional) lets a small batch split each token over CTAs."""
    _need_attend(layout, params, pool, q, q_pe, topk_idx, block_table, query_start_loc, out, lse)
    _need(workspace, torch.uint8, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().smla_attend(ctypes.byref(layout), ctypes.byref(params), _ptr(pool), layer, _ptr(q), _ptr(q_pe),
                             _ptr(topk_idx), _ptr(block_table), block_table.shape[1], _ptr(query_start_loc),
                             query_start_loc.numel() - 1, q.shape[0], _ptr(out), _ptr(lse), _ptr(workspace),
                             ws_bytes, _stream(stream)),
           "smla_attend")


def smla_attend_hisparse(layout, params, pool, layer, host_records, host_block_map, q, q_pe, topk_idx, block_table,
                         query_start_loc, out, lse, stream=None):
    """smla_attend with the records of mapped blocks read from a pinned host buffer (host_records, uint8)."""
    _need_attend(layout, params, pool, q, q_pe, topk_idx, block_table, query_start_loc, out, lse)
    _need(host_block_map, torch.int32, "host_block_map", layout.num_blocks)
    _expect(host_records, torch.uint8, "host_records")
    if host_records.is_cuda or not host_records.is_pinned():
        raise ValueError("host_records must be pinned host memory")
    if not host_block_map.is_cuda:
        raise ValueError("host_block_map must be a CUDA tensor")
    rec_bytes = layout.n_layers * layout.block_size * layout.rec_stride
    n_host = host_records.numel() // rec_bytes
    _check(lib().smla_attend_hisparse(ctypes.byref(layout), ctypes.byref(params), _ptr(pool), layer,
                                      ctypes.c_void_p(host_records.data_ptr()), _ptr(host_block_map), n_host, _ptr(q),
                                      _ptr(q_pe), _ptr(topk_idx), _ptr(block_table), block_table.shape[1],
                                      _ptr(query_start_loc), query_start_loc.numel() - 1, q.shape[0], _ptr(out),
                                      _ptr(lse), _stream(stream)), "smla_attend_hisparse")


def smla_decode(layout, params, pool, layer, new_latent, new_rope, new_idx_k, new_idx_scale, slot_mapping, q, q_pe,
                q_idx, w, block_table, seq_lens, query_start_loc, max_q, max_ctx, out, lse, workspace,
                topk_idx_out=None, stream=None):
    T = q.shape[0]
    _need_step(layout, params, pool, q, q_pe, q_idx, w, out, lse, topk_idx_out)
    _need_geometry(block_table, seq_lens, query_start_loc, seq_lens.numel())
    if slot_mapping is not None:
        _need_new_tokens(layout, T, new_latent, new_rope, new_idx_k, new_idx_scale, slot_mapping)
    _need(workspace, torch.uint8, "workspace")
    _check(lib().smla_decode(ctypes.byref(layout), ctypes.byref(params), _ptr(pool), layer, _ptr(new_latent),
                             _ptr(new_rope), _ptr(new_idx_k), _ptr(new_idx_scale), _ptr(slot_mapping), _ptr(q),
                             _ptr(q_pe), _ptr(q_idx), _ptr(w), _ptr(block_table), block_table.shape[1],
                             _ptr(seq_lens), _ptr(query_start_loc), seq_lens.numel(), q.shape[0], max_q, max_ctx,
                             _ptr(out), _ptr(lse), _ptr(topk_idx_out), _ptr(workspace), workspace.numel(),
                             _stream(stream)), "smla_decode")


def smla_decode_static(layout, params, pool, layer, new_latent, new_rope, new_idx_k, new_idx_scale, slot_mapping,
                       q, q_pe, q_idx, w, block_table, seq_lens, query_start_loc, max_q, max_ctx, out, lse,
                       topk_idx_out=None, stream=None):
    """smla_decode without a workspace argument, for callers that cannot allocate device memory.

    The scores and top-k scratch live in the library's static 64 MiB device
    array; calls share it, so calls that overlap on the GPU race on it.
    """
    T = q.shape[0]
    _need_step(layout, params, pool, q, q_pe, q_idx, w, out, lse, topk_idx_out)
    _need_geometry(block_table, seq_lens, query_start_loc, seq_lens.numel())
    if slot_mapping is not None:
        _need_new_tokens(layout, T, new_latent, new_rope, new_idx_k, new_idx_scale, slot_mapping)
    _check(lib().smla_decode_static(ctypes.byref(layout), ctypes.byref(params), _ptr(pool), layer, _ptr(new_latent),
                                    _ptr(new_rope), _ptr(new_idx_k), _ptr(new_idx_scale), _ptr(slot_mapping), _ptr(q),
                                    _ptr(q_pe), _ptr(q_idx), _ptr(w), _ptr(block_table), block_table.shape[1],
                                    _ptr(seq_lens), _ptr(query_start_loc), seq_lens.numel(), q.shape[0], max_q,
                                    max_ctx, _ptr(out), _ptr(lse), _ptr(topk_idx_out), _stream(stream)),
           "smla_decode_static")


def smla_prefill_chunk(layout, params, pool, layer, chunk_latent, chunk_rope, chunk_idx_k, chunk_idx_scale,
                       slot_mapping, q, q_pe, q_idx, w, block_table, seq_lens, query_start_loc, chunk_len, max_ctx,
                       out, lse, workspace, topk_idx_out=None, stream=None):
    """A prefill chunk per sequence (its keys stored first), causal within the chunk."""
    T = q.shape[0]
    _need_step(layout, params, pool, q, q_pe, q_idx, w, out, lse, topk_idx_out)
    _need_geometry(block_table, seq_lens, query_start_loc, seq_lens.numel())
    _need_new_tokens(layout, T, chunk_latent, chunk_rope, chunk_idx_k, chunk_idx_scale, slot_mapping, "chunk")
    _need(workspace, torch.uint8, "workspace")
    _check(lib().smla_prefill_chunk(ctypes.byref(layout), ctypes.byref(params), _ptr(pool), layer, _ptr(chunk_latent),
                                    _ptr(chunk_rope), _ptr(chunk_idx_k), _ptr(chunk_idx_scale), _ptr(slot_mapping),
                                    _ptr(q), _ptr(q_pe), _ptr(q_idx), _ptr(w), _ptr(block_table), block_table.shape[1],
                                    _ptr(seq_lens), _ptr(query_start_loc), seq_lens.numel(), q.shape[0], chunk_len,
                                    max_ctx, _ptr(out), _ptr(lse), _ptr(topk_idx_out), _ptr(workspace),
                                    workspace.numel(), _stream(stream)), "smla_prefill_chunk")


def smla_dcp_topk_merge(shard_scores, shard_topk, shard_sel, merged=None, stream=None):
    """Candidate merge over token shards.  shard_scores [N, T, stride] fp32, shard_topk / shard_sel [N, T, k] int32."""
    _need(shard_topk, torch.int32, "shard_topk", dims=3)
    n, t, k = shard_topk.shape
    _need(shard_scores, torch.float32, "shard_scores", dims=3)
    if shard_scores.shape[0] < n or shard_scores.shape[1] < t:
        raise ValueError(f"shard_scores: needs [{n}, {t}, >= visible] for shard_topk {tuple(shard_topk.shape)}, "
                         f"got {tuple(shard_scores.shape)}")
    _need(shard_sel, torch.int32, "shard_sel", n * t * k)
    _need(merged, torch.int32, "merged", t * k)
    _check(lib().smla_dcp_topk_merge(_ptr(shard_scores), shard_scores.stride(0), shard_scores.stride(1),
                                     _ptr(shard_topk), n, t, k, _ptr(shard_sel), _ptr(merged), _stream(stream)),
           "smla_dcp_topk_merge")


def smla_lse_merge(parts_out, parts_lse, out, lse, stream=None):
    """LSE merge of partial outputs.  parts_out [N, T, H, D] bf16, parts_lse [N, T, H] fp32."""
    _need(parts_out, torch.bfloat16, "parts_out", dims=4)
    n, t, h, d = parts_out.shape
    _need(parts_lse, torch.float32, "parts_lse", n * t * h)
    _need(out, torch.bfloat16, "out", t * h * d)
    _need(lse, torch.float32, "lse", t * h)
    _check(lib().smla_lse_merge(_ptr(parts_out), _ptr(parts_lse), n, t, h, d, _ptr(out), _ptr(lse), _stream(stream)),
           "smla_lse_merge")


def make_rope(cos_sin, interleaved, idx_interleaved=False, idx_rope=True) -> Rope:
    """Rotation table of kvpack_append and smla_query_prep: cos_sin fp32 [n_positions, d_rope], cosines
    of a position's d_rope / 2 angles, then their sines."""
    _need(cos_sin, torch.float32, "cos_sin", dims=2)
    if not cos_sin.is_contiguous():
        raise ValueError("cos_sin: a contiguous table expected")
    rope = Rope(cos_sin.data_ptr(), cos_sin.shape[0], int(interleaved), int(idx_interleaved), int(idx_rope))
    rope.table = cos_sin
    return rope


# The calls below take a few microseconds of GPU time for a decode step, so their checks are kept lean: what a
# tensor must hold is checked argument by argument (_take), where it lies is checked once for the whole call
# (_on_device).

_BF16, _F32, _U8, _I32, _I64T = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64


def _take(t, dtype, name, n):
    """Address of a contiguous tensor of `dtype` with at least n elements; None passes."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() < n:
        raise ValueError(f"{name}: needs at least {n} elements, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: libsmla takes contiguous tensors only")
    return t.data_ptr()


def _take_rows(t, name, shape):
    """(address, element strides of the leading axes) of a bf16 tensor of exactly `shape` whose last axis is
    contiguous; its leading axes may have any stride.  None passes."""
    if t is None:
        return None, (0,) * (len(shape) - 1)
    if t.dtype is not _BF16:
        raise TypeError(f"{name}: expected {_BF16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    strides = t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: its last axis has to be contiguous, got strides {strides}")
    return t.data_ptr(), strides[:-1]


def _on_device(tensors, stream):
    """The stream's handle, after checking that every tensor lies on the current device."""
    dev = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d < 0:
                raise ValueError("libsmla takes CUDA tensors only")
            if dev < 0:
                dev = torch.cuda.current_device()
            if d != dev:
                raise ValueError(f"tensor on cuda:{d}, but the current device is cuda:{dev}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _rope_args(layout, rope, positions, n):
    """(descriptor, address of the positions) of an optional rotation whose table fits the layout."""
    if rope is None:
        return None, None
    if rope.table.shape[1] != layout.d_rope:
        raise ValueError(f"cos_sin: rows of d_rope = {layout.d_rope} expected, got shape {tuple(rope.table.shape)}")
    if positions is None:
        raise ValueError("positions: needed with a rotation")
    return ctypes.byref(rope), _take(positions, _I64T, "positions", n)


def kvpack_append(layout, pool, layer, latent, rope_key, idx_k, rope, positions, slot_mapping, latent_norm=None,
                  idx_norm=None, idx_bias=None, eps=1e-6, stream=None):
    """Norm, rotate, quantise and store new tokens.  latent [n, d_latent], rope_key [n, d_rope] and idx_k
    [n, d_index] (or None) are bf16 with contiguous rows any distance apart; rope is a Rope or None."""
    n = slot_mapping.numel()
    d_latent, d_rope, d_index = layout.d_latent, layout.d_rope, layout.d_index
    slots = _take(slot_mapping, _I64T, "slot_mapping", n)
    pl = _take(pool, _U8, "pool", layout.pool_bytes)
    ln = _take(latent_norm, _F32, "latent_norm", d_latent)
    kn = _take(idx_norm, _F32, "idx_norm", d_index)
    kb = _take(idx_bias, _F32, "idx_bias", d_index)
    rp, pos = _rope_args(layout, rope, positions, n)
    lat, (lat_s,) = _take_rows(latent, "latent", (n, d_latent))
    rk, (rk_s,) = _take_rows(rope_key if d_rope else None, "rope_key", (n, d_rope))
    ik, (ik_s,) = _take_rows(idx_k, "idx_k", (n, d_index))
    st = _on_device((pool, latent, rope_key if d_rope else None, idx_k, slot_mapping, latent_norm, idx_norm, idx_bias,
                     None if rp is None else rope.table, None if rp is None else positions), stream)
    _check((_LIB or lib()).kvpack_append(ctypes.byref(layout), pl, layer, lat, lat_s, rk, rk_s, ik, ik_s, ln, kn, kb,
                                         eps, rp, pos, slots, n, st), "kvpack_append")


def smla_query_prep(layout, params, rope, positions, q_pe=None, q_pe_out=None, q_idx=None, w=None, w_scale=1.0,
                    q_idx_out=None, w_out=None, idx_norm=None, eps=1e-6, stream=None):
    """Rotate q_pe [T, n_heads, d_rope]; norm, rotate and quantise q_idx [T, n_idx_heads, d_index] and fold
    each head's scale into w [T, n_idx_heads].  Either may be None; both may be slices of wider tensors."""
    if q_pe is None and q_idx is None:
        raise ValueError("smla_query_prep: needs q_pe or q_idx")
    n = (q_idx if q_pe is None else q_pe).shape[0]
    H, HI, d_rope, d_index = params.n_heads, params.n_idx_heads, layout.d_rope, layout.d_index
    rp, pos = _rope_args(layout, rope, positions, n)
    pe, (pe_t, pe_h) = _take_rows(q_pe, "q_pe", (n, H, d_rope))
    ix, (ix_t, ix_h) = _take_rows(q_idx, "q_idx", (n, HI, d_index))
    po = wp = co = wo = None
    if q_pe is not None:
        if q_pe_out is None:
            raise ValueError("q_pe_out: needed with q_pe")
        po = _take(q_pe_out, _BF16, "q_pe_out", n * H * d_rope)
    if q_idx is not None:
        if w is None or q_idx_out is None or w_out is None:
            raise ValueError("w, q_idx_out and w_out: needed with q_idx")
        wp = _take(w, _F32, "w", n * HI)
        co = _take(q_idx_out, _U8, "q_idx_out", n * HI * d_index)
        wo = _take(w_out, _F32, "w_out", n * HI)
    kn = _take(idx_norm, _F32, "idx_norm", d_index)
    st = _on_device((q_pe, q_idx, q_pe_out, q_idx_out, w, w_out, idx_norm, None if rp is None else rope.table,
                     None if rp is None else positions), stream)
    _check((_LIB or lib()).smla_query_prep(ctypes.byref(layout), ctypes.byref(params), rp, pos, pe, pe_t, pe_h, po, ix,
                                           ix_t, ix_h, kn, eps, wp, w_scale, co, wo, n, st), "smla_query_prep")


def attend_dense_workspace_size(layout, params, n_tokens) -> int:
    return int(lib().smla_attend_dense_workspace_size(ctypes.byref(layout), ctypes.byref(params), n_tokens))


def smla_attend_dense(layout, params, pool, layer, q, q_pe, block_table, seq_lens, query_start_loc, out, lse=None,
                      workspace=None, stream=None):
    """Latent attention over the whole visible context.  `lse` is optional; `workspace` (uint8 device tensor
    of at least attend_dense_workspace_size(...) bytes, optional) lets long contexts split over the SMs."""
    T = q.shape[0]
    rows = T * params.n_heads
    batch = seq_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] < batch:
        raise ValueError(f"block_table: needs a row per sequence ({batch}), got shape {tuple(block_table.shape)}")
    pl = _take(pool, _U8, "pool", layout.pool_bytes)
    qa = _take(q, _BF16, "q", rows * layout.d_latent)
    pe = _take(q_pe, _BF16, "q_pe", rows * layout.d_rope)
    bt = _take(block_table, _I32, "block_table", 0)
    sl = _take(seq_lens, _I32, "seq_lens", batch)
    qs = _take(query_start_loc, _I32, "query_start_loc", batch + 1)
    oa = _take(out, _BF16, "out", rows * layout.d_latent)
    la = _take(lse, _F32, "lse", rows)
    ws = _take(workspace, _U8, "workspace", 0)
    st = _on_device((q, pool, q_pe, block_table, seq_lens, query_start_loc, out, lse, workspace), stream)
    _check((_LIB or lib()).smla_attend_dense(ctypes.byref(layout), ctypes.byref(params), pl, layer, qa, pe, bt,
                                             block_table.shape[1], sl, qs, batch, T, oa, la, ws,
                                             0 if workspace is None else workspace.numel(), st), "smla_attend_dense")


def kvpack_load(layout, pool, layer, block_table, row_loc, latent_out, rope_out=None, starts=None, stream=None):
    """Positions starts[b] .. of each sequence (starts None: from 0 on) as bf16 rows row_loc[b] .. row_loc[b + 1] - 1 of
    latent_out [n, d_latent] and rope_out [n, d_rope] (or None), whose rows may be any distance apart."""
    n = latent_out.shape[0]
    if row_loc.numel() < 2:
        raise ValueError(f"row_loc: needs at least 2 elements, got shape {tuple(row_loc.shape)}")
    batch = row_loc.numel() - 1
    if block_table.dim() != 2 or block_table.shape[0] < batch:
        raise ValueError(f"block_table: needs a row per sequence ({batch}), got shape {tuple(block_table.shape)}")
    pl = _take(pool, _U8, "pool", layout.pool_bytes)
    bt = _take(block_table, _I32, "block_table", 0)
    rl = _take(row_loc, _I32, "row_loc", 2)
    sa = _take(starts, _I32, "starts", batch)
    lo, (ls,) = _take_rows(latent_out, "latent_out", (n, layout.d_latent))
    if layout.d_rope == 0:
        rope_out = None
    ro, (rs,) = _take_rows(rope_out, "rope_out", (n, layout.d_rope))
    if n == 1:  # the distance of a single row's rows is whatever it was sliced from, or left over
        ls, rs = max(ls, layout.d_latent), max(rs, layout.d_rope)
    st = _on_device((latent_out, pool, block_table, row_loc, starts, rope_out), stream)
    _check((_LIB or lib()).kvpack_load(ctypes.byref(layout), pl, layer, bt, block_table.shape[1], sa, rl, batch, n, lo, ls, ro, rs, st),
           "kvpack_load")


def step_tables_workspace_size(batch) -> int:
    return int(lib().smla_step_tables_workspace_size(batch))


def smla_step_tables(layout, lens, new_lens, table, held, held_out, free_blocks, free_used, free_used_out, seq_lens,
                     query_start_loc, positions, slot_mapping, rows=None, block_table=None, workspace=None, stream=None):
    """Block tables, positions and slots of a step whose entry i adds new_lens[i] tokens to row rows[i] (None: row i) of
    the persistent table [n_rows, blocks].  lens, held and held_out have an element per row, free_used and
    free_used_out are int64 tensors of one element; workspace: uint8, step_tables_workspace_size(batch) bytes."""
    batch = new_lens.numel()
    if table.dim() != 2:
        raise ValueError(f"table: expected 2 dimensions, got shape {tuple(table.shape)}")
    n_rows, stride = table.shape
    if block_table is not None and (block_table.dim() != 2 or block_table.shape[0] < batch):
        raise ValueError(f"block_table: needs a row per entry ({batch}), got shape {tuple(block_table.shape)}")
    if workspace is None or workspace.numel() < 24 * batch:
        raise ValueError("workspace: needs step_tables_workspace_size(batch) bytes")
    n = positions.numel()
    args = (_take(rows, _I32, "rows", batch), _take(lens, _I32, "lens", n_rows), _take(new_lens, _I32, "new_lens", batch), batch,
            _take(table, _I32, "table", 0), n_rows, stride, _take(held, _I32, "held", n_rows),
            _take(held_out, _I32, "held_out", n_rows), _take(free_blocks, _I32, "free_blocks", 0), free_blocks.numel(),
            _take(free_used, _I64T, "free_used", 1), _take(free_used_out, _I64T, "free_used_out", 1), n,
            _take(seq_lens, _I32, "seq_lens", batch), _take(query_start_loc, _I32, "query_start_loc", batch + 1),
            _take(positions, _I64T, "positions", n), _take(slot_mapping, _I64T, "slot_mapping", n),
            _take(block_table, _I32, "block_table", 0), 0 if block_table is None else block_table.shape[1],
            _take(workspace, _U8, "workspace", 0), workspace.numel())
    st = _on_device((lens, rows, new_lens, table, held, held_out, free_blocks, free_used, free_used_out, seq_lens,
                     query_start_loc, positions, slot_mapping, block_table, workspace), stream)
    _check((_LIB or lib()).smla_step_tables(ctypes.byref(layout), *args, st), "smla_step_tables")


def smla_selftest_wait(limit_ns, stream=None):
    """Launch the bounded-wait self-check (one wait never completes; it gives up after limit_ns)."""
    _check(lib().smla_selftest_wait(int(limit_ns), _stream(stream)), "smla_selftest_wait")


def smla_get_last_error(stream=None) -> int:
    return int(lib().smla_get_last_error(_stream(stream)))
