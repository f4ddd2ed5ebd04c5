"""GB300-native QSA token indexer: pool -> score -> select, behind libqsa.so.

This package is a thin ctypes binding over the C ABI declared in
``include/qsa.h``.  Every function has the C entry point's name and argument
order; device buffers are passed as CUDA torch tensors (their data pointers),
``stream`` is a torch CUDA stream (default: the current stream).  The binding
only marshals arguments: all work runs in the library's CUDA kernels.  There is
no CPU fallback: importing the package fails loudly when libqsa.so is missing
(build it with ``python sparse_attention_token_qsa_gb300/build.py``).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqsa.so")

QSA_OK = 0
QSA_ERR_INVALID_VALUE = 1
QSA_ERR_LAUNCH = 2
QSA_ERR_ROW_RANGE = 3
QSA_ERR_NONFINITE = 4
QSA_ERR_TIMEOUT = 5
QSA_ERR_TOKEN_RANGE = 6
QSA_ERR_NO_PAGES = 7

QSA_SCORE_AUTO = 0
QSA_SCORE_SIMT = 1
QSA_SCORE_TCGEN05 = 2
QSA_SCORE_STREAM = 3

HEADS, HEAD_DIM, RATIO, ROT_DIM, FUSED_WIDTH = 4, 128, 4, 64, 640

EXPORTED = ("qsa_version", "qsa_status_string", "qsa_rope_tables", "qsa_pool_blocks",
            "qsa_score_rows", "qsa_score_rows_with", "qsa_score_workspace_bytes",
            "qsa_score_rows_noalloc", "qsa_select_mask", "qsa_index_select",
            "qsa_decode_workspace_bytes", "qsa_decode_index_select", "qsa_mask_tokens",
            "qsa_gather_kv", "qsa_sparse_attn", "qsa_qk_proj", "qsa_tree_attn",
            "qsa_tree_workspace_bytes", "qsa_attn_mass", "qsa_evict_select", "qsa_cache_compact",
            "qsa_page_plan", "qsa_qkv_write", "qsa_cache8_attn", "qsa_cache8_workspace_bytes",
            "qsa_reset_status",
            "qsa_read_status", "qsa_set_wait_limit_cycles", "qsa_wait_limit_cycles")


class QsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: status {code} ({status_string(code)})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libqsa.so is not built ({LIB_PATH}); run "
                          "`python sparse_attention_token_qsa_gb300/build.py` (needs nvcc)")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, f64 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_double)
    sig = {
        "qsa_version": ([], i32),
        "qsa_status_string": ([i32], ctypes.c_char_p),
        "qsa_rope_tables": ([i32, f64, P, P], i32),
        "qsa_pool_blocks": ([P, i64, i32, i32, P, P, P, i32, f32, P, P], i32),
        "qsa_score_rows": ([P, i64, P, P, i32, i32, P, P, P, i32, f32, P, P, P, i64, P, P, i64, P],
                           i32),
        "qsa_score_rows_with": ([P, i64, P, P, i32, i32, P, P, P, i32, f32, P, P, P, i64, P, i32, P,
                                 i64, P], i32),
        "qsa_score_workspace_bytes": ([i32], i64),
        "qsa_score_rows_noalloc": ([P, i64, P, P, i32, i32, P, P, P, i32, f32, P, P, i64, P, P], i32),
        "qsa_select_mask": ([P, i64, P, i32, i32, i32, P, P, P], i32),
        "qsa_index_select": ([P, i64, i32, i32, P, P, i64, P, i32, i32, P, P, P, i32, f32, i32, P, P,
                              i64, P, P, P, i64, P], i32),
        "qsa_decode_workspace_bytes": ([i32, i32], i64),
        "qsa_decode_index_select": ([P, i64, i32, i32, P, P, i64, P, i32, i32, P, P, P, i32, f32, i32,
                                     P, P, i64, P, P, P, i64, P], i32),
        "qsa_mask_tokens": ([P, i32, i32, P, i64, P, P], i32),
        "qsa_gather_kv": ([P, P, i32, i32, P, i32, i64, i32, P, i64, P, i32, i32, P, P, i64, P, P],
                          i32),
        "qsa_sparse_attn": ([P, i64, i32, i32, i32, P, P, i32, i32, P, i32, i64, P, i64, P, i32,
                             i32, f32, P, i64, P, P], i32),
        "qsa_qk_proj": ([P, i64, P, i32, i32, i32, P, i64, P, P], i32),
        "qsa_tree_attn": ([P, i64, i32, i32, i32, P, P, i32, i32, P, i32, i64, P, P, i32, i32, P,
                           i32, f32, P, i64, P, P, P, i64, P], i32),
        "qsa_tree_workspace_bytes": ([i32, i32, i32, i32, i32], i64),
        "qsa_attn_mass": ([P, i64, i32, i32, i32, P, i32, i32, P, i32, i64, P, P, i32, i32, P, i32,
                           f32, P, P, f32, P, i64, P, P], i32),
        "qsa_evict_select": ([P, i64, i32, P, i32, i32, i32, i32, i32, i32, P, i64, P, P, P], i32),
        "qsa_cache_compact": ([P, P, i32, i32, P, i32, i64, i32, P, i64, P, i32, i32, P, P, i64,
                               i32, P, P, P, P], i32),
        "qsa_page_plan": ([P, P, i32, i32, i32, P, i32, i64, P, P, P, P, P, i32, P, P, P, P, P, P],
                          i32),
        "qsa_qkv_write": ([P, i64, i32, P, i64, P, i64, i32, i32, P, P, f32, P, P, i32, P, P, P, i32,
                           i32, P, P, P, P, i32, i32, i32, P, i32, i64, P, i64, P, P], i32),
        "qsa_cache8_attn": ([P, i64, i32, i32, i32, P, P, P, P, i32, i32, i32, P, i32, i64, P, P, i32,
                             i32, P, i32, i32, i32, f32, P, i64, P, P, P, i64, P], i32),
        "qsa_cache8_workspace_bytes": ([i32, i32, i32, i32, i32], i64),
        "qsa_reset_status": ([P, P], i32),
        "qsa_read_status": ([P, P, P, P], i32),
        "qsa_set_wait_limit_cycles": ([i64], i32),
        "qsa_wait_limit_cycles": ([], i64),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def status_string(code: int) -> str:
    return _lib.qsa_status_string(int(code)).decode()


def _dev(t: torch.Tensor | None, name: str):
    """The device-addressable pointer of a CUDA tensor, or of a pinned host tensor
    (page-locked host memory is mapped into the unified address space, so the
    kernels read and write it directly over the CPU-GPU link).  Anything else is
    refused: every computation runs in the library's kernels."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory: libqsa has no "
                         "CPU path")
    return t.data_ptr()


def _home(t, name: str) -> int:
    """The device a cache operator works on: that of its first tensor, which has to be
    the current one (the launch goes there, and the others' memory is not mapped).  None,
    which the library takes for nothing to do and refuses otherwise: the current one."""
    if t is None:
        return torch.cuda.current_device()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    d = t.get_device()
    if d < 0:
        _dev(t, name)
        return torch.cuda.current_device()
    here = torch.cuda.current_device()
    if d != here:
        raise ValueError(f"{name} is on cuda:{d}, the current device is cuda:{here}")
    return d


def _at(t, name: str, home: int):
    """_dev of a tensor that has to be on the operator's device, or pinned."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        d = t.get_device()
        if d == home:
            return t.data_ptr()
        if d >= 0:
            raise ValueError(f"{name} is on cuda:{d}, the other tensors on cuda:{home}")
    return _dev(t, name)


def _raw(stream, device: int) -> int:
    """The cudaStream_t of a torch stream (default: the device's current one, asked for
    without making a stream object: 3 us a call on a Grace core)."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _stream(stream) -> int:
    return _raw(stream, torch.cuda.current_device() if stream is None else 0)


def _check(rc: int, where: str) -> None:
    if rc != QSA_OK:
        raise QsaError(rc, where)


def qsa_version() -> int:
    return int(_lib.qsa_version())


def qsa_set_wait_limit_cycles(cycles: int) -> None:
    """The limit, in SM clock cycles, of the waits a caller may shorten (the
    streaming scorers' key-copy, operand and accumulator waits, the fused decode
    step's waits and barrier, the waits of tree attention, of attention over an 8-bit
    cache and of attention mass)."""
    _check(_lib.qsa_set_wait_limit_cycles(int(cycles)), "qsa_set_wait_limit_cycles")


def qsa_wait_limit_cycles() -> int:
    return int(_lib.qsa_wait_limit_cycles())


def qsa_rope_tables(max_pos: int, theta: float = 10000.0) -> tuple[np.ndarray, np.ndarray]:
    """Host cos/sin tables [max_pos, 64] as uint16 bf16 bit patterns."""
    cos_t = np.zeros((max_pos, ROT_DIM), np.uint16)
    sin_t = np.zeros((max_pos, ROT_DIM), np.uint16)
    _check(_lib.qsa_rope_tables(int(max_pos), float(theta),
                                cos_t.ctypes.data_as(ctypes.c_void_p),
                                sin_t.ctypes.data_as(ctypes.c_void_p)), "qsa_rope_tables")
    return cos_t, sin_t


def qsa_pool_blocks(keys, key_stride, first_block, n_blocks, k_norm_w, cos_t, sin_t, table_rows,
                    eps, block_keys, stream=None) -> None:
    _check(_lib.qsa_pool_blocks(_dev(keys, "keys"), int(key_stride), int(first_block),
                                int(n_blocks), _dev(k_norm_w, "k_norm_w"), _dev(cos_t, "cos_t"),
                                _dev(sin_t, "sin_t"), int(table_rows), float(eps),
                                _dev(block_keys, "block_keys"), _stream(stream)),
           "qsa_pool_blocks")


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


def qsa_score_workspace_bytes(n_rows: int) -> int:
    return int(_lib.qsa_score_workspace_bytes(int(n_rows)))


def new_workspace(n_rows: int, device="cuda") -> torch.Tensor:
    """A device workspace large enough for the tensor-core scorer."""
    return torch.empty(max(1, qsa_score_workspace_bytes(n_rows)), dtype=torch.uint8, device=device)


def qsa_score_rows_with(q, q_stride, pos, visible_len, n_rows, tokens, q_norm_w, cos_t, sin_t,
                        table_rows, eps, block_keys, key_base, scores, score_cols, dev_status,
                        path=QSA_SCORE_AUTO, workspace=None, stream=None) -> None:
    ws, wsb = _ws(workspace)
    _check(_lib.qsa_score_rows_with(_dev(q, "q"), int(q_stride), _dev(pos, "pos"),
                                    _dev(visible_len, "visible_len"), int(n_rows), int(tokens),
                                    _dev(q_norm_w, "q_norm_w"), _dev(cos_t, "cos_t"),
                                    _dev(sin_t, "sin_t"), int(table_rows), float(eps),
                                    _dev(block_keys, "block_keys"), _dev(key_base, "key_base"),
                                    _dev(scores, "scores"), int(score_cols),
                                    _dev(dev_status, "dev_status"), int(path), ws, int(wsb),
                                    _stream(stream)),
           "qsa_score_rows_with")


def qsa_score_rows(q, q_stride, pos, visible_len, n_rows, tokens, q_norm_w, cos_t, sin_t,
                   table_rows, eps, block_keys, key_base, scores, score_cols, dev_status,
                   workspace=None, stream=None) -> None:
    ws, wsb = _ws(workspace)
    _check(_lib.qsa_score_rows(_dev(q, "q"), int(q_stride), _dev(pos, "pos"),
                               _dev(visible_len, "visible_len"), int(n_rows), int(tokens),
                               _dev(q_norm_w, "q_norm_w"), _dev(cos_t, "cos_t"),
                               _dev(sin_t, "sin_t"), int(table_rows), float(eps),
                               _dev(block_keys, "block_keys"), _dev(key_base, "key_base"),
                               _dev(scores, "scores"), int(score_cols),
                               _dev(dev_status, "dev_status"), ws, int(wsb), _stream(stream)),
           "qsa_score_rows")


QSA_NOALLOC_MAX_ROWS = 8192


def qsa_score_rows_noalloc(q, q_stride, pos, visible_len, n_rows, tokens, q_norm_w, cos_t, sin_t,
                           table_rows, eps, block_keys, scores, score_cols, dev_status,
                           stream=None) -> None:
    """Tensor-core scoring with the library's built-in workspace (no allocation
    by anyone); at most QSA_NOALLOC_MAX_ROWS rows, calls must not overlap."""
    _check(_lib.qsa_score_rows_noalloc(_dev(q, "q"), int(q_stride), _dev(pos, "pos"),
                                       _dev(visible_len, "visible_len"), int(n_rows), int(tokens),
                                       _dev(q_norm_w, "q_norm_w"), _dev(cos_t, "cos_t"),
                                       _dev(sin_t, "sin_t"), int(table_rows), float(eps),
                                       _dev(block_keys, "block_keys"), _dev(scores, "scores"),
                                       int(score_cols), _dev(dev_status, "dev_status"),
                                       _stream(stream)),
           "qsa_score_rows_noalloc")


def qsa_select_mask(scores, score_cols, pos, n_rows, tokens, budget, mask, dev_status,
                    stream=None) -> None:
    _check(_lib.qsa_select_mask(_dev(scores, "scores"), int(score_cols), _dev(pos, "pos"),
                                int(n_rows), int(tokens), int(budget), _dev(mask, "mask"),
                                _dev(dev_status, "dev_status"), _stream(stream)),
           "qsa_select_mask")


def qsa_index_select(keys, key_stride, pool_first_block, pool_n_blocks, k_norm_w, q, q_stride, pos,
                     n_rows, tokens, q_norm_w, cos_t, sin_t, table_rows, eps, budget, block_keys,
                     scores, score_cols, mask, dev_status, workspace=None, stream=None) -> None:
    ws, wsb = _ws(workspace)
    _check(_lib.qsa_index_select(_dev(keys, "keys"), int(key_stride), int(pool_first_block),
                                 int(pool_n_blocks), _dev(k_norm_w, "k_norm_w"), _dev(q, "q"),
                                 int(q_stride), _dev(pos, "pos"), int(n_rows), int(tokens),
                                 _dev(q_norm_w, "q_norm_w"), _dev(cos_t, "cos_t"),
                                 _dev(sin_t, "sin_t"), int(table_rows), float(eps), int(budget),
                                 _dev(block_keys, "block_keys"), _dev(scores, "scores"),
                                 int(score_cols), _dev(mask, "mask"),
                                 _dev(dev_status, "dev_status"), ws, int(wsb), _stream(stream)),
           "qsa_index_select")


def qsa_decode_workspace_bytes(n_rows: int, tokens: int) -> int:
    return int(_lib.qsa_decode_workspace_bytes(int(n_rows), int(tokens)))


def new_decode_workspace(n_rows: int, tokens: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for qsa_decode_index_select (each completed call
    leaves it zero again)."""
    n = max(16, qsa_decode_workspace_bytes(n_rows, tokens))
    return torch.zeros(n, dtype=torch.uint8, device=device)


def qsa_decode_index_select(keys, key_stride, pool_first_block, pool_n_blocks, k_norm_w, q, q_stride,
                            pos, n_rows, tokens, q_norm_w, cos_t, sin_t, table_rows, eps, budget,
                            block_keys, scores, score_cols, mask, dev_status, decode_ws,
                            stream=None) -> None:
    ws, wsb = _ws(decode_ws)
    _check(_lib.qsa_decode_index_select(_dev(keys, "keys"), int(key_stride), int(pool_first_block),
                                        int(pool_n_blocks), _dev(k_norm_w, "k_norm_w"),
                                        _dev(q, "q"), int(q_stride), _dev(pos, "pos"), int(n_rows),
                                        int(tokens), _dev(q_norm_w, "q_norm_w"),
                                        _dev(cos_t, "cos_t"), _dev(sin_t, "sin_t"),
                                        int(table_rows), float(eps), int(budget),
                                        _dev(block_keys, "block_keys"), _dev(scores, "scores"),
                                        int(score_cols), _dev(mask, "mask"),
                                        _dev(dev_status, "dev_status"), ws, int(wsb),
                                        _stream(stream)),
           "qsa_decode_index_select")


def qsa_mask_tokens(mask, n_rows, tokens, sel, sel_cols, n_sel, stream=None) -> None:
    _check(_lib.qsa_mask_tokens(_dev(mask, "mask"), int(n_rows), int(tokens), _dev(sel, "sel"),
                                int(sel_cols), _dev(n_sel, "n_sel"), _stream(stream)),
           "qsa_mask_tokens")


def qsa_gather_kv(k_pool, v_pool, width, pool_pages, table, table_len, table_cols, page_size, sel,
                  sel_cols, n_sel, n_rows, max_sel, k_out, v_out, out_rows, dev_status,
                  stream=None) -> None:
    _check(_lib.qsa_gather_kv(_dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"), int(width),
                              int(pool_pages), _dev(table, "table"), int(table_len),
                              int(table_cols), int(page_size), _dev(sel, "sel"), int(sel_cols),
                              _dev(n_sel, "n_sel"), int(n_rows), int(max_sel),
                              _dev(k_out, "k_out"), _dev(v_out, "v_out"), int(out_rows),
                              _dev(dev_status, "dev_status"), _stream(stream)),
           "qsa_gather_kv")


def qsa_sparse_attn(q, q_stride, nq, nkv, head_dim, k_pool, v_pool, pool_pages, page_size, table,
                    table_len, table_cols, sel, sel_cols, n_sel, n_rows, max_sel, scale, out,
                    out_stride, dev_status, stream=None) -> None:
    _check(_lib.qsa_sparse_attn(_dev(q, "q"), int(q_stride), int(nq), int(nkv), int(head_dim),
                                _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"), int(pool_pages),
                                int(page_size), _dev(table, "table"), int(table_len),
                                int(table_cols), _dev(sel, "sel"), int(sel_cols),
                                _dev(n_sel, "n_sel"), int(n_rows), int(max_sel), float(scale),
                                _dev(out, "out"), int(out_stride), _dev(dev_status, "dev_status"),
                                _stream(stream)),
           "qsa_sparse_attn")


def qsa_qk_proj(x, x_stride, w, n_rows, hidden, out_cols, y, y_stride, dev_status,
                stream=None) -> None:
    _check(_lib.qsa_qk_proj(_dev(x, "x"), int(x_stride), _dev(w, "w"), int(n_rows), int(hidden),
                            int(out_cols), _dev(y, "y"), int(y_stride),
                            _dev(dev_status, "dev_status"), _stream(stream)),
           "qsa_qk_proj")


def qsa_tree_workspace_bytes(n_seqs: int, n_rows: int, nq: int, nkv: int, head_dim: int) -> int:
    return int(_lib.qsa_tree_workspace_bytes(int(n_seqs), int(n_rows), int(nq), int(nkv),
                                             int(head_dim)))


def new_tree_workspace(n_seqs: int, n_rows: int, nq: int, nkv: int, head_dim: int,
                       device="cuda") -> torch.Tensor:
    """A workspace for qsa_tree_attn calls of at most these n_seqs, n_rows and head_dim, and
    of at most nq / nkv query heads a KV head."""
    n = qsa_tree_workspace_bytes(n_seqs, n_rows, nq, nkv, head_dim)
    if n < 0:
        raise ValueError(f"no tree workspace for n_seqs={n_seqs}, n_rows={n_rows}, nq={nq}, nkv={nkv}, "
                         f"head_dim={head_dim}")
    return torch.empty(max(16, n), dtype=torch.uint8, device=device)


def qsa_tree_attn(q, q_stride, nq, nkv, head_dim, k_pool, v_pool, pool_pages, page_size, table,
                  table_len, table_cols, ctx_len, row_start, n_seqs, n_rows, tree_mask, mask_words,
                  scale, out, out_stride, lse, dev_status, workspace, stream=None) -> None:
    home = _home(q, "q")
    ws = _at(workspace, "workspace", home)
    wsb = 0 if ws is None else workspace.numel() * workspace.element_size()
    _check(_lib.qsa_tree_attn(_at(q, "q", home), int(q_stride), int(nq), int(nkv), int(head_dim),
                              _at(k_pool, "k_pool", home), _at(v_pool, "v_pool", home), int(pool_pages),
                              int(page_size), _at(table, "table", home), int(table_len),
                              int(table_cols), _at(ctx_len, "ctx_len", home),
                              _at(row_start, "row_start", home), int(n_seqs), int(n_rows),
                              _at(tree_mask, "tree_mask", home), int(mask_words), float(scale),
                              _at(out, "out", home), int(out_stride), _at(lse, "lse", home),
                              _at(dev_status, "dev_status", home), ws, wsb, _raw(stream, home)),
           "qsa_tree_attn")


def qsa_attn_mass(q, q_stride, nq, nkv, head_dim, k_pool, pool_pages, page_size, table, table_len,
                  table_cols, ctx_len, row_start, n_seqs, n_rows, tree_mask, mask_words, scale,
                  lse, row_weight, carry, mass, mass_cols, dev_status, stream=None) -> None:
    home = _home(q, "q")
    _check(_lib.qsa_attn_mass(_at(q, "q", home), int(q_stride), int(nq), int(nkv), int(head_dim),
                              _at(k_pool, "k_pool", home), int(pool_pages), int(page_size),
                              _at(table, "table", home), int(table_len), int(table_cols),
                              _at(ctx_len, "ctx_len", home), _at(row_start, "row_start", home), int(n_seqs),
                              int(n_rows), _at(tree_mask, "tree_mask", home), int(mask_words),
                              float(scale), _at(lse, "lse", home), _at(row_weight, "row_weight", home),
                              float(carry), _at(mass, "mass", home), int(mass_cols),
                              _at(dev_status, "dev_status", home), _raw(stream, home)),
           "qsa_attn_mass")


def qsa_evict_select(mass, mass_cols, nkv, length, n_seqs, tokens, keep, n_first, n_last, unit,
                     sel, sel_cols, n_sel, dev_status, stream=None) -> None:
    home = _home(mass, "mass")
    _check(_lib.qsa_evict_select(_at(mass, "mass", home), int(mass_cols), int(nkv),
                                 _at(length, "length", home), int(n_seqs), int(tokens), int(keep),
                                 int(n_first), int(n_last), int(unit), _at(sel, "sel", home),
                                 int(sel_cols), _at(n_sel, "n_sel", home),
                                 _at(dev_status, "dev_status", home), _raw(stream, home)),
           "qsa_evict_select")


def qsa_cache_compact(k_pool, v_pool, width, pool_pages, table, table_len, table_cols, page_size,
                      keep, keep_cols, n_keep, n_seqs, max_keep, first, mass, mass_cols, nkv,
                      block_keys, key_base, dev_status, stream=None) -> None:
    home = _home(k_pool, "k_pool")
    _check(_lib.qsa_cache_compact(_at(k_pool, "k_pool", home), _at(v_pool, "v_pool", home), int(width),
                                  int(pool_pages), _at(table, "table", home), int(table_len),
                                  int(table_cols), int(page_size), _at(keep, "keep", home),
                                  int(keep_cols), _at(n_keep, "n_keep", home), int(n_seqs),
                                  int(max_keep), _at(first, "first", home), _at(mass, "mass", home),
                                  int(mass_cols), int(nkv), _at(block_keys, "block_keys", home),
                                  _at(key_base, "key_base", home), _at(dev_status, "dev_status", home),
                                  _raw(stream, home)),
           "qsa_cache_compact")


def qsa_page_plan(ctx_len, new_rows, n_seqs, page_size, pool_pages, table, table_len, table_cols,
                  held, held_out, free_pages, n_free, n_free_out, max_rows, row_start, slot, pos,
                  row_seq, dev_status, stream=None) -> None:
    home = _home(ctx_len, "ctx_len")
    _check(_lib.qsa_page_plan(_at(ctx_len, "ctx_len", home), _at(new_rows, "new_rows", home),
                              int(n_seqs), int(page_size), int(pool_pages), _at(table, "table", home),
                              int(table_len), int(table_cols), _at(held, "held", home),
                              _at(held_out, "held_out", home), _at(free_pages, "free_pages", home),
                              _at(n_free, "n_free", home), _at(n_free_out, "n_free_out", home),
                              int(max_rows), _at(row_start, "row_start", home), _at(slot, "slot", home),
                              _at(pos, "pos", home), _at(row_seq, "row_seq", home),
                              _at(dev_status, "dev_status", home), _raw(stream, home)),
           "qsa_page_plan")


def qsa_qkv_write(q, q_stride, nq, k, k_stride, v, v_stride, nkv, head_dim, q_norm_w, k_norm_w, eps,
                  cos_t, sin_t, table_rows, pos, ctx_len, row_start, n_seqs, n_rows, k_pool, v_pool,
                  k_scale, v_scale, unit, pool_pages, page_size, table, table_len, table_cols,
                  q_out, out_stride, dev_status, stream=None) -> None:
    home = _home(q, "q")
    _check(_lib.qsa_qkv_write(_at(q, "q", home), int(q_stride), int(nq), _at(k, "k", home), int(k_stride),
                              _at(v, "v", home), int(v_stride), int(nkv), int(head_dim),
                              _at(q_norm_w, "q_norm_w", home), _at(k_norm_w, "k_norm_w", home),
                              float(eps), _at(cos_t, "cos_t", home), _at(sin_t, "sin_t", home),
                              int(table_rows), _at(pos, "pos", home), _at(ctx_len, "ctx_len", home),
                              _at(row_start, "row_start", home), int(n_seqs), int(n_rows),
                              _at(k_pool, "k_pool", home), _at(v_pool, "v_pool", home),
                              _at(k_scale, "k_scale", home), _at(v_scale, "v_scale", home), int(unit),
                              int(pool_pages), int(page_size), _at(table, "table", home), int(table_len),
                              int(table_cols), _at(q_out, "q_out", home), int(out_stride),
                              _at(dev_status, "dev_status", home), _raw(stream, home)),
           "qsa_qkv_write")


def qsa_cache8_workspace_bytes(n_seqs: int, n_rows: int, nq: int, nkv: int, head_dim: int) -> int:
    return int(_lib.qsa_cache8_workspace_bytes(int(n_seqs), int(n_rows), int(nq), int(nkv),
                                               int(head_dim)))


def new_cache8_workspace(n_seqs: int, n_rows: int, nq: int, nkv: int, head_dim: int,
                         device="cuda") -> torch.Tensor:
    """A workspace for qsa_cache8_attn calls of at most these n_seqs, n_rows and head_dim, and
    of at most nq / nkv query heads a KV head."""
    n = qsa_cache8_workspace_bytes(n_seqs, n_rows, nq, nkv, head_dim)
    if n < 0:
        raise ValueError(f"no workspace for n_seqs={n_seqs}, n_rows={n_rows}, nq={nq}, nkv={nkv}, "
                         f"head_dim={head_dim}")
    return torch.empty(max(16, n), dtype=torch.uint8, device=device)


def qsa_cache8_attn(q, q_stride, nq, nkv, head_dim, k_pool, v_pool, k_scale, v_scale, unit, pool_pages,
                    page_size, table, table_len, table_cols, ctx_len, row_start, n_seqs, n_rows,
                    tree_mask, mask_words, n_first, window, scale, out, out_stride, lse, dev_status,
                    workspace, stream=None) -> None:
    home = _home(q, "q")
    ws = _at(workspace, "workspace", home)
    wsb = 0 if ws is None else workspace.numel() * workspace.element_size()
    _check(_lib.qsa_cache8_attn(_at(q, "q", home), int(q_stride), int(nq), int(nkv), int(head_dim),
                                _at(k_pool, "k_pool", home), _at(v_pool, "v_pool", home),
                                _at(k_scale, "k_scale", home), _at(v_scale, "v_scale", home), int(unit),
                                int(pool_pages), int(page_size), _at(table, "table", home),
                                int(table_len), int(table_cols), _at(ctx_len, "ctx_len", home),
                                _at(row_start, "row_start", home), int(n_seqs), int(n_rows),
                                _at(tree_mask, "tree_mask", home), int(mask_words), int(n_first),
                                int(window), float(scale), _at(out, "out", home), int(out_stride),
                                _at(lse, "lse", home), _at(dev_status, "dev_status", home), ws, wsb,
                                _raw(stream, home)),
           "qsa_cache8_attn")


def qsa_reset_status(dev_status, stream=None) -> None:
    _check(_lib.qsa_reset_status(_dev(dev_status, "dev_status"), _stream(stream)),
           "qsa_reset_status")


def qsa_read_status(dev_status, stream=None) -> tuple[int, int]:
    code, row = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(_lib.qsa_read_status(_dev(dev_status, "dev_status"), _stream(stream),
                                ctypes.byref(code), ctypes.byref(row)), "qsa_read_status")
    return int(code.value), int(row.value)


def new_status(device="cuda") -> torch.Tensor:
    """A zeroed device status word (int32[2])."""
    return torch.zeros(2, dtype=torch.int32, device=device)
