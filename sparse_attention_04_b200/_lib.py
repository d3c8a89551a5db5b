"""ctypes binding of libdsa.so: argument marshalling only.

Every function below takes torch CUDA tensors, passes their device pointers
and the current CUDA stream to the C ABI of the same name (include/dsa.h) and
raises DSAError on a non-zero status.  No arithmetic of the method happens
here; there is no CPU fallback.  If libdsa.so is missing the import fails.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa.so")

DSA_BF16, DSA_E4M3, DSA_F32 = 0, 1, 2
STATUS = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED", 3: "DSA_ERR_WORKSPACE",
          4: "DSA_ERR_CUDA", 5: "DSA_ERR_TIMEOUT", 6: "DSA_ERR_BAD_INDEX", 7: "DSA_ERR_BAD_OFFSETS"}

EXPORTS = ("dsa_status_string", "dsa_version", "dsa_indexer_scores", "dsa_topk",
           "dsa_sparse_mla_workspace_size", "dsa_sparse_mla", "dsa_decode_step_workspace_size",
           "dsa_decode_step", "dsa_decode_step_workspace_layout", "dsa_sparse_mla_noalloc",
           "dsa_decode_step_launches", "dsa_cache_append", "dsa_quantize_queries", "dsa_indexer_prestage",
           "dsa_copy_host_to_device", "dsa_copy_device_to_host", "dsa_debug_stall_attention",
           "dsa_paged_append", "dsa_paged_mla_workspace_size", "dsa_paged_mla", "dsa_paged_weights",
           "dsa_evict_plan", "dsa_paged_move")


class DSAError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)}")
        self.code = code


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: run `python -m sparse_attention_04_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sig = {
        "dsa_status_string": ([I], ctypes.c_char_p),
        "dsa_version": ([], I),
        "dsa_indexer_scores": ([P, P, P, P, I, P, I, I, I64, P, I64, P, P], I),
        "dsa_topk": ([P, I64, P, I, I, I, P, P, P], I),
        "dsa_sparse_mla_workspace_size": ([I, I, I, I], SZ),
        "dsa_sparse_mla": ([P, P, P, P, I, I, I, I, F, I64, P, I, P, P, SZ, P, P], I),
        "dsa_decode_step_workspace_size": ([I, I, I, I], SZ),
        "dsa_decode_step": ([P, P, P, P, I, P, P, P, I, I, I64, I, I, F, P, I, P, P, SZ, P, P], I),
        "dsa_decode_step_workspace_layout": ([I, I, I, I, P, P, P, P], I),
        "dsa_sparse_mla_noalloc": ([P, P, P, P, I, I, I, I, F, I64, P, I, P, P, P], I),
        "dsa_decode_step_launches": ([I, I, I, I], I),
        "dsa_cache_append": ([P, P, P, I, I, I, P, P, P, I64, P, P], I),
        "dsa_quantize_queries": ([P, P, I, P, P, P], I),
        "dsa_indexer_prestage": ([P, P, I, I, P, P, I, P, P, P], I),
        "dsa_copy_host_to_device": ([P, P, SZ, P], I),
        "dsa_copy_device_to_host": ([P, P, SZ, P], I),
        "dsa_debug_stall_attention": ([I, ctypes.c_uint64], I),
        "dsa_paged_append": ([P, P, P, I64, I, I, I, I, I64, P, P, P, P, I64, P, P], I),
        "dsa_paged_mla_workspace_size": ([I, I, I], SZ),
        "dsa_paged_mla": ([P, P, P, I64, I, P, I, I, I, I, I64, F, P, I, P, P, SZ, P, P], I),
        "dsa_paged_weights": ([P, P, P, I64, I, P, P, I, I, I, I, I64, F, F, P, P, I64, P, P], I),
        "dsa_evict_plan": ([P, P, P, P, I, I64, I, I, P, P, P, P, I64, P, P], I),
        "dsa_paged_move": ([P, P, I64, I, I, I64, P, P, P, I64, I, P, P, I64, P, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


lib = _load()


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise DSAError(1, "tensor is not on a CUDA device")
    if not t.is_contiguous():
        raise DSAError(1, "tensor is not contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, what: str):
    if rc != 0:
        raise DSAError(rc, what)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DSA_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return DSA_E4M3
    raise DSAError(1, f"unsupported indexer dtype {t.dtype}")


def status_string(code: int) -> str:
    return lib.dsa_status_string(code).decode()


def indexer_scores(q_idx, w, k_idx, k_scale, offsets, B, T, kv_rows, scores, ld, status=None, stream=None):
    """dsa_indexer_scores: writes fp32 scores[(b*T+t)*ld + s]."""
    _check(lib.dsa_indexer_scores(_p(q_idx), _p(w), _p(k_idx), _p(k_scale), _dtype_code(q_idx), _p(offsets),
                                  B, T, kv_rows, _p(scores), ld, _p(status), _stream(stream)),
           "dsa_indexer_scores")


def topk(scores, ld, offsets, B, T, k, indices, status=None, stream=None):
    """dsa_topk: int32 indices [B*T, k], ascending, -1 padded."""
    _check(lib.dsa_topk(_p(scores), ld, _p(offsets), B, T, k, _p(indices), _p(status), _stream(stream)),
           "dsa_topk")


def sparse_mla_workspace_size(B, T, H, k) -> int:
    return int(lib.dsa_sparse_mla_workspace_size(B, T, H, k))


def sparse_mla(q, kv, offsets, indices, B, T, H, k, scale, kv_rows, out, lse=None, workspace=None,
               status=None, stream=None):
    """dsa_sparse_mla: out [B,T,H,512] (bf16 or fp32 by out's dtype)."""
    out_code = DSA_BF16 if out.dtype == torch.bfloat16 else DSA_F32
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.dsa_sparse_mla(_p(q), _p(kv), _p(offsets), _p(indices), B, T, H, k, float(scale), kv_rows,
                              _p(out), out_code, _p(lse), _p(workspace), ws_bytes, _p(status),
                              _stream(stream)),
           "dsa_sparse_mla")


def sparse_mla_noalloc(q, kv, offsets, indices, B, T, H, k, scale, kv_rows, out, lse=None, status=None,
                       stream=None):
    """dsa_sparse_mla_noalloc: dsa_sparse_mla with the library's built-in scratch (no workspace)."""
    out_code = DSA_BF16 if out.dtype == torch.bfloat16 else DSA_F32
    _check(lib.dsa_sparse_mla_noalloc(_p(q), _p(kv), _p(offsets), _p(indices), B, T, H, k, float(scale), kv_rows,
                                      _p(out), out_code, _p(lse), _p(status), _stream(stream)),
           "dsa_sparse_mla_noalloc")


def cache_append(k_new, kv_new, offsets, B, T, k_cache, k_scale, kv_cache, kv_rows, status=None, stream=None):
    """dsa_cache_append: the newest T tokens' key (e4m3-quantised when the key
    cache is uint8) and latent rows into each sequence's last T cache rows."""
    code = DSA_E4M3 if (k_cache is not None and k_cache.dtype in (torch.uint8, torch.float8_e4m3fn)) else DSA_BF16
    _check(lib.dsa_cache_append(_p(k_new), _p(kv_new), _p(offsets), B, T, code, _p(k_cache), _p(k_scale),
                                _p(kv_cache), kv_rows, _p(status), _stream(stream)), "dsa_cache_append")


def indexer_prestage(x, pos, rope_cos, rope_sin, y=None, status=None, stream=None):
    """dsa_indexer_prestage on x [n_rows, V, 128] bf16 (V vectors per row share
    pos[row]): rotary embedding of the rope half, then the Hadamard rotation,
    into y (a new tensor unless given; y may be x)."""
    if x.dim() != 3 or x.shape[-1] != 128:
        raise DSAError(1, "indexer_prestage: x must be [n_rows, V, 128]")
    if y is None:
        y = torch.empty_like(x)
    _check(lib.dsa_indexer_prestage(_p(x), _p(pos), x.shape[0], x.shape[1], _p(rope_cos), _p(rope_sin),
                                    rope_cos.shape[0], _p(y), _p(status), _stream(stream)), "dsa_indexer_prestage")
    return y


def quantize_queries(q_idx, w, n_rows, q_e4m3, w_out, stream=None):
    """dsa_quantize_queries: e4m3 codes of q_idx and w_out = w * q_scale."""
    _check(lib.dsa_quantize_queries(_p(q_idx), _p(w), n_rows, _p(q_e4m3), _p(w_out), _stream(stream)),
           "dsa_quantize_queries")


def _host_p(t: torch.Tensor):
    if t.is_cuda or not t.is_contiguous():
        raise DSAError(1, "host buffer must be a contiguous CPU tensor")
    return ctypes.c_void_p(t.data_ptr())


def copy_host_to_device(dst, src_host, stream=None):
    """dsa_copy_host_to_device: dst (CUDA) <- src_host (pinned CPU), by a kernel."""
    n = src_host.numel() * src_host.element_size()
    if dst.numel() * dst.element_size() != n:
        raise DSAError(1, "copy_host_to_device: sizes differ")
    _check(lib.dsa_copy_host_to_device(_p(dst), _host_p(src_host), n, _stream(stream)), "dsa_copy_host_to_device")


def copy_device_to_host(dst_host, src, stream=None):
    """dsa_copy_device_to_host: dst_host (pinned CPU) <- src (CUDA), by a kernel."""
    n = src.numel() * src.element_size()
    if dst_host.numel() * dst_host.element_size() != n:
        raise DSAError(1, "copy_device_to_host: sizes differ")
    _check(lib.dsa_copy_device_to_host(_host_p(dst_host), _p(src), n, _stream(stream)), "dsa_copy_device_to_host")


def debug_stall_attention(n_launches: int, wait_limit_ns: int = 0, at_product: bool = False):
    """dsa_debug_stall_attention: the next n_launches attention launches take
    their timeout path after wait_limit_ns (a test hook); at_product: in the
    middle of the paged attention's work."""
    _check(lib.dsa_debug_stall_attention(n_launches | (1 << 30 if at_product else 0), wait_limit_ns),
           "dsa_debug_stall_attention")


def decode_step_launches(B, max_end_pos, k, H) -> int:
    """Kernels one dsa_decode_step launches for these sizes."""
    return int(lib.dsa_decode_step_launches(B, max_end_pos, k, H))


def decode_step_workspace_size(B, max_end_pos, k, H) -> int:
    return int(lib.dsa_decode_step_workspace_size(B, max_end_pos, k, H))


def decode_step_workspace_layout(B, max_end_pos, k, H):
    """(scores byte offset, ld, indices byte offset, mla byte offset) inside the workspace."""
    so, ld, io, mo = ctypes.c_size_t(), ctypes.c_int64(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.dsa_decode_step_workspace_layout(B, max_end_pos, k, H, ctypes.byref(so), ctypes.byref(ld),
                                                ctypes.byref(io), ctypes.byref(mo)),
           "dsa_decode_step_workspace_layout")
    return so.value, ld.value, io.value, mo.value


def decode_step(q_idx, w, k_idx, k_scale, q, kv, offsets, B, max_end_pos, kv_rows, k, H, scale, out,
                lse=None, workspace=None, status=None, stream=None):
    """dsa_decode_step: indexer -> top-k -> sparse MLA for T=1 queries."""
    out_code = DSA_BF16 if out.dtype == torch.bfloat16 else DSA_F32
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.dsa_decode_step(_p(q_idx), _p(w), _p(k_idx), _p(k_scale), _dtype_code(q_idx), _p(q), _p(kv),
                               _p(offsets), B, max_end_pos, kv_rows, k, H, float(scale), _p(out), out_code,
                               _p(lse), _p(workspace), ws_bytes, _p(status), _stream(stream)),
           "dsa_decode_step")


# ---- paged cache.  Sizes are taken from the tensors and checked against each
# other here: the library sees pointers only.

def _arg(t, dtype, shape, what, dev, rows=False):
    """Pointer of a CUDA tensor of this type and shape on device number `dev`;
    None gives NULL.  rows: a 2-D tensor whose rows may lie further apart than
    they are long."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous() or (rows and t.stride(1) == 1 and (t.stride(0) >= shape[1] or shape[0] == 1)):
            return t.data_ptr()
    if t.dtype is not dtype or t.shape != shape:
        raise DSAError(1, f"{what} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")
    if t.get_device() != dev:
        raise DSAError(1, f"{what} is on {t.device}, not on cuda:{dev}")
    raise DSAError(1, f"the rows of {what} are not contiguous" if rows else f"{what} is not contiguous")


def _row_pitch(t):
    """Elements from one row of a 2-D tensor to the next."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


# The current stream's handle by device number: torch.cuda.current_stream()
# builds a Stream object first, 3.4 us a call against 0.07.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run_on(dev, stream, fn, what, *args):
    """fn(*args, stream) on device number `dev`, whatever device is current."""
    if stream is not None and stream.device.index != dev:
        raise DSAError(1, f"{what}: the stream is on {stream.device}, the tensors on cuda:{dev}")
    handle = _raw_stream(dev) if stream is None else stream.cuda_stream
    if dev == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc:
        raise DSAError(rc, what)


def _pages(kv_pages, page_table, what):
    """(device number, B, page_size, n_pages, pool pointer, table pointer, table
    row pitch, max_pages) of a paged cache, checked."""
    shape = kv_pages.shape
    if len(shape) != 3 or shape[2] != 576:
        raise DSAError(1, f"{what}: kv_pages must be bfloat16 [n_pages, page_size, 576]")
    dev = kv_pages.get_device()
    if dev < 0:
        raise DSAError(1, f"{what}: kv_pages is not on a CUDA device")
    table = page_table.shape
    if len(table) != 2:
        raise DSAError(1, f"{what}: page_table must be [B, max_pages]")
    # the plain case without a second look at the shapes (0.5 us a call less)
    if kv_pages.dtype is torch.bfloat16 and kv_pages.is_contiguous():
        kv = kv_pages.data_ptr()
    else:
        kv = _arg(kv_pages, torch.bfloat16, shape, "kv_pages", dev)
    if page_table.dtype is torch.int32 and page_table.is_contiguous() and page_table.get_device() == dev:
        return dev, table[0], shape[1], shape[0], kv, page_table.data_ptr(), table[1], table[1]
    return (dev, table[0], shape[1], shape[0], kv, _arg(page_table, torch.int32, table, "page_table", dev, rows=True),
            _row_pitch(page_table), table[1])


def _slots(acc, pos, B, dev):
    """(acc, pos, ld_slots): pointers and row length of the per-slot arrays [B, slots]."""
    one = acc if acc is not None else pos
    if one is None:
        return None, None, 0
    shape = one.shape
    if len(shape) != 2:
        raise DSAError(1, "acc and pos must be [B, slots]")
    shape = (B, shape[1])
    return _arg(acc, torch.float32, shape, "acc", dev), _arg(pos, torch.int32, shape, "pos", dev), shape[1]


def _out_code(out, shape, dev):
    """DSA_BF16 or DSA_F32 of an output tensor, and its pointer."""
    if out.dtype is not torch.bfloat16 and out.dtype is not torch.float32:
        raise DSAError(1, f"out must be bfloat16 or float32, not {out.dtype}")
    return (DSA_BF16 if out.dtype is torch.bfloat16 else DSA_F32), _arg(out, out.dtype, shape, "out", dev)


def paged_append(kv_new, kv_pages, page_table, lens, acc=None, pos=None, end_pos=None, status=None, stream=None):
    """dsa_paged_append: the newest T tokens' rows kv_new [B,T,576] into each
    sequence's last T slots, acc = 0 and pos = end_pos - T + t beside them."""
    dev, B, P, n_pages, kv, table, ld_table, max_pages = _pages(kv_pages, page_table, "paged_append")
    if kv_new.dim() != 3:
        raise DSAError(1, "paged_append: kv_new must be [B, T, 576]")
    T = kv_new.shape[1]
    a, p, ld = _slots(acc, pos, B, dev)
    _run_on(dev, stream, lib.dsa_paged_append, "dsa_paged_append",
            _arg(kv_new, torch.bfloat16, (B, T, 576), "kv_new", dev), _arg(lens, torch.int32, (B,), "lens", dev), table,
            ld_table, max_pages, B, T, P, n_pages, kv, a, p, _arg(end_pos, torch.int32, (B,), "end_pos", dev), ld,
            _arg(status, torch.int32, (1,), "status", dev))


def paged_mla_workspace_size(B, T, H) -> int:
    """Workspace bytes of paged_mla on the current device."""
    return int(lib.dsa_paged_mla_workspace_size(B, T, H))


def paged_mla(q, kv_pages, page_table, lens, scale, out, lse=None, workspace=None, status=None, stream=None):
    """dsa_paged_mla: attention of q [B,T,H,576] over the whole paged cache
    into out [B,T,H,512] (bf16 or fp32 by out's dtype) and lse [B,T,H]."""
    dev, B, P, n_pages, kv, table, ld_table, max_pages = _pages(kv_pages, page_table, "paged_mla")
    if q.dim() != 4:
        raise DSAError(1, "paged_mla: q must be [B, T, H, 576]")
    T, H = q.shape[1], q.shape[2]
    code, o = _out_code(out, (B, T, H, 512), dev)
    ws = None if workspace is None else _arg(workspace, workspace.dtype, workspace.shape, "workspace", dev)
    _run_on(dev, stream, lib.dsa_paged_mla, "dsa_paged_mla", _arg(q, torch.bfloat16, (B, T, H, 576), "q", dev), kv, table,
            ld_table, max_pages, _arg(lens, torch.int32, (B,), "lens", dev), B, T, H, P, n_pages, float(scale), o, code,
            _arg(lse, torch.float32, (B, T, H), "lse", dev), ws, 0 if ws is None else workspace.nbytes,
            _arg(status, torch.int32, (1,), "status", dev))


def paged_weights(q, kv_pages, page_table, lens, lse, scale, acc, acc_out=None, decay=1.0, status=None, stream=None):
    """dsa_paged_weights: acc_out [B,slots] = decay * acc + the attention
    weight every slot gets from q [B,T,H,576].  acc_out: acc itself unless
    given; acc=None counts as zeros."""
    dev, B, P, n_pages, kv, table, ld_table, max_pages = _pages(kv_pages, page_table, "paged_weights")
    if q.dim() != 4:
        raise DSAError(1, "paged_weights: q must be [B, T, H, 576]")
    T, H = q.shape[1], q.shape[2]
    if acc_out is None:
        acc_out = acc
    if acc_out is None:
        raise DSAError(1, "paged_weights: acc or acc_out is needed")
    o, _, ld = _slots(acc_out, None, B, dev)
    a = o if acc is acc_out else _arg(acc, torch.float32, (B, ld), "acc", dev)
    _run_on(dev, stream, lib.dsa_paged_weights, "dsa_paged_weights", _arg(q, torch.bfloat16, (B, T, H, 576), "q", dev), kv,
            table, ld_table, max_pages, _arg(lens, torch.int32, (B,), "lens", dev),
            _arg(lse, torch.float32, (B, T, H), "lse", dev), B, T, H, P, n_pages, float(scale), float(decay), a, o, ld,
            _arg(status, torch.int32, (1,), "status", dev))


def evict_plan(acc, pos, lens, end_pos, budget, recent, new_lens, n_moves, move_dst, move_src, status=None, stream=None):
    """dsa_evict_plan: new lengths and the move list that cut every sequence
    to `budget` slots (pos and end_pos may be None when recent is 0)."""
    if acc.dim() != 2 or move_dst.dim() != 2:
        raise DSAError(1, "evict_plan: acc must be [B, slots], move_dst and move_src [B, moves]")
    dev, B, moves = acc.get_device(), acc.shape[0], move_dst.shape
    if dev < 0:
        raise DSAError(1, "evict_plan: acc is not on a CUDA device")
    if moves[0] != B:
        raise DSAError(1, "evict_plan: move_dst and move_src need a row per sequence")
    a, p, ld = _slots(acc, pos, B, dev)
    _run_on(dev, stream, lib.dsa_evict_plan, "dsa_evict_plan", a, p, _arg(lens, torch.int32, (B,), "lens", dev),
            _arg(end_pos, torch.int32, (B,), "end_pos", dev), B, ld, int(budget), int(recent),
            _arg(new_lens, torch.int32, (B,), "new_lens", dev), _arg(n_moves, torch.int32, (B,), "n_moves", dev),
            _arg(move_dst, torch.int32, moves, "move_dst", dev), _arg(move_src, torch.int32, moves, "move_src", dev),
            moves[1], _arg(status, torch.int32, (1,), "status", dev))


def paged_move(kv_pages, page_table, n_moves, move_dst, move_src, acc=None, pos=None, status=None, stream=None):
    """dsa_paged_move: carries an eviction plan out on the cache, acc and pos."""
    dev, B, P, n_pages, kv, table, ld_table, max_pages = _pages(kv_pages, page_table, "paged_move")
    if move_dst.dim() != 2 or move_dst.shape[0] != B:
        raise DSAError(1, "paged_move: move_dst and move_src must be [B, moves]")
    moves = move_dst.shape
    a, p, ld = _slots(acc, pos, B, dev)
    _run_on(dev, stream, lib.dsa_paged_move, "dsa_paged_move", kv, table, ld_table, max_pages, P, n_pages,
            _arg(n_moves, torch.int32, (B,), "n_moves", dev), _arg(move_dst, torch.int32, moves, "move_dst", dev),
            _arg(move_src, torch.int32, moves, "move_src", dev), moves[1], B, a, p, ld,
            _arg(status, torch.int32, (1,), "status", dev))
