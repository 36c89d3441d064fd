"""ctypes binding of the C ABI in include/ls.h.

Argument marshalling only: every function builds the C argument struct from torch
tensors (shapes and dtypes give the sizes), calls the library and raises LsError on a
non-OK status.  All arithmetic happens in the CUDA kernels of libls.so; there is no
other code path, and a missing library is an error.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libls.so")

LS_OK, LS_ERR_INVALID_ARG, LS_ERR_UNSUPPORTED, LS_ERR_CUDA, LS_ERR_DEVICE_STATUS = range(5)
LS_F32, LS_BF16, LS_E4M3 = 0, 1, 2
LS_ROWS_PAGED, LS_ROWS_SLOTS = 0, 1
LS_NORM_NONE, LS_NORM_RMS, LS_NORM_LAYER = 0, 1, 2
LS_ROPE_HALVES, LS_ROPE_PAIRS = 0, 1
LS_DEV_BOUNDS, LS_DEV_TIMEOUT, LS_DEV_CAPACITY = 1, 2, 4

_i32, _i64, _f32, _p = C.c_int32, C.c_int64, C.c_float, C.c_void_p


class IndexScoreArgs(C.Structure):
    _fields_ = [("batch", _i32), ("heads", _i32), ("dim", _i32), ("max_pages", _i32), ("max_len", _i32),
                ("key_dtype", _i32), ("w_dtype", _i32), ("variant", _i32), ("num_pages", _i64),
                ("q", _p), ("q_scale", _p), ("w", _p), ("key_pool", _p), ("key_scale", _p),
                ("page_table", _p), ("lens", _p), ("scores", _p)]


class TopkArgs(C.Structure):
    _fields_ = [("batch", _i32), ("k", _i32), ("max_len", _i32), ("scores", _p), ("lens", _p), ("idx", _p),
                ("sel_score", _p), ("pos_offset", _p)]


class BlockBoundPruneArgs(C.Structure):
    _fields_ = [("index", IndexScoreArgs), ("k", _i32), ("max_blocks", _i32), ("eps_rel", _f32),
                ("summaries", _p), ("block_scale", _p), ("idx", _p), ("sel_score", _p), ("survivors", _p),
                ("n_survivors", _p), ("ub", _p), ("keys_on_host", _i32), ("stage_blocks", _i32)]


class HotbufArgs(C.Structure):
    _fields_ = [("batch", _i32), ("k", _i32), ("n_slots", _i32), ("max_len", _i32), ("sel", _p),
                ("sel_score", _p), ("pos_of_slot", _p), ("recent_score", _p), ("slot_of_pos", _p),
                ("sel_slot", _p), ("miss_pos", _p), ("miss_slot", _p), ("n_miss", _p)]


class GatherArgs(C.Structure):
    _fields_ = [("batch", _i32), ("k", _i32), ("n_slots", _i32), ("max_pages", _i32), ("row_bytes", _i64),
                ("num_pages", _i64), ("host_kv", _p), ("page_table", _p), ("miss_pos", _p), ("miss_slot", _p),
                ("n_miss", _p), ("hbuf", _p)]


class SparseAttnArgs(C.Structure):
    _fields_ = [("batch", _i32), ("heads", _i32), ("dk", _i32), ("dv", _i32), ("k", _i32), ("dtype", _i32),
                ("variant", _i32), ("softmax_scale", _f32), ("addressing", _i32), ("max_pages", _i32),
                ("n_slots", _i32), ("row_stride", _i64), ("num_rows", _i64), ("q", _p), ("k_rows", _p),
                ("v_rows", _p), ("page_table", _p), ("sel", _p), ("o", _p), ("lse", _p), ("o_f32", _i32)]


class CpMergeArgs(C.Structure):
    _fields_ = [("shards", _i32), ("batch", _i32), ("k", _i32), ("cand_score", _p), ("cand_pos", _p),
                ("shard_begin", _p), ("shard_end", _p), ("idx", _p), ("sel_score", _p), ("local_sel", _p)]


class AttnMergeArgs(C.Structure):
    _fields_ = [("parts", _i32), ("batch", _i32), ("heads", _i32), ("dv", _i32), ("o_parts", _p),
                ("lse_parts", _p), ("o", _p), ("o_dtype", _i32), ("lse", _p)]


class DecodeStepArgs(C.Structure):
    _fields_ = [("index", IndexScoreArgs), ("k", _i32), ("use_c2f", _i32), ("max_blocks", _i32),
                ("eps_rel", _f32), ("summaries", _p), ("block_scale", _p), ("survivors", _p),
                ("n_survivors", _p), ("c2f_keys_on_host", _i32), ("c2f_stage_blocks", _i32),
                ("attn", SparseAttnArgs), ("use_hotbuf", _i32), ("n_slots", _i32),
                ("pos_of_slot", _p), ("recent_score", _p), ("slot_of_pos", _p), ("host_kv", _p),
                ("host_num_pages", _i64), ("hbuf", _p), ("n_miss", _p), ("idx", _p), ("sel_score", _p),
                ("events", _p), ("attn_q_ready", _p), ("sel_slot", _p), ("miss_pos", _p), ("miss_slot", _p)]


class HeadRows(C.Structure):
    _fields_ = [("heads", _i32), ("dim", _i32), ("norm", _i32), ("norm_dim", _i32), ("rope_begin", _i32),
                ("rope_layout", _i32), ("w_dtype", _i32), ("eps", _f32), ("token_stride", _i64), ("head_stride", _i64),
                ("x", _p), ("weight", _p), ("bias", _p)]


class HeadOut(C.Structure):
    _fields_ = [("dtype", _i32), ("token_stride", _i64), ("head_stride", _i64), ("out", _p), ("scale", _p)]


class QkNormRopeArgs(C.Structure):
    _refs, _device = (), None  # (see _check_device)
    _fields_ = [("tokens", _i32), ("dtype", _i32), ("rope_dim", _i32), ("max_pos", _i32), ("pos", _p),
                ("cos_sin", _p), ("q", HeadRows), ("k", HeadRows), ("q_out", HeadOut), ("k_out", HeadOut)]


class CacheAppendArgs(C.Structure):
    _refs, _device = (), None  # (see _check_device)
    _fields_ = [("batch", _i32), ("tokens", _i32), ("dtype", _i32), ("rope_dim", _i32), ("max_pos", _i32),
                ("max_pages", _i32), ("key_dtype", _i32), ("num_pages", _i64), ("kv_row_stride", _i64),
                ("key_row_stride", _i64), ("page_table", _p), ("start", _p), ("cu_tokens", _p), ("cos_sin", _p),
                ("kv", HeadRows), ("key", HeadRows), ("kv_pool", _p), ("key_pool", _p), ("key_scale", _p)]


class PrefixAttnArgs(C.Structure):
    _refs, _device = (), None  # (see _check_device)
    _fields_ = [("batch", _i32), ("heads", _i32), ("dk", _i32), ("dv", _i32), ("dtype", _i32), ("o_dtype", _i32),
                ("max_pages", _i32), ("prefix_len", _i32), ("softmax_scale", _f32), ("num_pages", _i64),
                ("row_stride", _i64), ("q", _p), ("kv_pool", _p), ("page_table", _p), ("lens", _p), ("o", _p),
                ("lse", _p)]


class PrefillStreamArgs(C.Structure):
    _fields_ = [("layers", _i32), ("batch", _i32), ("max_pages", _i32), ("max_len", _i32), ("max_blocks", _i32),
                ("n_slots", _i32), ("num_pages", _i64), ("row_bytes", _i64), ("page_table", _p), ("lens", _p),
                ("host_keys", _p), ("host_key_scales", _p), ("summaries", _p), ("block_scale", _p),
                ("host_kv", _p), ("hbuf", _p), ("pos_of_slot", _p), ("slot_of_pos", _p), ("recent_score", _p)]


STRUCTS = {"ls_index_score_args": IndexScoreArgs, "ls_topk_args": TopkArgs,
           "ls_prefill_stream_args": PrefillStreamArgs, "ls_cp_merge_args": CpMergeArgs,
           "ls_attn_merge_args": AttnMergeArgs, "ls_prefix_attn_args": PrefixAttnArgs,
           "ls_head_rows": HeadRows, "ls_head_out": HeadOut, "ls_qk_norm_rope_args": QkNormRopeArgs,
           "ls_cache_append_args": CacheAppendArgs,
           "ls_block_bound_prune_args": BlockBoundPruneArgs, "ls_hotbuf_args": HotbufArgs,
           "ls_gather_args": GatherArgs, "ls_sparse_attn_args": SparseAttnArgs,
           "ls_decode_step_args": DecodeStepArgs}


class LsError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"ls status {status}: {message}")
        self.status = status


_lib = None


def lib():
    """Load libls.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise LsError(LS_ERR_UNSUPPORTED, f"{LIB_PATH} is missing: run "
                          "`python -m sparse_attention_decode_ls_b200.build`")
        L = C.CDLL(LIB_PATH)
        P = C.POINTER
        for name, st in [("ls_index_score", IndexScoreArgs), ("ls_topk_select", TopkArgs),
                         ("ls_hotbuf_resolve", HotbufArgs), ("ls_gather_misses", GatherArgs),
                         ("ls_qk_norm_rope", QkNormRopeArgs), ("ls_cache_append", CacheAppendArgs)]:
            f = getattr(L, name)
            f.argtypes = [P(st), _p]
            f.restype = C.c_int
        for name, st in [("ls_sparse_attn_decode", SparseAttnArgs), ("ls_block_bound_prune", BlockBoundPruneArgs),
                         ("ls_decode_step", DecodeStepArgs), ("ls_prefix_attn_decode", PrefixAttnArgs)]:
            f = getattr(L, name)
            f.argtypes = [P(st), _p, C.c_size_t, _p]
            f.restype = C.c_int
        for name, st in [("ls_sparse_attn_workspace_size", SparseAttnArgs),
                         ("ls_block_bound_prune_workspace_size", BlockBoundPruneArgs),
                         ("ls_decode_step_workspace_size", DecodeStepArgs),
                         ("ls_prefix_attn_workspace_size", PrefixAttnArgs)]:
            f = getattr(L, name)
            f.argtypes = [P(st)]
            f.restype = C.c_size_t
        L.ls_cp_merge_workspace_size.argtypes = [P(CpMergeArgs)]
        L.ls_cp_merge_workspace_size.restype = C.c_size_t
        L.ls_cp_merge_topk.argtypes = [P(CpMergeArgs), _p, C.c_size_t, _p]
        L.ls_cp_merge_topk.restype = C.c_int
        L.ls_attn_merge.argtypes = [P(AttnMergeArgs), _p]
        L.ls_attn_merge.restype = C.c_int
        L.ls_prefill_stream_workspace_size.argtypes = [P(PrefillStreamArgs)]
        L.ls_prefill_stream_workspace_size.restype = C.c_size_t
        L.ls_prefill_stream.argtypes = [P(PrefillStreamArgs), _p, C.c_size_t, _p]
        L.ls_prefill_stream.restype = C.c_int
        L.ls_sparse_attn_decode_noalloc.argtypes = [P(SparseAttnArgs), _p]
        L.ls_sparse_attn_decode_noalloc.restype = C.c_int
        L.ls_build_block_summaries.argtypes = [P(IndexScoreArgs), _p, _p, _i32, _p]
        L.ls_build_block_summaries.restype = C.c_int
        L.ls_set_wait_limit.argtypes = [C.c_uint64]
        L.ls_set_wait_limit.restype = C.c_int
        L.ls_selftest_bounded_wait.argtypes = [_p]
        L.ls_selftest_bounded_wait.restype = C.c_int
        L.ls_get_error_string.restype = C.c_char_p
        L.ls_version.restype = C.c_char_p
        L.ls_check_device_status.argtypes = [_p, P(C.c_uint32)]
        L.ls_check_device_status.restype = C.c_int
        _lib = L
    return _lib


def _check(status):
    if status != LS_OK:
        raise LsError(status, lib().ls_get_error_string().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _hold(a, *objs):
    """Keep the tensors whose addresses an argument struct holds alive for as long as the
    struct: without this, a temporary such as ``x.to("cuda")`` passed to a builder is
    freed on return and its memory handed to the next allocation (often the workspace)
    before the kernel that reads it runs.  Nested structs bring their own references."""
    refs = list(getattr(a, "_refs", ()))
    for o in objs:
        if o is None:
            continue
        if isinstance(o, dict):
            refs.extend(v for v in o.values() if v is not None)
        elif isinstance(o, C.Structure):
            refs.extend(getattr(o, "_refs", ()))
        else:
            refs.append(o)
    a._refs = refs
    return a


# the current stream's handle without a Stream object around it (0.1 us instead of 3)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if device is None else device)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_DTYPES = {torch.float32: LS_F32, torch.bfloat16: LS_BF16, torch.uint8: LS_E4M3, torch.float8_e4m3fn: LS_E4M3}


def _dt(t):
    return _DTYPES[t.dtype]


def version() -> str:
    return lib().ls_version().decode()


# ------------------------------------------------------------------------------- a1
def index_args(*, q, w, key_pool, page_table, lens, scores=None, q_scale=None, key_scale=None, max_len=None,
               variant=0) -> IndexScoreArgs:
    B, H, D = q.shape
    a = IndexScoreArgs()
    a.batch, a.heads, a.dim = B, H, D
    a.max_pages = page_table.shape[1]
    a.max_len = int(max_len if max_len is not None else scores.shape[1])
    a.key_dtype = _dt(key_pool)
    a.w_dtype = _dt(w)
    a.variant = variant
    a.num_pages = key_pool.shape[0]
    a.q, a.q_scale, a.w = _ptr(q), _ptr(q_scale), _ptr(w)
    a.key_pool, a.key_scale = _ptr(key_pool), _ptr(key_scale)
    a.page_table, a.lens, a.scores = _ptr(page_table), _ptr(lens), _ptr(scores)
    return _hold(a, q, q_scale, w, key_pool, key_scale, page_table, lens, scores)


def ls_index_score(*, q, w, key_pool, page_table, lens, scores, q_scale=None, key_scale=None, variant=0,
                   stream=None):
    a = index_args(q=q, w=w, key_pool=key_pool, page_table=page_table, lens=lens, scores=scores,
                   q_scale=q_scale, key_scale=key_scale, variant=variant)
    _check(lib().ls_index_score(C.byref(a), _stream(stream)))


# ------------------------------------------------------------------------------- a2
def ls_topk_select(*, scores, lens, idx, sel_score=None, pos_offset=None, stream=None):
    a = TopkArgs()
    a.batch, a.k, a.max_len = scores.shape[0], idx.shape[1], scores.shape[1]
    a.scores, a.lens, a.idx, a.sel_score = _ptr(scores), _ptr(lens), _ptr(idx), _ptr(sel_score)
    a.pos_offset = _ptr(pos_offset)
    _check(lib().ls_topk_select(C.byref(a), _stream(stream)))


# ------------------------------------------------------------------------------- a3
def ls_build_block_summaries(*, q, w, key_pool, key_scale, q_scale, page_table, lens, max_len, summaries,
                             block_scale, stream=None):
    a = index_args(q=q, w=w, key_pool=key_pool, page_table=page_table, lens=lens, q_scale=q_scale,
                   key_scale=key_scale, max_len=max_len)
    _check(lib().ls_build_block_summaries(C.byref(a), _ptr(summaries), _ptr(block_scale),
                                          summaries.shape[1], _stream(stream)))


def c2f_args(*, index: IndexScoreArgs, k, summaries, block_scale, idx, sel_score=None, survivors=None,
             n_survivors=None, ub=None, eps_rel=0.0, keys_on_host=False, stage_blocks=0) -> BlockBoundPruneArgs:
    """keys_on_host: index's key_pool / key_scale are pinned CPU tensors (only the summaries
    are on the GPU); stage_blocks: staging capacity per request and pass (0: default)."""
    a = BlockBoundPruneArgs()
    a.keys_on_host = 1 if keys_on_host else 0
    a.stage_blocks = stage_blocks
    a.index = index
    a.k = k
    a.max_blocks = summaries.shape[1]
    a.eps_rel = eps_rel
    a.summaries, a.block_scale = _ptr(summaries), _ptr(block_scale)
    a.idx, a.sel_score, a.survivors = _ptr(idx), _ptr(sel_score), _ptr(survivors)
    a.n_survivors, a.ub = _ptr(n_survivors), _ptr(ub)
    return _hold(a, index, summaries, block_scale, idx, sel_score, survivors, n_survivors, ub)


def ls_block_bound_prune_workspace_size(a: BlockBoundPruneArgs) -> int:
    return lib().ls_block_bound_prune_workspace_size(C.byref(a))


def ls_block_bound_prune(a: BlockBoundPruneArgs, workspace, stream=None):
    _check(lib().ls_block_bound_prune(C.byref(a), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                      _stream(stream)))


# ------------------------------------------------------------------------------- a4, a5
def ls_hotbuf_resolve(*, sel, sel_score, pos_of_slot, recent_score, slot_of_pos, sel_slot, miss_pos, miss_slot,
                      n_miss, stream=None):
    a = HotbufArgs()
    a.batch, a.k = sel.shape
    a.n_slots = pos_of_slot.shape[1]
    a.max_len = slot_of_pos.shape[1]
    a.sel, a.sel_score = _ptr(sel), _ptr(sel_score)
    a.pos_of_slot, a.recent_score, a.slot_of_pos = _ptr(pos_of_slot), _ptr(recent_score), _ptr(slot_of_pos)
    a.sel_slot, a.miss_pos, a.miss_slot, a.n_miss = _ptr(sel_slot), _ptr(miss_pos), _ptr(miss_slot), _ptr(n_miss)
    _check(lib().ls_hotbuf_resolve(C.byref(a), _stream(stream)))


def ls_gather_misses(*, host_kv, page_table, miss_pos, miss_slot, n_miss, hbuf, stream=None):
    """host_kv: pinned CPU tensor [num_pages, 64, row] (its address is device-accessible
    under unified addressing); hbuf: CUDA tensor [B, n_slots, row]."""
    a = GatherArgs()
    a.batch, a.k = miss_pos.shape
    a.n_slots = hbuf.shape[1]
    a.max_pages = page_table.shape[1]
    a.row_bytes = hbuf.shape[2] * hbuf.element_size()
    a.num_pages = host_kv.shape[0]
    a.host_kv, a.page_table = _ptr(host_kv), _ptr(page_table)
    a.miss_pos, a.miss_slot, a.n_miss, a.hbuf = _ptr(miss_pos), _ptr(miss_slot), _ptr(n_miss), _ptr(hbuf)
    _check(lib().ls_gather_misses(C.byref(a), _stream(stream)))


# ------------------------------------------------------------------------------- a6
def attn_args(*, q, k_rows, v_rows=None, sel=None, o, lse, scale, page_table=None, n_slots=0, dv=None,
              variant=0, k=None) -> SparseAttnArgs:
    """k_rows / v_rows: row pools [..., row_width] (paged pool [NP,64,W] or hot buffer [B,S,W])."""
    v_rows = k_rows if v_rows is None else v_rows
    a = SparseAttnArgs()
    a.batch, a.heads, a.dk = q.shape
    a.dv = int(dv if dv is not None else o.shape[2])
    a.k = int(k if k is not None else sel.shape[1])
    a.dtype = _dt(q)
    a.variant = variant
    a.softmax_scale = scale
    a.addressing = LS_ROWS_PAGED if page_table is not None else LS_ROWS_SLOTS
    a.max_pages = 0 if page_table is None else page_table.shape[1]
    a.n_slots = n_slots if page_table is None else 0
    a.row_stride = k_rows.shape[-1]
    a.num_rows = k_rows.numel() // k_rows.shape[-1]
    a.q, a.k_rows, a.v_rows = _ptr(q), _ptr(k_rows), _ptr(v_rows)
    a.page_table, a.sel, a.o, a.lse = _ptr(page_table), _ptr(sel), _ptr(o), _ptr(lse)
    a.o_f32 = 1 if (o.dtype == torch.float32 and q.dtype == torch.bfloat16) else 0
    return _hold(a, q, k_rows, v_rows, page_table, sel, o, lse)


def ls_sparse_attn_workspace_size(a: SparseAttnArgs) -> int:
    return lib().ls_sparse_attn_workspace_size(C.byref(a))


def ls_sparse_attn_decode(a: SparseAttnArgs, workspace=None, stream=None):
    _check(lib().ls_sparse_attn_decode(C.byref(a), _ptr(workspace),
                                       0 if workspace is None else workspace.numel(), _stream(stream)))


def ls_sparse_attn_decode_noalloc(a: SparseAttnArgs, stream=None):
    """Allocation-free attention: the split-KV partials use the library's built-in
    scratch instead of a caller workspace (see include/ls.h)."""
    _check(lib().ls_sparse_attn_decode_noalloc(C.byref(a), _stream(stream)))


# ------------------------------------------------------------------------------- head rows
def head_rows(x, *, norm=LS_NORM_NONE, norm_dim=None, weight=None, bias=None, eps=1e-6, rope_begin=None,
              rope_layout=LS_ROPE_HALVES) -> HeadRows:
    """One operand of ls_qk_norm_rope (x [tokens, heads, dim]) or ls_cache_append (x [tokens, dim]);
    x may be a slice of a wider projection (its last stride 1).  norm_dim None: the whole row.
    weight / bias [norm_dim], contiguous and of one dtype; either may be absent."""
    shape, stride = x.shape, x.stride()
    dim = shape[-1]
    if stride[-1] != 1 and dim > 1:
        raise LsError(LS_ERR_INVALID_ARG, "the values of a row must be contiguous")
    if len(shape) == 3:
        heads, head_stride = shape[1], stride[1]
    elif len(shape) == 2:
        heads, head_stride = 1, 0
    else:
        raise LsError(LS_ERR_INVALID_ARG, "x must be [tokens, heads, dim] or [tokens, dim]")
    n = dim if norm_dim is None else norm_dim
    w_dtype, w, b = LS_BF16, None, None
    if bias is not None:
        if not bias.is_contiguous() or bias.numel() < n or (weight is not None and weight.dtype is not bias.dtype):
            raise LsError(LS_ERR_INVALID_ARG, "bias must be contiguous, hold norm_dim values and have the weight's dtype")
        w_dtype, b = _DTYPES[bias.dtype], bias.data_ptr()
    if weight is not None:
        if not weight.is_contiguous() or weight.numel() < n:
            raise LsError(LS_ERR_INVALID_ARG, "weight must be contiguous and hold norm_dim values")
        w_dtype, w = _DTYPES[weight.dtype], weight.data_ptr()
    r = HeadRows(heads, dim, norm, n, -1 if rope_begin is None else rope_begin, rope_layout, w_dtype, eps, stride[0],
                 head_stride, x.data_ptr(), w, b)
    r._refs = (x, weight, bias)
    r._like = shape, x.dtype
    return r


def _check_device(a, device):
    """Every tensor of a call lies on the current device, where the kernel runs, or in pinned host
    memory; looked at once per argument struct and device."""
    for t in a._refs:
        if t is not None and t.get_device() != device and not (t.get_device() < 0 and t.is_pinned()):
            raise LsError(LS_ERR_INVALID_ARG, "a tensor is neither on the current device nor in pinned host memory")
    a._device = device


def _ints(t, n, what):
    """Positions, lengths, page ids: int32, as the library reads them (torch makes int64 by default)."""
    if t.dtype is not torch.int32 or not t.is_contiguous() or t.numel() < n:
        raise LsError(LS_ERR_INVALID_ARG, what + " must be int32, contiguous and long enough")
    return t.data_ptr()


def _angle_table(t):
    if t is None:
        return 0, 0, None
    shape = t.shape
    if t.dtype is not torch.float32 or not t.is_contiguous() or len(shape) != 2:
        raise LsError(LS_ERR_INVALID_ARG, "cos_sin must be float32 [max_pos, rope_dim], contiguous")
    return shape[0], shape[1], t.data_ptr()


_NO_ROWS, _NO_OUT = HeadRows(), HeadOut()


def _head_out(r, t, scale, tokens) -> HeadOut:
    """t [>= tokens, heads, dim] (or [>= tokens, dim] for one head), any strides but the last's."""
    if t is None:
        raise LsError(LS_ERR_INVALID_ARG, "an operand has no output")
    shape, stride = t.shape, t.stride()
    if shape != r._like[0] and (shape[0] < tokens or shape[-1] != r.dim or
                                not (len(shape) == 2 and r.heads == 1 or len(shape) == 3 and shape[1] == r.heads)):
        raise LsError(LS_ERR_INVALID_ARG, "an output must be [tokens, heads, dim]")
    if stride[-1] != 1 and shape[-1] > 1:
        raise LsError(LS_ERR_INVALID_ARG, "the values of an output row must be contiguous")
    if scale is None:
        return HeadOut(_DTYPES[t.dtype], stride[0], stride[1], t.data_ptr())
    if scale.dtype is not torch.float32 or not scale.is_contiguous() or scale.numel() < tokens * r.heads:
        raise LsError(LS_ERR_INVALID_ARG, "a scale must be float32 [tokens, heads], contiguous")
    return HeadOut(_DTYPES[t.dtype], stride[0], stride[1], t.data_ptr(), scale.data_ptr())


def _operands(r, s, tokens):
    """Both operands (either may be absent, not both) have one dtype and a row for every token (None: as
    many as the first one has).  The first one that is given, and the tokens."""
    if r is None:
        r = s
        if r is None:
            raise LsError(LS_ERR_INVALID_ARG, "neither operand is given")
    shape, dtype = r._like
    if tokens is None:
        tokens = shape[0]
    if shape[0] < tokens:
        raise LsError(LS_ERR_INVALID_ARG, "an operand has fewer rows than there are tokens")
    if s is not None and (s._like[1] is not dtype or s._like[0][0] < tokens):
        raise LsError(LS_ERR_INVALID_ARG, "the second operand has another dtype than the first or too few rows")
    return r, dtype, tokens


def qk_norm_rope_args(*, pos, cos_sin=None, q=None, q_out=None, q_scale=None, k=None, k_out=None,
                      k_scale=None) -> QkNormRopeArgs:
    """q / k: head_rows operands (or None); q_out / k_out [tokens, heads, dim] of x's dtype, or uint8 /
    float8_e4m3fn with a scale [tokens, heads]; cos_sin [max_pos, rope_dim] float32; pos [tokens] int32."""
    max_pos, rope_dim, angles = _angle_table(cos_sin)
    r, dtype, tokens = _operands(q, k, pos.numel())
    a = QkNormRopeArgs(tokens, _DTYPES[dtype], rope_dim, max_pos, _ints(pos, tokens, "pos"), angles,
                       _NO_ROWS if q is None else q, _NO_ROWS if k is None else k,
                       _NO_OUT if q is None else _head_out(q, q_out, q_scale, tokens),
                       _NO_OUT if k is None else _head_out(k, k_out, k_scale, tokens))
    a._refs = r._refs + (pos, cos_sin, q_out, q_scale, k_out, k_scale) + (() if k is None or k is r else k._refs)
    return a


def ls_qk_norm_rope(*, args=None, stream=None, **tensors):
    """qk_norm_rope_args' tensors, or `args` built from them before."""
    a = qk_norm_rope_args(**tensors) if args is None else args
    device = torch.cuda.current_device()
    if a._device != device:
        _check_device(a, device)
    _check(lib().ls_qk_norm_rope(C.byref(a), _stream(stream, device)))


def _pool(t, width):
    """Pages and row stride of a pool [num_pages, 64, >= width], which may be a view: the library takes
    64 rows of it from page to page."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != 64 or shape[2] < width:
        raise LsError(LS_ERR_INVALID_ARG, "a pool is [num_pages, 64, row], its rows no shorter than x's")
    if stride[2] != 1 or (stride[0] != 64 * stride[1] and shape[0] > 1):
        raise LsError(LS_ERR_INVALID_ARG, "the rows of a pool must be contiguous and its pages 64 row strides apart")
    return shape[0], stride[1]


def cache_append_args(*, page_table, start, cu_tokens=None, cos_sin=None, kv=None, kv_pool=None, key=None,
                      key_pool=None, key_scale=None) -> CacheAppendArgs:
    """kv / key: head_rows operands of one row per token (or None); kv_pool [num_pages, 64, W] of x's
    dtype; key_pool the same, or uint8 / float8_e4m3fn with key_scale [num_pages, 64].  A pool may be a
    view whose pages are 64 row strides apart (a slice of wider rows, a layer of [layers, num_pages, 64, W])."""
    r, dtype, tokens = _operands(kv, key, None)
    max_pos, rope_dim, angles = _angle_table(cos_sin)
    batch, max_pages = page_table.shape
    num_pages, kv_stride, key_stride = 1 << 62, 0, 0
    if kv is not None:
        if kv_pool is None or kv_pool.dtype is not dtype:
            raise LsError(LS_ERR_INVALID_ARG, "kv_pool must be given, in x's dtype")
        num_pages, kv_stride = _pool(kv_pool, kv.dim)
    if key is not None:
        if key_pool is None:
            raise LsError(LS_ERR_INVALID_ARG, "key_pool must be given")
        n, key_stride = _pool(key_pool, key.dim)
        num_pages = min(num_pages, n)
        if key_scale is not None and (key_scale.dtype is not torch.float32 or not key_scale.is_contiguous() or
                                      key_scale.numel() < 64 * num_pages):
            raise LsError(LS_ERR_INVALID_ARG, "key_scale must be float32 [num_pages, 64], contiguous")
    a = CacheAppendArgs(batch, tokens, _DTYPES[dtype], rope_dim, max_pos, max_pages,
                        0 if key_pool is None else _DTYPES[key_pool.dtype], num_pages, kv_stride, key_stride,
                        _ints(page_table, 0, "page_table"), _ints(start, batch, "start"),
                        None if cu_tokens is None else _ints(cu_tokens, batch + 1, "cu_tokens"), angles,
                        _NO_ROWS if kv is None else kv, _NO_ROWS if key is None else key,
                        _ptr(kv_pool), _ptr(key_pool), _ptr(key_scale))
    a._refs = r._refs + (page_table, start, cu_tokens, cos_sin, kv_pool, key_pool, key_scale) + (
        () if key is None or key is r else key._refs)
    return a


def ls_cache_append(*, args=None, stream=None, **tensors):
    """cache_append_args' tensors, or `args` built from them before."""
    a = cache_append_args(**tensors) if args is None else args
    device = torch.cuda.current_device()
    if a._device != device:
        _check_device(a, device)
    _check(lib().ls_cache_append(C.byref(a), _stream(stream, device)))


# ------------------------------------------------------------------------------- shared prefix
def prefix_attn_args(*, q, kv_pool, page_table, lens, o, lse, scale, prefix_len=0) -> PrefixAttnArgs:
    """q [B,H,576], kv_pool [num_pages,64,W] latent rows, o [B,H,512] bf16 or float32, lse [B,H]."""
    B, H, D = q.shape
    rows, heads, dv = o.shape
    dtype = q.dtype
    if kv_pool.dtype is not dtype:
        raise LsError(LS_ERR_INVALID_ARG, "kv_pool must have q's dtype")
    if not q.is_contiguous() or not o.is_contiguous() or rows < B or heads != H:
        raise LsError(LS_ERR_INVALID_ARG, "q and o must be contiguous, o [B, H, dv]")
    if lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.numel() < B * H:
        raise LsError(LS_ERR_INVALID_ARG, "lse must be float32 [B, H], contiguous")
    max_pages = page_table.shape[1]
    a = PrefixAttnArgs(B, H, D, dv, _DTYPES[dtype], _DTYPES[o.dtype], max_pages, int(prefix_len), scale, *_pool(kv_pool, D),
                       q.data_ptr(), kv_pool.data_ptr(), _ints(page_table, B * max_pages, "page_table"), _ints(lens, B, "lens"),
                       o.data_ptr(), lse.data_ptr())
    a._refs = (q, kv_pool, page_table, lens, o, lse)
    return a


def ls_prefix_attn_workspace_size(a: PrefixAttnArgs) -> int:
    return lib().ls_prefix_attn_workspace_size(C.byref(a))


def ls_prefix_attn_decode(a: PrefixAttnArgs, workspace=None, stream=None):
    device = torch.cuda.current_device()
    if a._device != device:
        _check_device(a, device)
    if workspace is not None and workspace.get_device() != device:
        raise LsError(LS_ERR_INVALID_ARG, "the workspace is not on the current device")
    _check(lib().ls_prefix_attn_decode(C.byref(a), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                       _stream(stream, device)))


# ------------------------------------------------------------------------------- a7
def decode_step_args(*, index: IndexScoreArgs, k, attn: SparseAttnArgs, c2f=None, hotbuf=None, idx=None,
                     sel_score=None, events=None) -> DecodeStepArgs:
    """c2f: dict(summaries, block_scale, survivors=None, n_survivors=None, eps_rel=0.0,
    keys_on_host=False, stage_blocks=0);
    hotbuf: dict(pos_of_slot, recent_score, slot_of_pos, host_kv, hbuf, n_miss=None,
    sel_slot=None, miss_pos=None, miss_slot=None).
    events: optional ctypes array of 6 cudaEvent_t handles."""
    a = DecodeStepArgs()
    a.index = index
    a.k = k
    a.attn = attn
    if c2f is not None:
        a.use_c2f = 1
        a.max_blocks = c2f["summaries"].shape[1]
        a.eps_rel = c2f.get("eps_rel", 0.0)
        a.summaries, a.block_scale = _ptr(c2f["summaries"]), _ptr(c2f["block_scale"])
        a.survivors, a.n_survivors = _ptr(c2f.get("survivors")), _ptr(c2f.get("n_survivors"))
        a.c2f_keys_on_host = 1 if c2f.get("keys_on_host") else 0
        a.c2f_stage_blocks = int(c2f.get("stage_blocks", 0))
    if hotbuf is not None:
        a.use_hotbuf = 1
        a.n_slots = hotbuf["pos_of_slot"].shape[1]
        a.pos_of_slot, a.recent_score = _ptr(hotbuf["pos_of_slot"]), _ptr(hotbuf["recent_score"])
        a.slot_of_pos, a.host_kv = _ptr(hotbuf["slot_of_pos"]), _ptr(hotbuf["host_kv"])
        a.host_num_pages = hotbuf["host_kv"].shape[0]
        a.hbuf, a.n_miss = _ptr(hotbuf["hbuf"]), _ptr(hotbuf.get("n_miss"))
        a.sel_slot, a.miss_pos = _ptr(hotbuf.get("sel_slot")), _ptr(hotbuf.get("miss_pos"))
        a.miss_slot = _ptr(hotbuf.get("miss_slot"))
    a.idx, a.sel_score = _ptr(idx), _ptr(sel_score)
    a.events = None if events is None else C.cast(events, C.c_void_p).value
    return _hold(a, index, attn, c2f, hotbuf, idx, sel_score, events)


def ls_decode_step_workspace_size(a: DecodeStepArgs) -> int:
    return lib().ls_decode_step_workspace_size(C.byref(a))


def ls_decode_step(a: DecodeStepArgs, workspace, stream=None):
    _check(lib().ls_decode_step(C.byref(a), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                _stream(stream)))


def ls_check_device_status(stream=None) -> int:
    """Synchronise, return and clear the device status bits (LS_DEV_*)."""
    flags = C.c_uint32(0)
    st = lib().ls_check_device_status(_stream(stream), C.byref(flags))
    if st not in (LS_OK, LS_ERR_DEVICE_STATUS):
        _check(st)
    return int(flags.value)


def event_array(events):
    """ctypes array of raw cudaEvent_t handles from torch.cuda.Event objects (None:
    that stage boundary is not recorded)."""
    arr = (C.c_void_p * len(events))()
    for i, e in enumerate(events):
        arr[i] = None if e is None else e.cuda_event
    return arr


# ------------------------------------------------------------------------------- prefill
def _ptr_array(ts):
    arr = (C.c_void_p * len(ts))(*[None if t is None else t.data_ptr() for t in ts])
    return arr


def prefill_args(*, page_table, lens, max_len, host_keys, host_key_scales, summaries, block_scale,
                 host_kv=None, hbuf=None, pos_of_slot=None, slot_of_pos=None, recent_score=None) -> PrefillStreamArgs:
    """Per-layer lists: host_keys / host_key_scales / host_kv are pinned CPU tensors, the rest
    CUDA tensors; the hot-buffer lists are given together or not at all (no seeding)."""
    a = PrefillStreamArgs()
    a.layers = len(host_keys)
    a.batch = page_table.shape[0]
    a.max_pages = page_table.shape[1]
    a.max_len = int(max_len)
    a.max_blocks = summaries[0].shape[1]
    a.num_pages = host_keys[0].shape[0]
    seed = hbuf is not None
    a.n_slots = hbuf[0].shape[1] if seed else 0
    a.row_bytes = hbuf[0].shape[2] * hbuf[0].element_size() if seed else 0
    a.page_table, a.lens = _ptr(page_table), _ptr(lens)
    arrays = {"host_keys": host_keys, "host_key_scales": host_key_scales, "summaries": summaries,
              "block_scale": block_scale}
    if seed:
        arrays.update(host_kv=host_kv, hbuf=hbuf, pos_of_slot=pos_of_slot, slot_of_pos=slot_of_pos,
                      recent_score=recent_score)
    held = []
    for name, ts in arrays.items():
        arr = _ptr_array(ts)
        setattr(a, name, C.cast(arr, C.c_void_p).value)
        held.append(arr)
        held.extend(ts)
    return _hold(a, page_table, lens, *held)


def ls_prefill_stream_workspace_size(a: PrefillStreamArgs) -> int:
    return lib().ls_prefill_stream_workspace_size(C.byref(a))


def ls_prefill_stream(a: PrefillStreamArgs, workspace, stream=None):
    _check(lib().ls_prefill_stream(C.byref(a), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                   _stream(stream)))


# ------------------------------------------------------------------------------- context parallel
def cp_merge_args(*, cand_score, cand_pos, shard_begin, shard_end, idx, sel_score=None, local_sel=None):
    """cand_score / cand_pos: [G, B, k] gathered candidates (CUDA tensors)."""
    a = CpMergeArgs()
    a.shards, a.batch, a.k = cand_score.shape
    a.cand_score, a.cand_pos = _ptr(cand_score), _ptr(cand_pos)
    a.shard_begin, a.shard_end = _ptr(shard_begin), _ptr(shard_end)
    a.idx, a.sel_score, a.local_sel = _ptr(idx), _ptr(sel_score), _ptr(local_sel)
    return _hold(a, cand_score, cand_pos, shard_begin, shard_end, idx, sel_score, local_sel)


def ls_cp_merge_workspace_size(a: CpMergeArgs) -> int:
    return lib().ls_cp_merge_workspace_size(C.byref(a))


def ls_cp_merge_topk(a: CpMergeArgs, workspace, stream=None):
    _check(lib().ls_cp_merge_topk(C.byref(a), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                  _stream(stream)))


def ls_attn_merge(*, o_parts, lse_parts, o, lse, stream=None):
    """o_parts [G, B, H, dv] float32, lse_parts [G, B, H]; o [B, H, dv] bf16 or float32."""
    a = AttnMergeArgs()
    a.parts, a.batch, a.heads, a.dv = o_parts.shape
    a.o_parts, a.lse_parts, a.o, a.lse = _ptr(o_parts), _ptr(lse_parts), _ptr(o), _ptr(lse)
    a.o_dtype = LS_F32 if o.dtype == torch.float32 else LS_BF16
    _check(lib().ls_attn_merge(C.byref(a), _stream(stream)))


# ------------------------------------------------------------------------------- diagnostics
def ls_set_wait_limit(ns: int):
    _check(lib().ls_set_wait_limit(int(ns)))


def ls_selftest_bounded_wait(stream=None):
    _check(lib().ls_selftest_bounded_wait(_stream(stream)))
