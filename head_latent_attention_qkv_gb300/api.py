"""Python entry points with the C ABI's names, taking torch tensors.

Marshalling only: pointers, sizes and the current CUDA stream are passed to
``libmla_draft.so``; torch allocates the caller-owned device buffers (weight
arena, workspace, outputs).  Tensors must already be on the CUDA device, of the
layer's dtype (weights, hidden, cache, out) or int32/int64/uint8 for indices.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from ._lib import check, lib

_TORCH_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def torch_dtype(dims) -> torch.dtype:
    return _TORCH_DTYPE[dims.dtype]


def make_config(dims, page_size: int) -> _lib.mla_config_t:
    return _lib.mla_config_t(
        hidden_size=dims.hidden_size, num_heads=dims.num_heads, q_lora_rank=dims.q_lora_rank,
        kv_lora_rank=dims.kv_lora_rank, qk_nope_head_dim=dims.qk_nope_head_dim,
        qk_rope_head_dim=dims.qk_rope_head_dim, v_head_dim=dims.v_head_dim,
        rope=_lib.MLA_ROPE_INTERLEAVED if dims.rope_style == "interleaved" else _lib.MLA_ROPE_NEOX,
        use_output_gate=int(bool(dims.use_output_gate)),
        dtype=_lib.MLA_BF16 if dims.dtype == "bf16" else _lib.MLA_FP32, page_size=page_size,
        max_position=dims.max_position, rope_theta=dims.rope_theta,
        rms_norm_eps=dims.rms_norm_eps, softmax_scale=dims.softmax_scale)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _buf(nbytes: int, device) -> torch.Tensor:
    # 256-byte aligned: the caching allocator hands out 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class Handle:
    """A library handle plus the device buffers the caller owns for it."""

    def __init__(self, dims, weights: dict, page_size: int, device="cuda", stream=None):
        self.dims, self.page_size, self.device = dims, page_size, torch.device(device)
        self.device_index = torch.cuda.current_device() if self.device.index is None else self.device.index
        self.cfg = make_config(dims, page_size)
        self.arena = _buf(lib.mla_weight_arena_bytes(C.byref(self.cfg)), self.device)
        w = _lib.mla_weights_t(**{k: (weights[k].data_ptr() if weights.get(k) is not None else None)
                                  for k in _lib.WEIGHT_FIELDS})
        h = C.c_void_p()
        check(lib.mla_draft_init(C.byref(self.cfg), C.byref(w), _ptr(self.arena),
                                 self.arena.numel(), _stream(stream), C.byref(h)), "mla_draft_init")
        self.h = h
        self._ws = None

    def workspace(self, nbytes: int) -> torch.Tensor:
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = _buf(nbytes, self.device)
        return self._ws

    def close(self):
        if self.h:
            lib.mla_draft_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mla_draft_init(dims, weights: dict, page_size: int, device="cuda", stream=None) -> Handle:
    return Handle(dims, weights, page_size, device, stream)


def mla_latent_cache_append(h: Handle, hidden, positions, slot_mapping, cache, stream=None,
                            workspace=None):
    n = hidden.shape[0]
    need = lib.mla_append_workspace_bytes(h.h, n)
    ws = workspace if workspace is not None else h.workspace(need)
    check(lib.mla_latent_cache_append(h.h, _ptr(hidden), _ptr(positions), _ptr(slot_mapping), n,
                                      _ptr(cache), cache.shape[0], _ptr(ws), ws.numel(),
                                      _stream(stream)), "mla_latent_cache_append")


def make_desc(block_table, kv_len, window=None, q_visible=None, block_len=16, vis_stats=None):
    return _lib.mla_attn_desc_t(
        num_blocks=block_table.shape[0], block_len=block_len, max_pages=block_table.shape[1],
        reserved=0, block_table=block_table.data_ptr(), kv_len=kv_len.data_ptr(),
        window=None if window is None else window.data_ptr(),
        q_visible=None if q_visible is None else q_visible.data_ptr(),
        vis_stats=None if vis_stats is None else vis_stats.data_ptr())


def mla_draft_forward(h: Handle, hidden, positions, block_slot_mapping, cache, desc, out=None,
                      stream=None, workspace=None):
    M = desc.num_blocks * desc.block_len
    if out is None:
        out = torch.empty(M, h.dims.hidden_size, dtype=torch_dtype(h.dims), device=h.device)
    need = lib.mla_forward_workspace_bytes(h.h, M)
    ws = workspace if workspace is not None else h.workspace(need)
    check(lib.mla_draft_forward(h.h, _ptr(hidden), _ptr(positions), _ptr(block_slot_mapping),
                                _ptr(cache), cache.shape[0], C.byref(desc), _ptr(out), _ptr(ws),
                                ws.numel(), _stream(stream)), "mla_draft_forward")
    return out


def make_shared_ctx(ctx_len, ctx_block_start, ctx_rows):
    """Context list for mla_draft_forward_shared: device int32 ``ctx_len``
    [num_ctx] and ``ctx_block_start`` [num_ctx + 1]; ``ctx_rows`` (host int)
    is the sum of ``ctx_len``."""
    return _lib.mla_shared_ctx_t(num_ctx=ctx_len.shape[0], ctx_rows=int(ctx_rows),
                                 ctx_len=ctx_len.data_ptr(), ctx_block_start=ctx_block_start.data_ptr())


def mla_draft_forward_shared(h: Handle, hidden, positions, block_slot_mapping, cache, desc, ctx,
                             out=None, stream=None, workspace=None):
    """mla_draft_forward for blocks that share contexts (``ctx`` from
    make_shared_ctx): the expanded form where the layer allows it."""
    M = desc.num_blocks * desc.block_len
    if out is None:
        out = torch.empty(M, h.dims.hidden_size, dtype=torch_dtype(h.dims), device=h.device)
    need = lib.mla_forward_shared_workspace_bytes(h.h, M, ctx.ctx_rows)
    ws = workspace if workspace is not None else h.workspace(need)
    check(lib.mla_draft_forward_shared(h.h, _ptr(hidden), _ptr(positions), _ptr(block_slot_mapping),
                                       _ptr(cache), cache.shape[0], C.byref(desc), C.byref(ctx),
                                       _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
          "mla_draft_forward_shared")
    return out


def mla_draft_forward_shared_after(h: Handle, hidden, positions, block_slot_mapping, cache, desc,
                                   ctx, cache_ready=None, out=None, stream=None, workspace=None):
    """mla_draft_forward_shared whose attention waits for ``cache_ready``
    (a recorded torch.cuda.Event, or None)."""
    M = desc.num_blocks * desc.block_len
    if out is None:
        out = torch.empty(M, h.dims.hidden_size, dtype=torch_dtype(h.dims), device=h.device)
    need = lib.mla_forward_shared_workspace_bytes(h.h, M, ctx.ctx_rows)
    ws = workspace if workspace is not None else h.workspace(need)
    ev = None if cache_ready is None else C.c_void_p(cache_ready.cuda_event)
    check(lib.mla_draft_forward_shared_after(h.h, _ptr(hidden), _ptr(positions),
                                             _ptr(block_slot_mapping), _ptr(cache), cache.shape[0],
                                             C.byref(desc), C.byref(ctx), _ptr(out), _ptr(ws),
                                             ws.numel(), _stream(stream), ev),
          "mla_draft_forward_shared_after")
    return out


def mla_shared_attention(h: Handle, positions, desc, ctx, workspace=None, stream=None):
    """The expanded attention step alone, on the intermediates the last
    mla_draft_forward_shared left in the workspace (the handle's unless
    given); rewrites that workspace's per-head output o."""
    M = desc.num_blocks * desc.block_len
    need = lib.mla_forward_shared_workspace_bytes(h.h, M, ctx.ctx_rows)
    ws = workspace if workspace is not None else h.workspace(need)
    check(lib.mla_shared_attention(h.h, _ptr(positions), C.byref(desc), C.byref(ctx), _ptr(ws),
                                   ws.numel(), _stream(stream)), "mla_shared_attention")


def mla_draft_forward_after(h: Handle, hidden, positions, block_slot_mapping, cache, desc,
                            cache_ready=None, out=None, stream=None, workspace=None):
    """mla_draft_forward whose attention waits for ``cache_ready`` (a
    recorded torch.cuda.Event, or None)."""
    M = desc.num_blocks * desc.block_len
    if out is None:
        out = torch.empty(M, h.dims.hidden_size, dtype=torch_dtype(h.dims), device=h.device)
    need = lib.mla_forward_workspace_bytes(h.h, M)
    ws = workspace if workspace is not None else h.workspace(need)
    ev = None if cache_ready is None else C.c_void_p(cache_ready.cuda_event)
    check(lib.mla_draft_forward_after(h.h, _ptr(hidden), _ptr(positions), _ptr(block_slot_mapping),
                                      _ptr(cache), cache.shape[0], C.byref(desc), _ptr(out),
                                      _ptr(ws), ws.numel(), _stream(stream), ev),
          "mla_draft_forward_after")
    return out


def mla_latent_attention(h: Handle, q_abs, positions, cache, desc, o_lat=None, lse=None,
                         stream=None, workspace=None):
    """The latent attention step alone: ``o_lat`` [rows, kv_lora_rank] (fp16
    for bf16 layers) and, when ``lse`` is given, its fp32 [rows] log-sum-exp.
    The workspace the few-row kernel needs comes from the handle unless given."""
    rows = desc.num_blocks * desc.block_len * h.dims.num_heads
    if o_lat is None:
        dt = torch.float16 if h.dims.dtype == "bf16" else torch.float32
        o_lat = torch.empty(rows, h.dims.kv_lora_rank, dtype=dt, device=h.device)
    need = lib.mla_latent_attention_workspace_bytes(h.h, C.byref(desc))
    ws = workspace if workspace is not None else (h.workspace(need) if need else None)
    check(lib.mla_latent_attention(h.h, _ptr(q_abs), _ptr(positions), _ptr(cache),
                                   cache.shape[0], C.byref(desc), _ptr(o_lat), _ptr(lse),
                                   _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
          "mla_latent_attention")
    return o_lat


def mla_latent_attention_workspace_bytes(h: Handle, desc) -> int:
    return int(lib.mla_latent_attention_workspace_bytes(h.h, C.byref(desc)))


def mla_latent_attention_backward(h: Handle, q_abs, positions, cache, desc, o_lat, lse, d_o_lat,
                                  d_q_abs, d_cache, stream=None):
    """Gradients of the latent attention step: d_q_abs (written) and d_cache
    (added to; fp32, zeroed by the caller)."""
    check(lib.mla_latent_attention_backward(h.h, _ptr(q_abs), _ptr(positions), _ptr(cache),
                                            cache.shape[0], C.byref(desc), _ptr(o_lat), _ptr(lse),
                                            _ptr(d_o_lat), _ptr(d_q_abs), _ptr(d_cache),
                                            _stream(stream)), "mla_latent_attention_backward")


def _take(name, t, dtype, shape, h):
    """The pointer of `t`, checked: on the handle's device, contiguous, of this
    type and shape."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != h.device_index or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:"
                         f"{h.device_index}, got {t.dtype} {tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


# torch's allocation without the dispatcher: not a public name, so a torch that
# lacks it takes torch.empty
_empty_strided_cuda = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _new(h: Handle, shape, dtype):
    """An uninitialised tensor on the handle's device, of which the call writes
    every element.  Right after a launch torch.empty takes 5 us of host time and
    the other allocation of the same pool 2; that one takes place on the current
    device, which a handle needs to be its own."""
    if _empty_strided_cuda is None or torch._C._cuda_getDevice() != h.device_index:
        return torch.empty(shape, dtype=dtype, device=h.device)
    return _empty_strided_cuda(shape, (1,) if len(shape) == 1 else (shape[1], 1), dtype)


def _new_workspace(h: Handle, nbytes):
    return _new(h, (nbytes,), torch.uint8) if nbytes else None


def _take_cache(h: Handle, cache):
    return _take("cache", cache, torch_dtype(h.dims), (cache.shape[0], h.page_size, h.dims.cache_dim), h)


def _take_rows(name, t, dtype, n, h):
    """A matrix of n rows: its pointer and row length."""
    return _take(name, t, dtype, (n, t.shape[-1]), h), t.shape[-1]


def _take_workspace(workspace, h):
    """The pointer and the bytes of a workspace, None for none."""
    if workspace is None:
        return None, 0
    return (_take("workspace", workspace, workspace.dtype, workspace.shape, h),
            workspace.numel() * workspace.element_size())


def _run(fn, h: Handle, *args):
    """The entry point `fn` on the current stream (a caller's stream argument is
    made the current one, so that what the call allocates belongs to it)."""
    status = fn(h.h, *args, torch._C._cuda_getCurrentRawStream(h.device_index))
    if status:
        check(status, fn.__name__)


def _tree_args(h: Handle, q_abs, positions, cache, desc, parent):
    d = h.dims
    tokens = desc.num_blocks * desc.block_len
    if q_abs.numel() != tokens * d.num_heads * d.cache_dim:
        raise ValueError(f"q_abs: expected {tokens * d.num_heads} rows of {d.cache_dim}, got {tuple(q_abs.shape)}")
    return (_take("q_abs", q_abs, torch_dtype(d), q_abs.shape, h),
            _take("positions", positions, torch.int32, (tokens,), h), _take_cache(h, cache),
            None if parent is None else _take("parent", parent, torch.int32, (tokens,), h))


def mla_tree_attention(h: Handle, q_abs, positions, cache, desc, parent, o_lat=None, lse=None,
                       stream=None, workspace=None):
    """Latent attention of trees of drafted tokens: ``parent`` int32 [blocks *
    nodes] (-1: a child of the context, -2: padding, else an earlier node), the
    nodes' own keys the last ``block_len`` of each sequence.  ``o_lat`` [rows,
    kv_lora_rank] (fp16 for bf16 layers) and, when ``lse`` is given, its fp32
    [rows] log-sum-exp."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_tree_attention(h, q_abs, positions, cache, desc, parent, o_lat, lse, None, workspace)
    q, pos, c, par = _tree_args(h, q_abs, positions, cache, desc, parent)
    rows, rank = desc.num_blocks * desc.block_len * h.dims.num_heads, h.dims.kv_lora_rank
    dt = torch.float16 if h.dims.dtype == "bf16" else torch.float32
    lse_p = None if lse is None else _take("lse", lse, torch.float32, (rows,), h)
    if o_lat is None:
        o_lat = _new(h, (rows, rank), dt)
    out = _take("o_lat", o_lat, dt, (rows, rank), h)
    ref = C.byref(desc)
    if workspace is None:
        workspace = _new_workspace(h, lib.mla_tree_attention_workspace_bytes(h.h, ref))
    _run(lib.mla_tree_attention, h, q, pos, c, cache.shape[0], ref, par, out, lse_p,
         *_take_workspace(workspace, h))
    return o_lat


def mla_tree_attention_workspace_bytes(h: Handle, desc) -> int:
    return int(lib.mla_tree_attention_workspace_bytes(h.h, C.byref(desc)))


def mla_draft_forward_tree(h: Handle, hidden, positions, block_slot_mapping, cache, desc, parent,
                           out=None, stream=None, workspace=None):
    """mla_draft_forward over trees of drafted tokens (``parent`` as in
    mla_tree_attention).  A ``workspace`` of the caller's keeps the absorbed
    queries and their log-sum-exps for mla_key_weights
    (mla_forward_workspace_offset, MLA_WS_Q_ABS and MLA_WS_LSE)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_draft_forward_tree(h, hidden, positions, block_slot_mapping, cache, desc, parent, out,
                                          None, workspace)
    D, dt, M = h.dims.hidden_size, torch_dtype(h.dims), desc.num_blocks * desc.block_len
    args = (_take("hidden", hidden, dt, (M, D), h), _take("positions", positions, torch.int32, (M,), h),
            None if block_slot_mapping is None else
            _take("block_slot_mapping", block_slot_mapping, torch.int64, (M,), h), _take_cache(h, cache))
    par = _take("parent", parent, torch.int32, (M,), h)
    if out is None:
        out = _new(h, (M, D), dt)
    ref = C.byref(desc)
    if workspace is None:
        workspace = _new_workspace(h, lib.mla_forward_tree_workspace_bytes(h.h, ref))
    _run(lib.mla_draft_forward_tree, h, *args, cache.shape[0], ref, par, _take("out", out, dt, (M, D), h),
         *_take_workspace(workspace, h))
    return out


def mla_forward_tree_workspace_bytes(h: Handle, desc) -> int:
    return int(lib.mla_forward_tree_workspace_bytes(h.h, C.byref(desc)))


def mla_key_weights(h: Handle, q_abs, positions, cache, desc, lse, weights_out, prior=None, decay=1.0,
                    parent=None, stream=None, workspace=None):
    """``weights_out[b, j] = decay * prior[b, j] + `` the attention weight key j
    of block b received from the block's rows, whose log-sum-exp is ``lse``
    (mla_tree_attention's with ``parent``, mla_latent_attention's without);
    ``prior`` may be ``weights_out`` itself, fp32 [blocks, keys or more]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_key_weights(h, q_abs, positions, cache, desc, lse, weights_out, prior, decay, parent,
                                   None, workspace)
    q, pos, c, par = _tree_args(h, q_abs, positions, cache, desc, parent)
    nb = desc.num_blocks
    out, ldw = _take_rows("weights_out", weights_out, torch.float32, nb, h)
    lse_p = _take("lse", lse, torch.float32, (nb * desc.block_len * h.dims.num_heads,), h)
    prior_p = None if prior is None else _take("prior", prior, torch.float32, (nb, ldw), h)
    ref = C.byref(desc)
    if workspace is None:
        workspace = _new_workspace(h, lib.mla_key_weights_workspace_bytes(h.h, ref, ldw))
    _run(lib.mla_key_weights, h, q, pos, c, cache.shape[0], ref, par, lse_p, decay, prior_p, out, ldw,
         *_take_workspace(workspace, h))
    return weights_out


def mla_key_weights_workspace_bytes(h: Handle, desc, ldw: int) -> int:
    return int(lib.mla_key_weights_workspace_bytes(h.h, C.byref(desc), ldw))


def mla_cache_select(h: Handle, weights, kv_len, budget: int, sink: int = 0, recent: int = 0,
                     keep=None, keep_len=None, stream=None):
    """``(keep, keep_len)``: per sequence the ascending indices of the keys that
    stay under ``budget`` (the first ``sink``, the last ``recent``, then the
    heaviest; -1 behind the last) and how many they are."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_cache_select(h, weights, kv_len, budget, sink, recent, keep, keep_len)
    n = kv_len.shape[0]
    w, ldw = _take_rows("weights", weights, torch.float32, n, h)
    if keep is None:
        keep = _new(h, (n, max(budget, 0)), torch.int32)
    if keep_len is None:
        keep_len = _new(h, (n,), torch.int32)
    _run(lib.mla_cache_select, h, w, ldw, _take("kv_len", kv_len, torch.int32, (n,), h), n, budget, sink, recent,
         _take("keep", keep, torch.int32, (n, max(budget, 0)), h),
         _take("keep_len", keep_len, torch.int32, (n,), h))
    return keep, keep_len


def mla_cache_compact(h: Handle, cache, block_table, kv_len, keep, keep_len, first=None,
                      dst_block_table=None, weights=None, weights_out=None, stream=None,
                      workspace=None):
    """Moves the kept entries of every sequence together (see the header): in
    place, ``weights`` with them, or into the pages of ``dst_block_table``,
    the weights into ``weights_out``.  The new lengths are ``keep_len`` (+
    ``first``)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_cache_compact(h, cache, block_table, kv_len, keep, keep_len, first, dst_block_table,
                                     weights, weights_out, None, workspace)
    _compact(h, lib.mla_cache_compact, lib.mla_cache_compact_workspace_bytes, _take_cache(h, cache), cache.shape[0],
             block_table, kv_len, keep, keep_len, first, dst_block_table, weights, weights_out, workspace)


def _compact(h, fn, workspace_bytes, cache, num_pages, block_table, kv_len, keep, keep_len, first, dst_block_table,
             weights, weights_out, workspace):
    n, i32 = kv_len.shape[0], torch.int32
    in_place = dst_block_table is None
    if weights is not None and weights_out is None and in_place:
        weights_out = weights
    table, max_pages = _take_rows("block_table", block_table, i32, n, h)
    keep_p, ldk = _take_rows("keep", keep, i32, n, h)
    dst, dst_pages = (None, 0) if in_place else _take_rows("dst_block_table", dst_block_table, i32, n, h)
    w, ldw = (None, 0) if weights is None else _take_rows("weights", weights, torch.float32, n, h)
    args = (cache, num_pages, table, max_pages, _take("kv_len", kv_len, i32, (n,), h), n,
            keep_p, ldk, _take("keep_len", keep_len, i32, (n,), h),
            None if first is None else _take("first", first, i32, (n,), h), dst, dst_pages, w,
            None if weights_out is None else _take("weights_out", weights_out, torch.float32, (n, ldw), h), ldw)
    if workspace is None and in_place:
        workspace = _new_workspace(h, workspace_bytes(h.h, n, ldk))
    _run(fn, h, *args, *_take_workspace(workspace, h))


def mla_cache_compact_workspace_bytes(h: Handle, num_seqs: int, ldk: int) -> int:
    return int(lib.mla_cache_compact_workspace_bytes(h.h, num_seqs, ldk))


class Cache8:
    """The latent cache in 8 bits (mla_cache8_t), of the caller's tensors: ``latent`` float8_e4m3fn
    [num_pages, page_size, 512], ``rope`` bfloat16 [num_pages, page_size, 64], ``scale``
    float32 [num_pages, page_size]; an entry stands for latent * scale and rope, its scale a power
    of two (or NaN: the attention reports another number).  They are
    looked at here, once, like a descriptor's, and cannot be replaced; a call checks the page size and
    the device."""
    __slots__ = ("latent", "rope", "scale", "num_pages", "page_size", "device_index", "_c", "_ref")

    def __init__(self, latent, rope, scale):
        n, page = scale.shape if scale.dim() == 2 else (-1, -1)
        device = scale.get_device()
        for name, t, dtype, shape in (("latent", latent, torch.float8_e4m3fn, (n, page, 512)),
                                      ("rope", rope, torch.bfloat16, (n, page, 64)),
                                      ("scale", scale, torch.float32, (n, page))):
            if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
                raise ValueError(f"cache {name}: expected a contiguous {dtype} tensor of shape {shape} on the "
                                 f"scale's device, got {t.dtype} {tuple(t.shape)} on {t.device}")
        c = _lib.mla_cache8_t(latent.data_ptr(), rope.data_ptr(), scale.data_ptr())
        for name, value in zip(self.__slots__, (latent, rope, scale, n, page, device, c, C.byref(c))):
            object.__setattr__(self, name, value)

    # (the C form holds the tensors' addresses, and these attributes what keeps the tensors alive)
    def __setattr__(self, name, value):
        raise AttributeError(f"Cache8.{name} is fixed: make another Cache8 for other tensors")

    def __delattr__(self, name):
        raise AttributeError(f"Cache8.{name} is fixed")

    def __iter__(self):
        return iter((self.latent, self.rope, self.scale))


def make_cache8(h: Handle, num_pages: int) -> Cache8:
    """An 8-bit cache of ``num_pages`` pages whose entries are all zero."""
    def zeros(*width, dtype):
        return torch.zeros(num_pages, h.page_size, *width, dtype=dtype, device=h.device)
    return Cache8(zeros(512, dtype=torch.uint8).view(torch.float8_e4m3fn), zeros(64, dtype=torch.bfloat16),
                  zeros(dtype=torch.float32) + 1)


def _take_cache8(h: Handle, c: Cache8):
    """The cache's C form, by reference, and its pages."""
    if c.page_size != h.page_size or c.device_index != h.device_index:
        raise ValueError(f"cache: expected pages of {h.page_size} on cuda:{h.device_index}, got pages of "
                         f"{c.page_size} on {c.scale.device}")
    return c._ref, c.num_pages


def mla_cache8_store(h: Handle, entries, slot_mapping, cache: Cache8, stream=None):
    """bf16 ``entries`` [n, 576] into the slots ``slot_mapping`` (int64 [n]) of the 8-bit cache."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_cache8_store(h, entries, slot_mapping, cache)
    n = slot_mapping.shape[0]
    _run(lib.mla_cache8_store, h, _take("entries", entries, torch.bfloat16, (n, h.dims.cache_dim), h),
         _take("slot_mapping", slot_mapping, torch.int64, (n,), h), n, *_take_cache8(h, cache))


def mla_cache8_load(h: Handle, cache: Cache8, slot_mapping, out=None, stream=None):
    """The entries of the slots ``slot_mapping`` (int64 [n]) in bf16, [n, 576]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_cache8_load(h, cache, slot_mapping, out)
    n, width = slot_mapping.shape[0], h.dims.cache_dim
    if out is None:
        out = torch.zeros(n, width, dtype=torch.bfloat16, device=h.device)   # (bad slots leave their rows)
    _run(lib.mla_cache8_load, h, *_take_cache8(h, cache),
         _take("slot_mapping", slot_mapping, torch.int64, (n,), h), n,
         _take("out", out, torch.bfloat16, (n, width), h))
    return out


def mla_latent_cache_append8(h: Handle, hidden, positions, slot_mapping, cache: Cache8, stream=None,
                             workspace=None):
    """mla_latent_cache_append into the 8-bit cache."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_latent_cache_append8(h, hidden, positions, slot_mapping, cache, None, workspace)
    n = slot_mapping.shape[0]
    args = (_take("hidden", hidden, torch_dtype(h.dims), (n, h.dims.hidden_size), h),
            _take("positions", positions, torch.int32, (n,), h),
            _take("slot_mapping", slot_mapping, torch.int64, (n,), h), n, *_take_cache8(h, cache))
    if workspace is None:
        workspace = _new_workspace(h, lib.mla_append8_workspace_bytes(h.h, n))
    _run(lib.mla_latent_cache_append8, h, *args, *_take_workspace(workspace, h))


def mla_append8_workspace_bytes(h: Handle, n: int) -> int:
    return int(lib.mla_append8_workspace_bytes(h.h, n))


def mla_latent_attention8(h: Handle, q_abs, positions, cache: Cache8, desc, parent=None, o_lat=None,
                          lse=None, stream=None, workspace=None):
    """mla_latent_attention, or mla_tree_attention where ``parent`` is given, over the
    8-bit cache: ``o_lat`` fp16 [rows, kv_lora_rank] and, when ``lse`` is given, its
    fp32 [rows] log-sum-exp."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_latent_attention8(h, q_abs, positions, cache, desc, parent, o_lat, lse, None, workspace)
    d, tokens = h.dims, desc.num_blocks * desc.block_len
    rows = tokens * d.num_heads
    if q_abs.numel() != rows * d.cache_dim:
        raise ValueError(f"q_abs: expected {rows} rows of {d.cache_dim}, got {tuple(q_abs.shape)}")
    c, num_pages = _take_cache8(h, cache)
    q = _take("q_abs", q_abs, torch.bfloat16, q_abs.shape, h)
    pos = _take("positions", positions, torch.int32, (tokens,), h)
    par = None if parent is None else _take("parent", parent, torch.int32, (tokens,), h)
    lse_p = None if lse is None else _take("lse", lse, torch.float32, (rows,), h)
    if o_lat is None:
        o_lat = _new(h, (rows, 512), torch.float16)
        out = o_lat.data_ptr()
    else:
        out = _take("o_lat", o_lat, torch.float16, (rows, 512), h)
    ref = C.byref(desc)
    if workspace is None:
        workspace = _new_workspace(h, lib.mla_latent_attention8_workspace_bytes(h.h, ref))
    _run(lib.mla_latent_attention8, h, q, pos, c, num_pages, ref, par, out, lse_p,
         *_take_workspace(workspace, h))
    return o_lat


def mla_latent_attention8_workspace_bytes(h: Handle, desc) -> int:
    return int(lib.mla_latent_attention8_workspace_bytes(h.h, C.byref(desc)))


def mla_draft_forward8(h: Handle, hidden, positions, block_slot_mapping, cache: Cache8, desc, parent=None,
                       out=None, stream=None, workspace=None):
    """mla_draft_forward, or mla_draft_forward_tree where ``parent`` is given, over the 8-bit cache."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_draft_forward8(h, hidden, positions, block_slot_mapping, cache, desc, parent, out, None,
                                      workspace)
    D, dt, M = h.dims.hidden_size, torch_dtype(h.dims), desc.num_blocks * desc.block_len
    c, num_pages = _take_cache8(h, cache)
    args = (_take("hidden", hidden, dt, (M, D), h), _take("positions", positions, torch.int32, (M,), h),
            None if block_slot_mapping is None else
            _take("block_slot_mapping", block_slot_mapping, torch.int64, (M,), h))
    par = None if parent is None else _take("parent", parent, torch.int32, (M,), h)
    if out is None:
        out = _new(h, (M, D), dt)
    ref = C.byref(desc)
    if workspace is None:
        workspace = _new_workspace(h, lib.mla_forward8_workspace_bytes(h.h, ref))
    _run(lib.mla_draft_forward8, h, *args, c, num_pages, ref, par, _take("out", out, dt, (M, D), h),
         *_take_workspace(workspace, h))
    return out


def mla_forward8_workspace_bytes(h: Handle, desc) -> int:
    return int(lib.mla_forward8_workspace_bytes(h.h, C.byref(desc)))


def mla_cache8_compact(h: Handle, cache: Cache8, block_table, kv_len, keep, keep_len, first=None,
                       dst_block_table=None, weights=None, weights_out=None, stream=None, workspace=None):
    """mla_cache_compact of an 8-bit cache."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_cache8_compact(h, cache, block_table, kv_len, keep, keep_len, first, dst_block_table, weights,
                                      weights_out, None, workspace)
    _compact(h, lib.mla_cache8_compact, lib.mla_cache8_compact_workspace_bytes, *_take_cache8(h, cache), block_table,
             kv_len, keep, keep_len, first, dst_block_table, weights, weights_out, workspace)


def mla_cache8_compact_workspace_bytes(h: Handle, num_seqs: int, ldk: int) -> int:
    return int(lib.mla_cache8_compact_workspace_bytes(h.h, num_seqs, ldk))


_PROBABILITIES = {torch.float32: _lib.MLA_FP32, torch.bfloat16: _lib.MLA_BF16, torch.float16: _lib.MLA_FP16}


def _take_probabilities(name, t, shape, dtype, h):
    """The pointer and row stride of probabilities [n, rows, vocab], whose rows may be
    parts of longer ones."""
    n, rows, vocab = shape
    seq, row, one = t.stride()
    if not n * rows:                                   # (nothing to read, whatever the strides)
        seq, row, one = rows * vocab, vocab, 1
    elif n < 2:
        seq = rows * row
    if rows < 2:                                       # (a stride of no second row says nothing)
        row = seq // rows if n > 1 and rows else vocab
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != h.device_index or (one != 1 and vocab > 1) or
            row < vocab or seq != rows * row):
        raise ValueError(f"{name}: expected {dtype} {shape} on cuda:{h.device_index}, rows evenly spaced and "
                         f"contiguous, got {t.dtype} {tuple(t.shape)} of strides {t.stride()} on {t.device}")
    return t.data_ptr(), row


def mla_verify_drafts(h: Handle, target, draft, tokens, uniforms, parent=None, first=None, stream=None):
    """``(accepted, num_accepted, next_token)`` of drafted tokens (int32 [n, T]) against the
    probabilities ``target`` [n, T + 1, vocab] and ``draft`` [n, T, vocab] (None: the
    tokens were certain) by the random numbers ``uniforms`` (fp32 [n, T + 1]).
    ``parent``: int32 [n, T], None a chain; ``first``: int32 [n], added to the taken
    nodes, so that they are mla_cache_compact's ``keep``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mla_verify_drafts(h, target, draft, tokens, uniforms, parent, first)
    (n, T), vocab, i32 = tokens.shape, target.shape[-1], torch.int32
    if target.dtype not in _PROBABILITIES:
        raise ValueError(f"target: expected fp32, bf16 or fp16 probabilities, got {target.dtype}")
    p, ldt = _take_probabilities("target", target, (n, T + 1, vocab), target.dtype, h)
    q, ldd = (None, 0) if draft is None else _take_probabilities("draft", draft, (n, T, vocab), target.dtype, h)
    tok, u = _take("tokens", tokens, i32, (n, T), h), _take("uniforms", uniforms, torch.float32, (n, T + 1), h)
    par = None if parent is None else _take("parent", parent, i32, (n, T), h)
    fst = None if first is None else _take("first", first, i32, (n,), h)
    accepted, count, token = _new(h, (n, T), i32), _new(h, (n,), i32), _new(h, (n,), i32)
    _run(lib.mla_verify_drafts, h, p, ldt, q, ldd, _PROBABILITIES[target.dtype], tok, par, u, fst, n, T, vocab,
         accepted.data_ptr(), count.data_ptr(), token.data_ptr())
    return accepted, count, token


def mla_check_wait_timeout(h: Handle, max_rounds: int, gave_up, stream=None):
    """Self-check of the bounded-wait failure path (``gave_up``: a device
    int32 tensor of one element, set to 1 when the wait gave up)."""
    check(lib.mla_check_wait_timeout(h.h, max_rounds, _ptr(gave_up), _stream(stream)),
          "mla_check_wait_timeout")


def mla_forward_workspace_offset(h: Handle, num_tokens: int, part: int) -> int:
    return int(lib.mla_forward_workspace_offset(h.h, num_tokens, part))


def mla_latent_cache_append_noalloc(h: Handle, hidden, positions, slot_mapping, cache,
                                    stream=None):
    """The allocation-free append (library-owned fixed scratch; at most
    mla_append_noalloc_max_tokens(h) tokens per call)."""
    check(lib.mla_latent_cache_append_noalloc(h.h, _ptr(hidden), _ptr(positions),
                                              _ptr(slot_mapping), hidden.shape[0], _ptr(cache),
                                              cache.shape[0], _stream(stream)),
          "mla_latent_cache_append_noalloc")


def mla_append_noalloc_max_tokens(h: Handle) -> int:
    return int(lib.mla_append_noalloc_max_tokens(h.h))


def mla_kernel_launches(h: Handle) -> int:
    return int(lib.mla_kernel_launches(h.h))


def mla_cache_entry_dim(dims, page_size: int = 64) -> int:
    return int(lib.mla_cache_entry_dim(C.byref(make_config(dims, page_size))))


def mla_cache_page_bytes(dims, page_size: int) -> int:
    return int(lib.mla_cache_page_bytes(C.byref(make_config(dims, page_size))))


def mla_weight_arena_bytes(dims, page_size: int = 64) -> int:
    return int(lib.mla_weight_arena_bytes(C.byref(make_config(dims, page_size))))


def mla_get_device_status(h: Handle, stream=None) -> int:
    bits = C.c_int32(0)
    lib.mla_get_device_status(h.h, _stream(stream), C.byref(bits))
    return bits.value
