"""torch-facing binding of the device calls (marshalling only).

Each function checks tensor placement, dtype and layout, then hands raw
device pointers and the current CUDA stream to the C ABI.  All arithmetic
happens in the library's kernels; nothing here computes a result.
"""

import ctypes

import numpy as np
import torch

from . import _lib

_DTYPE_CODE = {torch.float16: _lib.PKV_F16, torch.bfloat16: _lib.PKV_BF16}
_SIZE_T_MAX = ctypes.c_size_t(-1).value


def _stream_handle(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _c_int(value, name):
    """``value`` as the int the C call takes (ctypes would drop higher bits)."""
    value = int(value)
    if not -2**31 <= value < 2**31:
        raise ValueError(f"{name} must fit 32 bits, got {value}")
    return value


def _launch(name, index, *args):
    """Call the library with the current stream of CUDA device ``index`` as the
    last argument and that device current (the calls plan, and launch, on the
    current device)."""
    fn = getattr(_lib.load(), name)
    if index == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, name)


def _cuda(t, name, dtype=None, ndim=None):
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()
            and (dtype is None or t.dtype is dtype) and (ndim is None or t.dim() == ndim)):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def decode_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len):
    """Tokens per partition the library picks on the current device."""
    return _lib.load().pkv_decode_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                 max_context_len)


def decode_uses_tensor_cores(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                             partition_size=0):
    """Whether a decode call of these sizes runs the tensor-core kernel."""
    r = _lib.load().pkv_decode_uses_tensor_cores(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                 max_context_len, partition_size)
    if r < 0:
        raise ValueError("invalid decode sizes")
    return bool(r)


def set_decode_path(path):
    """Process-wide decode kernel choice: 0 = library's choice, 1 = CUDA cores,
    2 = tensor cores where supported."""
    _lib.check(_lib.load().pkv_set_decode_path(int(path)), "pkv_set_decode_path")


def decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                          partition_size=0):
    """Bytes of scratch :func:`paged_attn_decode` needs (0 when it does not split)."""
    n = _lib.load().pkv_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                              max_context_len, partition_size)
    if n == _SIZE_T_MAX:
        raise ValueError("invalid decode sizes")
    return n


def paged_attn_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                      max_context_len, partition_size=0, workspace=None):
    """softmax(scale * q.K) V for every sequence and query head, K/V read
    through the block table.  Writes ``out`` ([S, Hq, D]) and returns it.

    ``workspace`` (uint8 CUDA tensor) is used when the context is split into
    partitions; if omitted and needed, one is allocated here with torch.
    """
    _cuda(q, "q", ndim=3)
    dtype = q.dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError("q must be float16 or bfloat16")
    _cuda(out, "out", dtype, 3)
    _cuda(k_cache, "k_cache", dtype, 4)
    _cuda(v_cache, "v_cache", dtype, 4)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    S, Hq, D = q.shape
    NB, Hkv, B, D2 = k_cache.shape
    if v_cache.shape != k_cache.shape or D2 != D or out.shape != q.shape:
        raise ValueError("shape mismatch between q, out and the caches")
    if block_tables.shape[0] != S or context_lens.shape[0] != S:
        raise ValueError("block_tables / context_lens must have one row per sequence")
    lib = _lib.load()
    ws_bytes = decode_workspace_size(S, Hq, Hkv, D, max_context_len, partition_size)
    ws_ptr, ws_len = None, 0
    if ws_bytes:
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        _cuda(workspace, "workspace")
        ws_ptr, ws_len = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib.pkv_paged_attn_decode(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(),
        int(max_context_len), S, Hq, Hkv, D, B, NB, float(scale), _DTYPE_CODE[dtype],
        int(partition_size), ws_ptr, ws_len, _stream_handle(q.device))
    _lib.check(st, "pkv_paged_attn_decode")
    return out


def paged_attn_decode_append(out, q, k_new, v_new, k_cache, v_cache, block_tables,
                             context_lens, scale, max_context_len, partition_size=0,
                             workspace=None):
    """One fused decode step: write each sequence's new token (``k_new``,
    ``v_new`` [S, Hkv, D], position ``context_lens[s] - 1``) into its slot and
    attend over the whole context in the same launch."""
    _cuda(q, "q", ndim=3)
    dtype = q.dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError("q must be float16 or bfloat16")
    for t, name in ((out, "out"), (k_new, "k_new"), (v_new, "v_new")):
        _cuda(t, name, dtype, 3)
    _cuda(k_cache, "k_cache", dtype, 4)
    _cuda(v_cache, "v_cache", dtype, 4)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    S, Hq, D = q.shape
    NB, Hkv, B, D2 = k_cache.shape
    if (v_cache.shape != k_cache.shape or D2 != D or out.shape != q.shape
            or k_new.shape != (S, Hkv, D) or v_new.shape != (S, Hkv, D)):
        raise ValueError("shape mismatch between q, out, new rows and the caches")
    if block_tables.shape[0] != S or context_lens.shape[0] != S:
        raise ValueError("block_tables / context_lens must have one row per sequence")
    lib = _lib.load()
    ws_bytes = decode_workspace_size(S, Hq, Hkv, D, max_context_len, partition_size)
    ws_ptr, ws_len = None, 0
    if ws_bytes:
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        _cuda(workspace, "workspace")
        ws_ptr, ws_len = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib.pkv_paged_attn_decode_append(
        out.data_ptr(), q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
        context_lens.data_ptr(), int(max_context_len), S, Hq, Hkv, D, B, NB, float(scale),
        _DTYPE_CODE[dtype], int(partition_size), ws_ptr, ws_len, _stream_handle(q.device))
    _lib.check(st, "pkv_paged_attn_decode_append")
    return out


def paged_attn_prefill(out, q, query_start, k_cache, v_cache, block_tables, context_lens, scale,
                       max_context_len, max_query_len):
    """Causal multi-query attention of each sequence's last L_s positions
    (``q[query_start[s]:query_start[s+1]]``) over its paged context, on the
    tensor cores.  Writes ``out`` ([total_queries, Hq, D]) and returns it."""
    _cuda(q, "q", ndim=3)
    dtype = q.dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError("q must be float16 or bfloat16")
    _cuda(out, "out", dtype, 3)
    _cuda(k_cache, "k_cache", dtype, 4)
    _cuda(v_cache, "v_cache", dtype, 4)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    _cuda(query_start, "query_start", torch.int32, 1)
    T, Hq, D = q.shape
    NB, Hkv, B, D2 = k_cache.shape
    S = context_lens.shape[0]
    if v_cache.shape != k_cache.shape or D2 != D or out.shape != q.shape:
        raise ValueError("shape mismatch between q, out and the caches")
    if block_tables.shape[0] != S or query_start.shape[0] != S + 1:
        raise ValueError("block_tables / query_start must match context_lens")
    st = _lib.load().pkv_paged_attn_prefill(
        out.data_ptr(), q.data_ptr(), T, query_start.data_ptr(), int(max_query_len),
        k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
        context_lens.data_ptr(), int(max_context_len), S, Hq, Hkv, D, B, NB, float(scale),
        _DTYPE_CODE[dtype], _stream_handle(q.device))
    _lib.check(st, "pkv_paged_attn_prefill")
    return out


def _same_device(first, *rest):
    """Index of the tensors' common CUDA device (None entries are skipped)."""
    index = first.get_device()
    if torch.cuda.device_count() > 1:  # (with one GPU there is no other)
        for t in rest:
            if t is not None and t.get_device() != index:
                raise ValueError("all tensors must be on one device")
    return index


def _workspace(workspace, size, like):
    """The caller's workspace, or one of ``size()`` bytes allocated here beside
    ``like``, an fp32 tensor (torch keeps its memory until the stream's work on
    it is done); and its address and bytes."""
    if workspace is None:
        workspace = like.new_empty((size() + 3) >> 2)
    else:
        _cuda(workspace, "workspace")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _attn_shapes(q, out, k_cache, v_cache):
    _cuda(q, "q", ndim=3)
    dtype = q.dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError("q must be float16 or bfloat16")
    _cuda(out, "out", dtype, 3)
    _cuda(k_cache, "k_cache", dtype, 4)
    _cuda(v_cache, "v_cache", dtype, 4)
    if v_cache.shape != k_cache.shape or k_cache.shape[3] != q.shape[2] or out.shape != q.shape:
        raise ValueError("shape mismatch between q, out and the caches")


def _weights(weights, num_seqs, num_kv_heads, max_context_len):
    _cuda(weights, "weights", torch.float32, 3)
    if (weights.shape[:2] != (num_seqs, num_kv_heads) or weights.shape[2] < max_context_len):
        raise ValueError("weights must be [num_seqs, num_kv_heads, >= max_context_len]")


def decode_weights_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                  partition_size=0):
    """Bytes of scratch :func:`paged_attn_decode_weights` needs."""
    n = _lib.load().pkv_decode_weights_workspace_size(
        num_seqs, num_q_heads, num_kv_heads, head_dim,
        _c_int(max_context_len, "max_context_len"), _c_int(partition_size, "partition_size"))
    if n == _SIZE_T_MAX:
        raise ValueError("invalid decode sizes")
    return n


def paged_attn_decode_weights(out, weights, q, k_cache, v_cache, block_tables, context_lens,
                              scale, max_context_len, decay=1.0, partition_size=0,
                              workspace=None):
    """:func:`paged_attn_decode` that also accumulates attention weights:
    ``weights`` (fp32 [S, Hkv, >= max_context_len]) becomes ``decay * weights``
    plus each held position's softmax weight, summed over the query heads of
    the KV head's group.  Groups of at most 32 query heads.  ``workspace`` (any
    CUDA tensor of at least :func:`decode_weights_workspace_size` bytes, which
    grow with ``max_context_len``, not with the contexts) is allocated here
    with torch if omitted.  Writes ``out`` and returns it."""
    _attn_shapes(q, out, k_cache, v_cache)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    S, Hq, D = q.shape
    NB, Hkv, B, _ = k_cache.shape
    _weights(weights, S, Hkv, max_context_len)
    if block_tables.shape[0] != S or context_lens.shape[0] != S:
        raise ValueError("block_tables / context_lens must have one row per sequence")
    dev = _same_device(q, out, weights, k_cache, v_cache, block_tables, context_lens, workspace)

    def size():
        sizes = (S, Hq, Hkv, D, max_context_len, partition_size)
        if dev == torch._C._cuda_getDevice():
            return decode_weights_workspace_size(*sizes)
        with torch.cuda.device(dev):
            return decode_weights_workspace_size(*sizes)

    workspace, ws_ptr, ws_len = _workspace(workspace, size, weights)
    _launch("pkv_paged_attn_decode_weights", dev, out.data_ptr(), weights.data_ptr(),
            weights.shape[2], float(decay), q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
            context_lens.data_ptr(), _c_int(max_context_len, "max_context_len"), S, Hq, Hkv, D, B,
            NB, float(scale), _DTYPE_CODE[q.dtype], _c_int(partition_size, "partition_size"),
            ws_ptr, ws_len)
    return out


def paged_attn_prefill_weights(out, weights, q, query_start, k_cache, v_cache, block_tables,
                               context_lens, scale, max_context_len, max_query_len, window=0,
                               decay=1.0, workspace=None):
    """:func:`paged_attn_prefill` that also accumulates attention weights:
    ``weights`` (fp32 [S, Hkv, >= max_context_len]) becomes ``decay * weights``
    plus each position's softmax weights, summed over the last ``window``
    queries of its sequence's chunk (0: all) and the query heads of the KV
    head's group.  ``workspace``: 4 bytes per query row and head (allocated
    here with torch if omitted).
    Writes ``out`` and returns it."""
    _attn_shapes(q, out, k_cache, v_cache)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    _cuda(query_start, "query_start", torch.int32, 1)
    T, Hq, D = q.shape
    NB, Hkv, B, _ = k_cache.shape
    S = context_lens.shape[0]
    _weights(weights, S, Hkv, max_context_len)
    if block_tables.shape[0] != S or query_start.shape[0] != S + 1:
        raise ValueError("block_tables / query_start must match context_lens")
    dev = _same_device(q, out, weights, query_start, k_cache, v_cache, block_tables,
                       context_lens, workspace)
    workspace, ws_ptr, ws_len = _workspace(
        workspace, lambda: _lib.load().pkv_prefill_weights_workspace_size(T, Hq), weights)
    _launch("pkv_paged_attn_prefill_weights", dev, out.data_ptr(), weights.data_ptr(),
            weights.shape[2], float(decay), _c_int(window, "window"), q.data_ptr(), T,
            query_start.data_ptr(), _c_int(max_query_len, "max_query_len"), k_cache.data_ptr(),
            v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
            context_lens.data_ptr(), _c_int(max_context_len, "max_context_len"), S, Hq, Hkv, D, B,
            NB, float(scale), _DTYPE_CODE[q.dtype], ws_ptr, ws_len)
    return out


def contiguous_attn_decode(out, q, k_cache, v_cache, context_lens, scale, partition_size=0,
                           workspace=None):
    """Decode over a contiguous cache ``[S, Hkv, capacity, D]`` (no block
    table): the baseline the paged layout is compared with.  It runs the
    CUDA-core decode kernel, whatever the decode-path setting."""
    _cuda(q, "q", ndim=3)
    dtype = q.dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError("q must be float16 or bfloat16")
    _cuda(out, "out", dtype, 3)
    _cuda(k_cache, "k_cache", dtype, 4)
    _cuda(v_cache, "v_cache", dtype, 4)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    S, Hq, D = q.shape
    S2, Hkv, cap, D2 = k_cache.shape
    if v_cache.shape != k_cache.shape or D2 != D or S2 != S or out.shape != q.shape:
        raise ValueError("shape mismatch between q, out and the caches")
    lib = _lib.load()
    ws_bytes = lib.pkv_contiguous_workspace_size(S, Hq, Hkv, D, cap, partition_size)
    if ws_bytes == _SIZE_T_MAX:
        raise ValueError("invalid decode sizes")
    ws_ptr, ws_len = None, 0
    if ws_bytes:
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        _cuda(workspace, "workspace")
        ws_ptr, ws_len = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib.pkv_contiguous_attn_decode(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        context_lens.data_ptr(), cap, S, Hq, Hkv, D, float(scale), _DTYPE_CODE[dtype],
        int(partition_size), ws_ptr, ws_len, _stream_handle(q.device))
    _lib.check(st, "pkv_contiguous_attn_decode")
    return out


def kv_append(k, v, k_cache, v_cache, slot_mapping):
    """Scatter token t's K/V ([T, Hkv, D]) into slot ``slot_mapping[t]`` (int64;
    negative = skip) of both caches."""
    _cuda(k, "k", ndim=3)
    dtype = k.dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError("k must be float16 or bfloat16")
    _cuda(v, "v", dtype, 3)
    _cuda(k_cache, "k_cache", dtype, 4)
    _cuda(v_cache, "v_cache", dtype, 4)
    _cuda(slot_mapping, "slot_mapping", torch.int64, 1)
    T, Hkv, D = k.shape
    NB, Hkv2, B, D2 = k_cache.shape
    if v.shape != k.shape or v_cache.shape != k_cache.shape or Hkv2 != Hkv or D2 != D:
        raise ValueError("shape mismatch between new tokens and the caches")
    if slot_mapping.shape[0] != T:
        raise ValueError("slot_mapping must have one entry per token")
    st = _lib.load().pkv_kv_append(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        slot_mapping.data_ptr(), T, Hkv, D, B, NB, _DTYPE_CODE[dtype], _stream_handle(k.device))
    _lib.check(st, "pkv_kv_append")


def _token_rows(t, name, dtype, shape):
    """Element stride between the tokens of a [T, H, D] tensor of this shape
    whose token rows are dense (a slice of a joint projection, say)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    T, H, D = shape
    s0, s1, s2 = t.stride()
    # (a dimension of one entry may carry any stride)
    if ((s2 != 1 and D > 1) or (s1 != D and H > 1)) and t.numel():
        raise ValueError(f"{name} must have dense token rows")
    return s0 if T > 1 else H * D


def rope_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original_len=None,
                     low=1.0, high=32.0, device="cuda"):
    """Frequencies ``base ** (-2i / rot_dim)`` in radians per position for
    :func:`rope_kv_append` (float64 [rot_dim / 2]), scaled for contexts
    ``factor`` times as long as the model was trained on:

    * ``None``: unscaled;
    * ``"linear"``: every frequency divided by ``factor`` (positions are
      interpolated);
    * ``"base"``: the base raised by ``factor ** (rot_dim / (rot_dim - 2))``,
      which leaves the highest frequency and divides the lowest by ``factor``;
    * ``"bands"``: frequencies that turn at least ``high`` times over
      ``original_len`` positions are kept, those that turn at most ``low``
      times are divided by ``factor``, and between them the two are mixed
      linearly in the number of turns.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    i = np.arange(0, rot_dim, 2, dtype=np.float64) / rot_dim
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("scaling the base needs rot_dim of at least 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = base ** -i
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "bands":
        if original_len is None or original_len <= 0 or not high > low:
            raise ValueError("bands need original_len above 0 and high above low")
        turns = original_len * freq / (2 * np.pi)
        kept = np.clip((turns - low) / (high - low), 0.0, 1.0)
        freq = freq * kept + freq / factor * (1.0 - kept)
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return torch.from_numpy(freq).to(device)


def rope_kv_append(q_out, q, k, v, positions, inv_freq, k_cache, v_cache, slot_mapping,
                   interleaved=False, attn_factor=1.0):
    """Rotary positions with append: ``q`` ([T, Hq, D]) turned into ``q_out``
    (which may be ``q``), ``k`` turned and ``v`` ([T, Hkv, D]) written into
    slot ``slot_mapping[t]`` (int64) of the caches.  ``positions`` (int32 [T]):
    negative = padding, nothing is written; a negative slot skips k and v
    only.  ``inv_freq``: float64 [rot_dim / 2] (:func:`rope_frequencies`);
    dimensions from rot_dim on pass through.  Pairs are neighbours if
    ``interleaved``, else rot_dim / 2 apart.  q, k, v and q_out may be slices
    of wider token rows.  Returns ``q_out``."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPE_CODE or q.dim() != 3:
        raise ValueError("q must be float16 or bfloat16 with 3 dimensions")
    dtype = q.dtype
    _cuda(k_cache, "k_cache", dtype, 4)
    _cuda(v_cache, "v_cache", dtype, 4)
    q_shape, cache_shape = q.shape, k_cache.shape
    T, Hq, D = q_shape
    NB, Hkv, B, D2 = cache_shape
    kv_shape = (T, Hkv, D)
    strides = (_token_rows(q_out, "q_out", dtype, q_shape), _token_rows(q, "q", dtype, q_shape),
               _token_rows(k, "k", dtype, kv_shape), _token_rows(v, "v", dtype, kv_shape))
    _cuda(positions, "positions", torch.int32, 1)
    _cuda(inv_freq, "inv_freq", torch.float64, 1)
    _cuda(slot_mapping, "slot_mapping", torch.int64, 1)
    if D2 != D or v_cache.shape != cache_shape:
        raise ValueError("shape mismatch between q and the caches")
    if positions.shape[0] != T or slot_mapping.shape[0] != T:
        raise ValueError("positions / slot_mapping must have one entry per token")
    dev = _same_device(q, q_out, k, v, positions, inv_freq, k_cache, v_cache, slot_mapping)
    _launch("pkv_rope_kv_append", dev, q_out.data_ptr(), strides[0], q.data_ptr(), strides[1],
            k.data_ptr(), strides[2], v.data_ptr(), strides[3], positions.data_ptr(),
            inv_freq.data_ptr(), 2 * inv_freq.shape[0], 1 if interleaved else 0,
            float(attn_factor), k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(),
            T, Hq, Hkv, D, B, NB, _DTYPE_CODE[dtype])
    return q_out


def kv_evict_select(keep, weights, context_lens, max_context_len, recent=0, sinks=0,
                    new_lens=None):
    """The positions each sequence and KV head keeps when it holds more than
    ``keep.shape[2]`` (``keep``: int32 [S, Hkv, budget], written): the first
    ``sinks``, the last ``recent`` and, of the others, those with the largest
    ``weights`` (fp32 [S, Hkv, >= max_context_len]; equal weights: the lowest
    positions), ascending, -1 past the end.  ``new_lens`` (int32 [S], not
    ``context_lens`` itself) receives the lengths after the eviction.  Returns
    ``keep``."""
    _cuda(keep, "keep", torch.int32, 3)
    S, Hkv, budget = keep.shape
    _weights(weights, S, Hkv, max_context_len)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    if new_lens is not None:
        _cuda(new_lens, "new_lens", torch.int32, 1)
    if context_lens.shape[0] != S or (new_lens is not None and new_lens.shape[0] != S):
        raise ValueError("context_lens / new_lens must have one entry per sequence")
    dev = _same_device(keep, weights, context_lens, new_lens)
    _launch("pkv_kv_evict_select", dev, keep.data_ptr(),
            None if new_lens is None else new_lens.data_ptr(), weights.data_ptr(),
            weights.shape[2], context_lens.data_ptr(),
            _c_int(max_context_len, "max_context_len"), S, Hkv, budget,
            _c_int(recent, "recent"), _c_int(sinks, "sinks"))
    return keep


def kv_compact(k_cache, v_cache, block_tables, keep, context_lens, weights=None,
               dst_tables=None, max_context_len=None):
    """Move the kept rows to each sequence's front: position i of (sequence s,
    KV head h) receives the K and V rows (and the weight) of position
    ``keep[s][h][i]``; the weights behind them become 0.  Rows move in place
    unless ``dst_tables`` names other blocks (``BlockAllocator.shrink_seqs``
    does for shared ones).  ``context_lens``: the lengths before the eviction,
    each at most ``max_context_len`` (default: what the tables and weights
    hold)."""
    _cuda(k_cache, "k_cache", ndim=4)
    dtype = k_cache.dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError("the caches must be float16 or bfloat16")
    _cuda(v_cache, "v_cache", dtype, 4)
    _cuda(block_tables, "block_tables", torch.int32, 2)
    _cuda(keep, "keep", torch.int32, 3)
    _cuda(context_lens, "context_lens", torch.int32, 1)
    if dst_tables is None:
        dst_tables = block_tables
    _cuda(dst_tables, "dst_tables", torch.int32, 2)
    NB, Hkv, B, D = k_cache.shape
    S, H2, budget = keep.shape
    if v_cache.shape != k_cache.shape or H2 != Hkv:
        raise ValueError("shape mismatch between keep and the caches")
    if block_tables.shape[0] != S or dst_tables.shape[0] != S or context_lens.shape[0] != S:
        raise ValueError("tables / context_lens must have one row per sequence")
    if max_context_len is None:
        max_context_len = block_tables.shape[1] * B
        if weights is not None:
            max_context_len = min(max_context_len, weights.shape[-1])
    if weights is not None:
        _weights(weights, S, Hkv, max_context_len)
    dev = _same_device(k_cache, v_cache, block_tables, keep, context_lens, weights, dst_tables)
    _launch("pkv_kv_compact", dev, k_cache.data_ptr(), v_cache.data_ptr(),
            None if weights is None else weights.data_ptr(),
            0 if weights is None else weights.shape[2], block_tables.data_ptr(),
            block_tables.shape[1], dst_tables.data_ptr(), dst_tables.shape[1], keep.data_ptr(),
            budget, context_lens.data_ptr(), _c_int(max_context_len, "max_context_len"), S, Hkv,
            D, B, NB, _DTYPE_CODE[dtype])


def check_copy_pairs(pairs, num_blocks):
    """Raise ValueError unless ``pairs`` ([P, 2] ids, host data) is a valid
    block_copy batch: ids in [0, num_blocks), destinations distinct, and no
    destination also a source (the pairs are copied in parallel)."""
    pairs = np.asarray(pairs, dtype=np.int64).reshape(-1, 2)
    if pairs.size and (pairs.min() < 0 or pairs.max() >= num_blocks):
        raise ValueError("block id outside [0, num_blocks)")
    dst = pairs[:, 1]
    if len(np.unique(dst)) != len(dst):
        raise ValueError("destinations must be distinct")
    if np.intersect1d(dst, pairs[:, 0]).size:
        raise ValueError("a destination is also a source")


def block_copy(k_cache, v_cache, src_dst_pairs, validate=False):
    """Copy whole physical blocks ``src -> dst`` (int64 [P, 2] CUDA tensor) in
    both caches.  ``validate=True`` reads the pairs back to the host and
    checks them first (see check_copy_pairs; this synchronises)."""
    _cuda(k_cache, "k_cache", ndim=4)
    _cuda(v_cache, "v_cache", k_cache.dtype, 4)
    _cuda(src_dst_pairs, "src_dst_pairs", torch.int64)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be [P, 2]")
    NB = k_cache.shape[0]
    if validate:
        check_copy_pairs(src_dst_pairs.cpu().numpy(), NB)
    block_bytes = k_cache[0].numel() * k_cache.element_size()
    st = _lib.load().pkv_block_copy(
        k_cache.data_ptr(), v_cache.data_ptr(), src_dst_pairs.data_ptr(),
        src_dst_pairs.shape[0], NB, block_bytes, _stream_handle(k_cache.device))
    _lib.check(st, "pkv_block_copy")


def debug_wait_timeout(device=None):
    """Enqueue one kernel whose bounded wait cannot complete: after the wait
    limit (2 s) it raises PKV_DEV_WAIT_TIMEOUT and ends (a check of the
    kernels' timeout path; the context stays usable)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _lib.check(_lib.load().pkv_debug_wait_timeout(_stream_handle(dev)), "pkv_debug_wait_timeout")


def device_status(clear=False, device=None):
    """Synchronise the current stream and return the device status flags."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    flags = ctypes.c_uint32(0)
    st = _lib.load().pkv_device_status(ctypes.byref(flags), 1 if clear else 0,
                                       _stream_handle(dev))
    _lib.check(st, "pkv_device_status")
    return flags.value
