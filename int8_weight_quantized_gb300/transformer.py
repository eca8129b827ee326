"""Binding of the operators around the linear layers: norms of queries and keys with the
position rotation, the paged key-value cache, attention over it and over whole prompts, and
the linear layer with 4-bit weights.

As in the rest of the package the functions have the C names and only marshal arguments.
Outputs and workspaces that the caller does not give come from torch's allocator on the
stream that the work is enqueued on, so concurrent streams never share them.
"""
import struct

import torch

import int8_weight_quantized_gb300 as ck

KV_BF16, KV_F16, KV_INT8 = 0, 1, 2
_ACT = {torch.bfloat16: 0, torch.float16: 1}
_KV = {torch.bfloat16: KV_BF16, torch.float16: KV_F16, torch.int8: KV_INT8}
_EPS = 1e-6


# ck_kv_cache_t: k, v, k_scale, v_scale, num_pages, page_size, kv_heads, head_dim, dtype
_CACHE = struct.Struct("@PPPPqqqqi")


class KVCache:
    """Keys and values in pages: k, v [num_pages, kv_heads, page_size, head_dim] of bf16, fp16
    or int8; int8 caches have fp32 k_scale, v_scale [num_pages, kv_heads, page_size]."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "page_size", "_struct", "_dim", "_heads")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        shape, dtype = k.shape, k.dtype
        if dtype not in _KV:
            raise TypeError("a cache is bf16, fp16 or int8, got %s" % dtype)
        if len(shape) != 4:
            raise ValueError("k must have shape [num_pages, kv_heads, page_size, head_dim], got %s" % (tuple(shape),))
        ck._req(k, dtype, shape, "k")
        ck._req(v, dtype, shape, "v")
        if dtype == torch.int8:
            if k_scale is None or v_scale is None:
                raise ValueError("an int8 cache needs k_scale and v_scale")
            ck._req(k_scale, torch.float32, shape[:3], "k_scale")
            ck._req(v_scale, torch.float32, shape[:3], "v_scale")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("only an int8 cache has scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        pages, self._heads, self.page_size, self._dim = shape
        self._struct = _CACHE.pack(k.data_ptr(), v.data_ptr(), ck._ptr(k_scale) or 0, ck._ptr(v_scale) or 0, pages,
                                   self.page_size, self._heads, self._dim, _KV[dtype])

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, dtype=torch.bfloat16, device="cuda"):
        """A cache of zeros."""
        shape = (num_pages, kv_heads, page_size, head_dim)
        scales = [torch.zeros(shape[:3], dtype=torch.float32, device=device) if dtype == torch.int8 else None
                  for _ in range(2)]
        return cls(torch.zeros(shape, dtype=dtype, device=device), torch.zeros(shape, dtype=dtype, device=device),
                   *scales)

    @property
    def num_pages(self):
        return self.k.shape[0]


def rope_table(max_pos, rot_dim, base=10000.0, device="cuda"):
    """The fp32 cos_sin table [max_pos, rot_dim] of ck_qk_norm_rope for the angles
    position * base^(-2i / rot_dim): rot_dim/2 cosines, then as many sines."""
    freq = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def _empty(shape, dtype, device, stream):
    # allocations belong to the stream that uses them
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _act(t, name):
    code = _ACT.get(t.dtype)
    if code is None:
        raise TypeError("%s must be torch.bfloat16 or torch.float16, got %s" % (name, t.dtype))
    return code


def _rows(t, dtype, dim, name):
    """Token stride in elements of t [tokens, heads, dim], whose rows are dense."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor of shape [tokens, heads, %d], got %s" % (name, dim, tuple(shape)))
    stride = t.stride()
    if (stride[2] != 1 and dim > 1) or (stride[1] != dim and shape[1] > 1):
        raise ValueError("the heads of a token must be contiguous in %s" % name)
    return stride[0] if shape[0] > 1 else max(stride[0], shape[1] * dim)


def ck_qk_norm_rope(qkv, positions, cos_sin, q_heads, kv_heads, q_weight=None, k_weight=None, eps=_EPS, norm=True,
                    interleaved=False, cache=None, slots=None, q=None, k=None, return_k=None, stream=None):
    """Norm and rotate the queries and keys of qkv [tokens, (q_heads + 2 kv_heads) * head_dim]
    (bf16 or fp16; rows may be strided) and put keys and values into `cache` at `slots` (int64
    [tokens]; negative: not cached).  positions int32 [tokens] index cos_sin fp32 [max_pos,
    rot_dim]; cos_sin None: no rotation.  Returns (q [tokens, q_heads, head_dim], k [tokens,
    kv_heads, head_dim] or None); k is returned if `k` or return_k says so, by default where
    there is no cache."""
    code = _act(qkv, "qkv")
    dtype = qkv.dtype
    stride = qkv.stride()
    if len(stride) != 2 or stride[1] != 1 or not qkv.is_cuda:
        raise ValueError("qkv must be a CUDA tensor [tokens, (q_heads + 2 kv_heads) * head_dim] with dense rows")
    tokens, width = qkv.shape
    heads = q_heads + 2 * kv_heads
    dim = width // heads if heads > 0 else 0
    if dim * heads != width:
        raise ValueError("qkv rows of %d values do not divide into %d + 2 * %d heads" % (width, q_heads, kv_heads))
    rot = max_pos = 0
    if cos_sin is not None:
        max_pos, rot = cos_sin.shape
        ck._req(cos_sin, torch.float32, (max_pos, rot), "cos_sin")
        ck._req(positions, torch.int32, (tokens,), "positions")
    else:
        positions = None
    if q_weight is not None:
        ck._req(q_weight, dtype, (dim,), "q_weight")
    if k_weight is not None:
        ck._req(k_weight, dtype, (dim,), "k_weight")
    if cache is not None:
        ck._req(slots, torch.int64, (tokens,), "slots")
    if q is None:
        q = _empty((tokens, q_heads, dim), dtype, qkv.device, stream)
    else:
        ck._req(q, dtype, (tokens, q_heads, dim), "q")
    if k is not None:
        ck._req(k, dtype, (tokens, kv_heads, dim), "k")
    elif return_k or (return_k is None and cache is None):
        k = _empty((tokens, kv_heads, dim), dtype, qkv.device, stream)
    stride = stride[0] if tokens > 1 else max(stride[0], width)
    status = (ck._lib or ck.load_library()).ck_qk_norm_rope(
        qkv.data_ptr(), stride, tokens, q_heads, kv_heads, dim, code, 1 if norm else 0, ck._ptr(q_weight),
        ck._ptr(k_weight), eps, rot, 1 if interleaved else 0, ck._ptr(positions), ck._ptr(cos_sin), max_pos,
        q.data_ptr(), ck._ptr(k), None if cache is None else cache._struct, ck._ptr(slots), ck._stream(stream))
    if status:
        ck._check(status)
    return q, k


def ck_paged_attention(q, cache, block_table, seq_lens, scale=None, window=0, sinks=0, out=None, lse=None,
                       return_lse=False, ws=None, stream=None):
    """Attention of one new token per sequence: q [batch, q_heads, head_dim] over the cached
    keys that seq_lens int32 [batch] and block_table int32 [batch, max_blocks] name.  Returns
    out, or (out, lse fp32 [batch, q_heads]) with return_lse."""
    code = _act(q, "q")
    batch, heads, dim = q.shape
    stride = _rows(q, q.dtype, dim, "q")
    max_blocks = block_table.shape[-1]
    ck._req(block_table, torch.int32, (batch, max_blocks), "block_table")
    ck._req(seq_lens, torch.int32, (batch,), "seq_lens")
    if cache._dim != dim:
        raise ValueError("q has heads of %d values, the cache of %d" % (dim, cache._dim))
    L = ck._lib or ck.load_library()
    if out is None:
        out = _empty((batch, heads, dim), q.dtype, q.device, stream)
    else:
        ck._req(out, q.dtype, (batch, heads, dim), "out")
    if lse is not None:
        ck._req(lse, torch.float32, (batch, heads), "lse")
    elif return_lse:
        lse = _empty((batch, heads), torch.float32, q.device, stream)
    if ws is None:
        need = L.ck_paged_attention_workspace_size(batch, heads, cache._heads, dim, max_blocks * cache.page_size)
        if need:
            ws = _empty(need, torch.uint8, q.device, stream)
    status = L.ck_paged_attention(
        q.data_ptr(), stride, cache._struct, block_table.data_ptr(), max_blocks, seq_lens.data_ptr(), batch, heads, code,
        dim ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(), ck._ptr(lse), ck._ptr(ws),
        0 if ws is None else ws.numel(), ck._stream(stream))
    if status:
        ck._check(status)
    return (out, lse) if return_lse else out


def ck_attention(q, k, v, cu_q, cu_k=None, scale=None, causal=True, window=0, sinks=0, out=None, lse=None,
                 return_lse=False, stream=None):
    """Attention over whole prompts: q [total_q, q_heads, head_dim], k and v [total_k, kv_heads,
    head_dim] (token strides free), sequence b owning rows cu[b] .. cu[b+1] - 1 (int32; cu_k
    None: cu_q).  Returns out, or (out, lse fp32 [q_heads, total_q]) with return_lse."""
    code = _act(q, "q")
    total_q, heads, dim = q.shape
    total_k, kv_heads = k.shape[:2]
    dtype = q.dtype
    strides = _rows(q, dtype, dim, "q"), _rows(k, dtype, dim, "k"), _rows(v, dtype, dim, "v")
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape, got %s and %s" % (tuple(k.shape), tuple(v.shape)))
    cu_k = cu_q if cu_k is None else cu_k
    batch = cu_q.shape[0] - 1
    if batch < 0:
        raise ValueError("cu_q must hold batch + 1 bounds, got none")
    ck._req(cu_q, torch.int32, (batch + 1,), "cu_q")
    if cu_k is not cu_q:
        ck._req(cu_k, torch.int32, (batch + 1,), "cu_k")
    if out is None:
        out = _empty((total_q, heads, dim), q.dtype, q.device, stream)
    else:
        ck._req(out, q.dtype, (total_q, heads, dim), "out")
    if lse is not None:
        ck._req(lse, torch.float32, (heads, total_q), "lse")
    elif return_lse:
        lse = _empty((heads, total_q), torch.float32, q.device, stream)
    status = (ck._lib or ck.load_library()).ck_attention(
        q.data_ptr(), strides[0], k.data_ptr(), strides[1], v.data_ptr(), strides[2], cu_q.data_ptr(),
        cu_k.data_ptr(), batch, total_q, total_k, heads, kv_heads, dim, code, dim ** -0.5 if scale is None else scale,
        1 if causal else 0, window, sinks, out.data_ptr(), ck._ptr(lse), ck._stream(stream))
    if status:
        ck._check(status)
    return (out, lse) if return_lse else out


def ck_int4_prepare_weight(W, group=128, w4=None, w_scale=None, stream=None):
    """fp32 W [N,K] -> (w4 int32 [N, K/8] packed codes, w_scale bf16 [N, K/group])."""
    N, K = W.shape
    ck._req(W, torch.float32, (N, K), "W")
    if group < 1 or K % group:
        raise ValueError("K must be a multiple of group (got K=%d group=%d)" % (K, group))
    w4 = _empty((N, K // 8), torch.int32, W.device, stream) if w4 is None else w4
    w_scale = _empty((N, K // group), torch.bfloat16, W.device, stream) if w_scale is None else w_scale
    ck._req(w4, torch.int32, (N, K // 8), "w4")
    ck._req(w_scale, torch.bfloat16, (N, K // group), "w_scale")
    ck._check(ck.load_library().ck_int4_prepare_weight(W.data_ptr(), N, K, group, w4.data_ptr(), w_scale.data_ptr(),
                                                       ck._stream(stream)))
    return w4, w_scale


def ck_int4_pack(codes, w4=None, stream=None):
    """int8 codes [N,K] in [-8, 7] -> w4 int32 [N, K/8]."""
    N, K = codes.shape
    ck._req(codes, torch.int8, (N, K), "codes")
    w4 = _empty((N, K // 8), torch.int32, codes.device, stream) if w4 is None else w4
    ck._req(w4, torch.int32, (N, K // 8), "w4")
    ck._check(ck.load_library().ck_int4_pack(codes.data_ptr(), N, K, w4.data_ptr(), ck._stream(stream)))
    return w4


def ck_int4_linear(x, w4, w_scale, bias=None, residual=None, y=None, out_dtype=None, stream=None):
    """y [M,N] of out_dtype (x's type by default) = x [M,K] (bf16 or fp16) times the 4-bit
    weight w4 int32 [N, K/8] with scales w_scale bf16 [N, K/group] (+ bias) (+ residual);
    residual has y's type and shape and may be y itself."""
    code = _act(x, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    out_code = ck._out_code(out_dtype)
    M, K = x.shape
    N, groups = w_scale.shape
    ck._req(x, x.dtype, (M, K), "x")
    ck._req(w4, torch.int32, (N, K // 8), "w4")
    ck._req(w_scale, torch.bfloat16, (N, groups), "w_scale")
    if groups < 1 or K % groups:
        raise ValueError("K=%d does not divide into %d groups" % (K, groups))
    if bias is not None:
        ck._req(bias, x.dtype, (N,), "bias")
    if y is None:
        y = _empty((M, N), out_dtype, x.device, stream)
    else:
        ck._req(y, out_dtype, (M, N), "y")
    if residual is not None:
        ck._req(residual, out_dtype, (M, N), "residual")
    status = (ck._lib or ck.load_library()).ck_int4_linear(
        x.data_ptr(), w4.data_ptr(), w_scale.data_ptr(), ck._ptr(bias), ck._ptr(residual), y.data_ptr(), M, N, K,
        K // groups, code, out_code, ck._stream(stream))
    if status:
        ck._check(status)
    return y
