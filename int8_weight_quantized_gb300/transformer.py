"""Binding of the operators around the linear layers: norms of queries and keys with the
position rotation, the paged key-value cache, attention over it (behind shared prefixes too) and
over whole prompts, its rows read back, the linear layer with 4-bit weights, low-rank adapters, and
log probabilities of tokens.

As in the rest of the package the functions have the C names and only marshal arguments; the
checks and allocations run in ``csrc/binding.cpp``.  Outputs and workspaces that the caller
does not give come from torch's allocator on the stream that the work is enqueued on, so
concurrent streams never share them.
"""
import collections
import ctypes
import importlib.machinery
import importlib.util
import os

import torch

import int8_weight_quantized_gb300 as ck
from . import build as _build

_CACHE_TYPES = (torch.bfloat16, torch.float16, torch.int8)
_EPS = 1e-6
_b = None


def _binding():
    """The compiled binding, on the loaded library's entry points (raises if not built)."""
    global _b
    if _b is None:
        L = ck.load_library()
        if not os.path.exists(_build.BINDING):
            raise RuntimeError("%s is not built; run `python -c 'import __graft_entry__ as g; g.build()'`" % _build.BINDING)
        loader = importlib.machinery.ExtensionFileLoader("_ck_binding", _build.BINDING)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_ck_binding", loader))
        loader.exec_module(module)
        module.init(*[ctypes.cast(getattr(L, n), ctypes.c_void_p).value
                      for n in ("ck_qk_norm_rope", "ck_paged_attention_workspace_size", "ck_paged_attention",
                                "ck_attention", "ck_int4_linear", "ck_prefix_attention_workspace_size",
                                "ck_prefix_attention", "ck_cache_read", "ck_adapter_linear_workspace_size",
                                "ck_adapter_linear", "ck_token_logprobs_workspace_size", "ck_token_logprobs")])
        _b = module
    return _b


class KVCache:
    """Keys and values in pages: k, v [num_pages, kv_heads, page_size, head_dim] of bf16, fp16
    or int8; int8 caches have fp32 k_scale, v_scale [num_pages, kv_heads, page_size].  (Shapes and
    types are checked by the calls that use the cache.)"""

    __slots__ = ("k", "v", "k_scale", "v_scale")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dtype not in _CACHE_TYPES:
            raise TypeError("a cache is bf16, fp16 or int8, got %s" % k.dtype)
        if k.dim() != 4:
            raise ValueError("k must have shape [num_pages, kv_heads, page_size, head_dim], got %s" % (tuple(k.shape),))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale

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

    @property
    def page_size(self):
        return self.k.shape[2]


def rope_table(max_pos, rot_dim, base=10000.0, device="cuda"):
    """The fp32 cos_sin table [max_pos, rot_dim] of ck_qk_norm_rope for the angles
    position * base^(-2i / rot_dim): rot_dim/2 cosines, then as many sines."""
    freq = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def ck_qk_norm_rope(qkv, positions, cos_sin, q_heads, kv_heads, q_weight=None, k_weight=None, eps=_EPS, norm=True,
                    interleaved=False, cache=None, slots=None, q=None, k=None, return_k=None, stream=None):
    """Norm and rotate the queries and keys of qkv [tokens, (q_heads + 2 kv_heads) * head_dim]
    (bf16 or fp16; rows may be strided) and put keys and values into `cache` at `slots` (int64
    [tokens]; negative: not cached).  positions int32 [tokens] index cos_sin fp32 [max_pos,
    rot_dim]; cos_sin None: no rotation.  Returns (q [tokens, q_heads, head_dim], k [tokens,
    kv_heads, head_dim] or None); k is returned if `k` or return_k says so, by default where
    there is no cache."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_qk_norm_rope(qkv, positions, cos_sin, q_heads, kv_heads, q_weight, k_weight, eps, norm, interleaved,
                                   cache, slots, q, k, return_k)
    if cache is None:
        r = (_b or _binding()).norm_rope(qkv, positions, cos_sin, q_heads, kv_heads, q_weight, k_weight, eps, norm,
                                         interleaved, None, None, None, None, None, q, k, return_k)
    else:
        r = (_b or _binding()).norm_rope(qkv, positions, cos_sin, q_heads, kv_heads, q_weight, k_weight, eps, norm,
                                         interleaved, cache.k, cache.v, cache.k_scale, cache.v_scale, slots, q, k,
                                         return_k)
    if r.__class__ is int:
        ck._check(r)
    return r


def ck_paged_attention(q, cache, block_table, seq_lens, scale=None, window=0, sinks=0, out=None, lse=None,
                       return_lse=False, ws=None, stream=None):
    """Attention of one new token per sequence: q [batch, q_heads, head_dim] over the cached
    keys that seq_lens int32 [batch] and block_table int32 [batch, max_blocks] name.  Returns
    out, or (out, lse fp32 [batch, q_heads]) with return_lse."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_paged_attention(q, cache, block_table, seq_lens, scale, window, sinks, out, lse, return_lse, ws)
    r = (_b or _binding()).paged_attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, block_table, seq_lens, scale,
                                           window, sinks, out, lse, return_lse, ws)
    if r.__class__ is int:
        ck._check(r)
    return r


def ck_prefix_attention(q, cache, prefix_table, prefix_lens, cu_prefix, block_table, seq_lens, scale=None, out=None,
                        lse=None, return_lse=False, ws=None, stream=None):
    """ck_paged_attention where sequences cu_prefix[i] .. cu_prefix[i + 1] - 1 (int32 [prefixes + 1]) also
    see the prefix_lens[i] keys of prefix i, whose pages prefix_table int32 [prefixes, max_prefix_blocks]
    names; block_table and seq_lens are each sequence's own tokens behind it."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_prefix_attention(q, cache, prefix_table, prefix_lens, cu_prefix, block_table, seq_lens, scale, out,
                                       lse, return_lse, ws)
    r = (_b or _binding()).prefix_attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, prefix_table, prefix_lens,
                                            cu_prefix, block_table, seq_lens, scale, out, lse, return_lse, ws)
    if r.__class__ is int:
        ck._check(r)
    return r


def ck_cache_read(cache, block_table, cu, total, dtype=None, k=None, v=None, stream=None):
    """Cached rows as contiguous (k, v), each [total, kv_heads, head_dim] of dtype (that of `k` or of a
    16-bit cache by default, else bf16): row cu[b] + t (cu int32 [batch + 1]) is token t of the sequence
    whose pages block_table int32 [batch, max_blocks] names.  Rows that no sequence has are left as
    they are (of new outputs: undefined)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_cache_read(cache, block_table, cu, total, dtype, k, v)
    if dtype is None:
        dtype = k.dtype if k is not None else torch.bfloat16 if cache.k.dtype == torch.int8 else cache.k.dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("dtype must be torch.bfloat16 or torch.float16, got %s" % (dtype,))
    r = (_b or _binding()).cache_read(cache.k, cache.v, cache.k_scale, cache.v_scale, block_table, cu, total,
                                      ck.OUT_DTYPES[dtype], k, v)
    if r.__class__ is int:
        ck._check(r)
    return r


def ck_attention(q, k, v, cu_q, cu_k=None, scale=None, causal=True, window=0, sinks=0, out=None, lse=None,
                 return_lse=False, stream=None):
    """Attention over whole prompts: q [total_q, q_heads, head_dim], k and v [total_k, kv_heads,
    head_dim] (token strides free), sequence b owning rows cu[b] .. cu[b+1] - 1 (int32; cu_k
    None: cu_q).  Returns out, or (out, lse fp32 [q_heads, total_q]) with return_lse."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_attention(q, k, v, cu_q, cu_k, scale, causal, window, sinks, out, lse, return_lse)
    r = (_b or _binding()).attention(q, k, v, cu_q, cu_k, scale, causal, window, sinks, out, lse, return_lse)
    if r.__class__ is int:
        ck._check(r)
    return r


def ck_int4_prepare_weight(W, group=128, w4=None, w_scale=None, stream=None):
    """fp32 W [N,K] -> (w4 int32 [N, K/8] packed codes, w_scale bf16 [N, K/group])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_int4_prepare_weight(W, group, w4, w_scale)
    N, K = W.shape
    ck._req(W, torch.float32, (N, K), "W")
    if group < 1 or K % group:
        raise ValueError("K must be a multiple of group (got K=%d group=%d)" % (K, group))
    w4 = torch.empty((N, K // 8), dtype=torch.int32, device=W.device) if w4 is None else w4
    w_scale = torch.empty((N, K // group), dtype=torch.bfloat16, device=W.device) if w_scale is None else w_scale
    ck._req(w4, torch.int32, (N, K // 8), "w4")
    ck._req(w_scale, torch.bfloat16, (N, K // group), "w_scale")
    ck._check(ck.load_library().ck_int4_prepare_weight(W.data_ptr(), N, K, group, w4.data_ptr(), w_scale.data_ptr(),
                                                       ck._stream(None)))
    return w4, w_scale


def ck_int4_pack(codes, w4=None, stream=None):
    """int8 codes [N,K] in [-8, 7] -> w4 int32 [N, K/8]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_int4_pack(codes, w4)
    N, K = codes.shape
    ck._req(codes, torch.int8, (N, K), "codes")
    w4 = torch.empty((N, K // 8), dtype=torch.int32, device=codes.device) if w4 is None else w4
    ck._req(w4, torch.int32, (N, K // 8), "w4")
    ck._check(ck.load_library().ck_int4_pack(codes.data_ptr(), N, K, w4.data_ptr(), ck._stream(None)))
    return w4


def ck_int4_linear(x, w4, w_scale, bias=None, residual=None, y=None, out_dtype=None, stream=None):
    """y [M,N] of out_dtype (x's type by default) = x [M,K] (bf16 or fp16) times the 4-bit
    weight w4 int32 [N, K/8] with scales w_scale bf16 [N, K/group] (+ bias) (+ residual);
    residual has y's type and shape and may be y itself."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_int4_linear(x, w4, w_scale, bias, residual, y, out_dtype)
    r = (_b or _binding()).int4_linear(x, w4, w_scale, bias, residual, y,
                                       -1 if out_dtype is None else ck._out_code(out_dtype))
    if r.__class__ is int:
        ck._check(r)
    return r


def ck_adapter_linear(x, a, b, index, scaling=None, residual=None, y=None, out_dtype=None, ws=None, stream=None):
    """y [M,N] of out_dtype (the residual's type by default, else x's) = residual + scaling[i] * (x[m] @ a[i].T)
    @ b[i].T with i = index[m] (int32 [M]; negative: none), for x [M,K], a [adapters, rank, K] and
    b [adapters, N, rank] of one 16-bit type, scaling fp32 [adapters]; residual may be y itself."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_adapter_linear(x, a, b, index, scaling, residual, y, out_dtype, ws)
    r = (_b or _binding()).adapter_linear(x, a, b, index, scaling, residual, y,
                                          -1 if out_dtype is None else ck._out_code(out_dtype), ws)
    if r.__class__ is int:
        ck._check(r)
    return r


TokenLogprobs = collections.namedtuple("TokenLogprobs", "logprob entropy lse top index")
TokenLogprobs.__doc__ = """What ck_token_logprobs returns: fp32 logprob (None without tokens), entropy and lse [rows],
fp32 log probabilities `top` and int32 `index` [rows, top] of the likeliest tokens (None for top=0)."""


def ck_token_logprobs(logits, tokens=None, top=0, scale=1.0, out=None, ws=None, stream=None):
    """Log probabilities of tokens int32 [rows] (negative: none, 0) under softmax(scale * logits), logits
    [rows, vocab] (bf16, fp16 or fp32; rows may be strided), with each row's entropy, log of the
    softmax's sum and `top` likeliest tokens.  Returns a TokenLogprobs, `out` itself where it is given (new ones
    share one allocation)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ck_token_logprobs(logits, tokens, top, scale, out, ws)
    given = (None,) * 5 if out is None else out
    r = (_b or _binding()).token_logprobs(logits, tokens, top, scale, *given, ws)
    if r.__class__ is int:
        ck._check(r)
    return TokenLogprobs(*r) if out is None else out
