// binding.cpp -- the Python side of the operators around the linear layers: checks the tensors,
// allocates the outputs that the caller did not give, and calls the C ABI on the current stream.
// (In Python with ctypes a call of these took 10-17 us of host time, several times what their
// smallest launches take on the GPU.)
#include <Python.h>

#include <cstdint>
#include <string>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ck_int8.h"

namespace {

// The library's entry points: their addresses come from the loaded library (init()).
decltype(&ck_qk_norm_rope) p_norm_rope = nullptr;
decltype(&ck_paged_attention_workspace_size) p_paged_ws = nullptr;
decltype(&ck_paged_attention) p_paged = nullptr;
decltype(&ck_attention) p_attention = nullptr;
decltype(&ck_int4_linear) p_int4 = nullptr;
decltype(&ck_prefix_attention_workspace_size) p_prefix_ws = nullptr;
decltype(&ck_prefix_attention) p_prefix = nullptr;
decltype(&ck_cache_read) p_cache_read = nullptr;
decltype(&ck_adapter_linear_workspace_size) p_adapter_ws = nullptr;
decltype(&ck_adapter_linear) p_adapter = nullptr;
decltype(&ck_token_logprobs_workspace_size) p_logprobs_ws = nullptr;
decltype(&ck_token_logprobs) p_logprobs = nullptr;

// A Python exception to raise, thrown through the checks.
struct Raise {
    PyObject* type;
    std::string text;
};

[[noreturn]] void type_error(const std::string& text)
{
    throw Raise{PyExc_TypeError, text};
}
[[noreturn]] void value_error(const std::string& text)
{
    throw Raise{PyExc_ValueError, text};
}

std::string shape_text(c10::IntArrayRef s)
{
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i)
        r += std::to_string(s[i]) + (s.size() == 1 ? "," : i + 1 < s.size() ? ", " : "");
    return r + ")";
}

const char* type_name(at::ScalarType t)
{
    switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kChar: return "torch.int8";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
    }
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o))
        type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// nullptr where the argument is None
const at::Tensor* optional_tensor(PyObject* o, const char* name)
{
    return o == Py_None ? nullptr : &tensor(o, name);
}

void require_type(const at::Tensor& t, at::ScalarType type, const char* name)
{
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
}

// a dense CUDA tensor of that type and shape
void require(const at::Tensor& t, at::ScalarType type, c10::IntArrayRef shape, const char* name)
{
    require_type(t, type, name);
    if (t.sizes() != shape)
        value_error(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    if (!t.is_contiguous())
        value_error(std::string(name) + " must be contiguous");
    if (!t.is_cuda())
        value_error(std::string(name) + " must be a CUDA tensor");
}

int act_type(const at::Tensor& t, const char* name)
{
    if (t.scalar_type() == at::kBFloat16)
        return CK_OUT_BF16;
    if (t.scalar_type() == at::kHalf)
        return CK_OUT_F16;
    type_error(std::string(name) + " must be torch.bfloat16 or torch.float16, got " + type_name(t.scalar_type()));
}

// Elements between the tokens of t [tokens, heads, dim], whose rows are dense.  (Of one token there is
// none, whatever the tensor says.)
int64_t token_stride(const at::Tensor& t, at::ScalarType type, int64_t dim, const char* name)
{
    require_type(t, type, name);
    if (t.dim() != 3 || t.size(2) != dim || !t.is_cuda())
        value_error(std::string(name) + " must be a CUDA tensor of shape [tokens, heads, " + std::to_string(dim) + "], got " +
                    shape_text(t.sizes()));
    if ((t.stride(2) != 1 && dim > 1) || (t.stride(1) != dim && t.size(1) > 1))
        value_error(std::string("the heads of a token must be contiguous in ") + name);
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * dim;
}

int64_t integer(PyObject* o, const char* name)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    return v;
}

double number(PyObject* o, const char* name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be a number");
    }
    return v;
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        type_error("expected a truth value");
    }
    return v != 0;
}

at::Tensor empty(c10::IntArrayRef shape, at::ScalarType type, const at::Tensor& like)
{
    // what at::empty comes to for a CUDA tensor, without the dispatcher's way there
    return at::detail::empty_cuda(shape, type, like.device(), c10::nullopt);
}

void* ptr(const at::Tensor* t)
{
    return t ? t->data_ptr() : nullptr;
}

void* current_stream(const at::Tensor& t)
{
    return c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
}

PyObject* wrapped(const at::Tensor& t)
{
    return THPVariable_Wrap(t);
}

// The argument itself where the caller gave the output, else the new tensor.
PyObject* given_or(PyObject* given, const at::Tensor& made)
{
    if (given == Py_None)
        return wrapped(made);
    Py_INCREF(given);
    return given;
}

// cache: None, or a KVCache's (k, v, k_scale, v_scale) with the shape checks of a call
struct Cache {
    ck_kv_cache_t c{};
    bool there = false;
};

Cache cache_of(PyObject* k_, PyObject* v_, PyObject* ks_, PyObject* vs_)
{
    Cache r;
    if (k_ == Py_None)
        return r;
    const at::Tensor &k = tensor(k_, "k"), &v = tensor(v_, "v");
    const at::ScalarType type = k.scalar_type();
    const int dtype = type == at::kBFloat16 ? CK_KV_BF16 : type == at::kHalf ? CK_KV_F16 : type == at::kChar ? CK_KV_INT8 : -1;
    if (dtype < 0)
        type_error(std::string("a cache is bf16, fp16 or int8, got ") + type_name(type));
    if (k.dim() != 4)
        value_error("k must have shape [num_pages, kv_heads, page_size, head_dim], got " + shape_text(k.sizes()));
    require(k, type, k.sizes(), "k");
    require(v, type, k.sizes(), "v");
    const at::Tensor *ks = optional_tensor(ks_, "k_scale"), *vs = optional_tensor(vs_, "v_scale");
    if (dtype == CK_KV_INT8) {
        if (!ks || !vs)
            value_error("an int8 cache needs k_scale and v_scale");
        require(*ks, at::kFloat, k.sizes().slice(0, 3), "k_scale");
        require(*vs, at::kFloat, k.sizes().slice(0, 3), "v_scale");
    } else if (ks || vs) {
        value_error("only an int8 cache has scales");
    }
    r.c.k = k.data_ptr();
    r.c.v = v.data_ptr();
    r.c.k_scale = static_cast<float*>(ptr(ks));
    r.c.v_scale = static_cast<float*>(ptr(vs));
    r.c.num_pages = k.size(0);
    r.c.kv_heads = k.size(1);
    r.c.page_size = k.size(2);
    r.c.head_dim = k.size(3);
    r.c.dtype = dtype;
    r.there = true;
    return r;
}

// Every function returns its outputs, or the library's status as an int where that is not CK_OK.
template <class Fn>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, Fn fn)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
        return nullptr;
    }
    try {
        return fn();
    } catch (const Raise& r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const c10::OutOfMemoryError& e) {  // as torch raises it, for callers that catch it
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type)
            PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded("init", n, 12, [&]() -> PyObject* {
        void* f[12];
        for (int i = 0; i < 12; ++i)
            f[i] = reinterpret_cast<void*>(static_cast<intptr_t>(integer(a[i], "address")));
        p_norm_rope = reinterpret_cast<decltype(p_norm_rope)>(f[0]);
        p_paged_ws = reinterpret_cast<decltype(p_paged_ws)>(f[1]);
        p_paged = reinterpret_cast<decltype(p_paged)>(f[2]);
        p_attention = reinterpret_cast<decltype(p_attention)>(f[3]);
        p_int4 = reinterpret_cast<decltype(p_int4)>(f[4]);
        p_prefix_ws = reinterpret_cast<decltype(p_prefix_ws)>(f[5]);
        p_prefix = reinterpret_cast<decltype(p_prefix)>(f[6]);
        p_cache_read = reinterpret_cast<decltype(p_cache_read)>(f[7]);
        p_adapter_ws = reinterpret_cast<decltype(p_adapter_ws)>(f[8]);
        p_adapter = reinterpret_cast<decltype(p_adapter)>(f[9]);
        p_logprobs_ws = reinterpret_cast<decltype(p_logprobs_ws)>(f[10]);
        p_logprobs = reinterpret_cast<decltype(p_logprobs)>(f[11]);
        Py_RETURN_NONE;
    });
}

// qkv, positions, cos_sin, q_heads, kv_heads, q_weight, k_weight, eps, norm, interleaved,
// cache k, v, k_scale, v_scale, slots, q, k, return_k -> (q, k)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded("norm_rope", n, 18, [&]() -> PyObject* {
        const at::Tensor& qkv = tensor(a[0], "qkv");
        const int dtype = act_type(qkv, "qkv");
        const at::ScalarType type = qkv.scalar_type();
        if (qkv.dim() != 2 || qkv.stride(1) != 1 || !qkv.is_cuda())
            value_error("qkv must be a CUDA tensor [tokens, (q_heads + 2 kv_heads) * head_dim] with dense rows");
        const int64_t tokens = qkv.size(0), width = qkv.size(1);
        const int64_t hq = integer(a[3], "q_heads"), hkv = integer(a[4], "kv_heads");
        const int64_t heads = hq > 0 && hkv > 0 && hq < (1 << 20) && hkv < (1 << 20) ? hq + 2 * hkv : 0;
        const int64_t dim = heads > 0 ? width / heads : 0;
        if (heads <= 0 || dim * heads != width)
            value_error("qkv rows of " + std::to_string(width) + " values do not divide into " + std::to_string(hq) +
                        " + 2 * " + std::to_string(hkv) + " heads");
        const at::Tensor *table = optional_tensor(a[2], "cos_sin"), *positions = nullptr;
        int64_t max_pos = 0, rot = 0;
        if (table) {
            if (table->dim() != 2)
                value_error("cos_sin must have shape [max_pos, rot_dim], got " + shape_text(table->sizes()));
            require(*table, at::kFloat, table->sizes(), "cos_sin");
            max_pos = table->size(0), rot = table->size(1);
            positions = &tensor(a[1], "positions");
            require(*positions, at::kInt, {tokens}, "positions");
        }
        const at::Tensor *qw = optional_tensor(a[5], "q_weight"), *kw = optional_tensor(a[6], "k_weight");
        if (qw)
            require(*qw, type, {dim}, "q_weight");
        if (kw)
            require(*kw, type, {dim}, "k_weight");
        const Cache cache = cache_of(a[10], a[11], a[12], a[13]);
        const at::Tensor* slots = nullptr;
        if (cache.there) {
            slots = &tensor(a[14], "slots");
            require(*slots, at::kLong, {tokens}, "slots");
        }
        at::Tensor q, k;
        if (a[15] == Py_None)
            q = empty({tokens, hq, dim}, type, qkv);
        else
            require(q = tensor(a[15], "q"), type, {tokens, hq, dim}, "q");
        const bool want_k = a[16] != Py_None || (a[17] == Py_None ? !cache.there : truth(a[17]));
        if (a[16] != Py_None)
            require(k = tensor(a[16], "k"), type, {tokens, hkv, dim}, "k");
        else if (want_k)
            k = empty({tokens, hkv, dim}, type, qkv);
        const int64_t stride = tokens > 1 ? qkv.stride(0) : width;
        const int st = p_norm_rope(qkv.data_ptr(), stride, tokens, hq, hkv, dim, dtype, truth(a[8]) ? 1 : 0, ptr(qw), ptr(kw),
                                   (float)number(a[7], "eps"), rot, truth(a[9]) ? 1 : 0,
                                   static_cast<const int32_t*>(ptr(positions)), static_cast<const float*>(ptr(table)), max_pos,
                                   q.data_ptr(), want_k ? k.data_ptr() : nullptr, cache.there ? &cache.c : nullptr,
                                   static_cast<const int64_t*>(ptr(slots)), current_stream(qkv));
        if (st != CK_OK)
            return PyLong_FromLong(st);
        PyObject* qo = given_or(a[15], q);
        PyObject* ko = want_k ? given_or(a[16], k) : Py_NewRef(Py_None);
        PyObject* r = PyTuple_Pack(2, qo, ko);
        Py_DECREF(qo);
        Py_DECREF(ko);
        return r;
    });
}

// q, cache k, v, k_scale, v_scale, block_table, seq_lens, scale, window, sinks, out, lse,
// return_lse, ws -> out, or (out, lse)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded("paged_attention", n, 14, [&]() -> PyObject* {
        const at::Tensor& q = tensor(a[0], "q");
        const int dtype = act_type(q, "q");
        const at::ScalarType type = q.scalar_type();
        const int64_t dim = q.dim() == 3 ? q.size(2) : 0;
        const int64_t stride = token_stride(q, type, dim, "q");
        const int64_t batch = q.size(0), heads = q.size(1);
        const Cache cache = cache_of(a[1], a[2], a[3], a[4]);
        if (!cache.there)
            type_error("cache must be a KVCache");
        if (cache.c.head_dim != dim)
            value_error("q has heads of " + std::to_string(dim) + " values, the cache of " + std::to_string(cache.c.head_dim));
        const at::Tensor &table = tensor(a[5], "block_table"), &lens = tensor(a[6], "seq_lens");
        const int64_t blocks = table.dim() == 2 ? table.size(1) : 0;
        require(table, at::kInt, {batch, blocks}, "block_table");
        require(lens, at::kInt, {batch}, "seq_lens");
        at::Tensor out, lse, ws;
        if (a[10] == Py_None)
            out = empty({batch, heads, dim}, type, q);
        else
            require(out = tensor(a[10], "out"), type, {batch, heads, dim}, "out");
        const bool return_lse = truth(a[12]);
        if (a[11] != Py_None)
            require(lse = tensor(a[11], "lse"), at::kFloat, {batch, heads}, "lse");
        else if (return_lse)
            lse = empty({batch, heads}, at::kFloat, q);
        int64_t ws_bytes = 0;
        if (a[13] != Py_None) {
            ws = tensor(a[13], "ws");
            require(ws, at::kByte, {ws.numel()}, "ws");
            ws_bytes = ws.numel();
        } else if (blocks > 0 && cache.c.page_size > 0 && blocks < (int64_t(1) << 40) / cache.c.page_size) {
            ws_bytes = (int64_t)p_paged_ws(batch, heads, cache.c.kv_heads, dim, blocks * cache.c.page_size);
            if (ws_bytes > 0)
                ws = empty({ws_bytes}, at::kByte, q);
        }
        const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)std::max<int64_t>(dim, 1)))
                                            : (float)number(a[7], "scale");
        const int st = p_paged(q.data_ptr(), stride, &cache.c, table.data_ptr<int32_t>(), blocks, lens.data_ptr<int32_t>(),
                               batch, heads, dtype, scale, integer(a[8], "window"), integer(a[9], "sinks"), out.data_ptr(),
                               lse.defined() ? lse.data_ptr<float>() : nullptr, ws.defined() ? ws.data_ptr() : nullptr,
                               (size_t)ws_bytes, current_stream(q));
        if (st != CK_OK)
            return PyLong_FromLong(st);
        PyObject* o = given_or(a[10], out);
        if (!return_lse)
            return o;
        PyObject* l = given_or(a[11], lse);
        PyObject* r = PyTuple_Pack(2, o, l);
        Py_DECREF(o);
        Py_DECREF(l);
        return r;
    });
}

// A workspace of `bytes` bytes, or the caller's own (whose size the library checks).
void* workspace_of(PyObject* given, size_t* bytes, const at::Tensor& like, at::Tensor* ws)
{
    if (given != Py_None) {
        *ws = tensor(given, "ws");
        require(*ws, at::kByte, {ws->numel()}, "ws");
        *bytes = (size_t)ws->numel();
    } else if (*bytes > 0) {
        *ws = empty({(int64_t)*bytes}, at::kByte, like);
    }
    return ws->defined() ? ws->data_ptr() : nullptr;
}

// q, cache k, v, k_scale, v_scale, prefix_table, prefix_lens, cu_prefix, block_table, seq_lens, scale, out,
// lse, return_lse, ws -> out, or (out, lse)
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded("prefix_attention", n, 15, [&]() -> PyObject* {
        const at::Tensor& q = tensor(a[0], "q");
        const int dtype = act_type(q, "q");
        const at::ScalarType type = q.scalar_type();
        const int64_t dim = q.dim() == 3 ? q.size(2) : 0;
        const int64_t stride = token_stride(q, type, dim, "q");
        const int64_t batch = q.size(0), heads = q.size(1);
        const Cache cache = cache_of(a[1], a[2], a[3], a[4]);
        if (!cache.there)
            type_error("cache must be a KVCache");
        if (cache.c.head_dim != dim)
            value_error("q has heads of " + std::to_string(dim) + " values, the cache of " + std::to_string(cache.c.head_dim));
        const at::Tensor &ptable = tensor(a[5], "prefix_table"), &plens = tensor(a[6], "prefix_lens"),
                         &cu = tensor(a[7], "cu_prefix"), &table = tensor(a[8], "block_table"),
                         &lens = tensor(a[9], "seq_lens");
        const int64_t prefixes = ptable.dim() == 2 ? ptable.size(0) : 0, pblocks = ptable.dim() == 2 ? ptable.size(1) : 0;
        const int64_t blocks = table.dim() == 2 ? table.size(1) : 0;
        require(ptable, at::kInt, {prefixes, pblocks}, "prefix_table");
        require(plens, at::kInt, {prefixes}, "prefix_lens");
        require(cu, at::kInt, {prefixes + 1}, "cu_prefix");
        require(table, at::kInt, {batch, blocks}, "block_table");
        require(lens, at::kInt, {batch}, "seq_lens");
        at::Tensor out, lse, ws;
        if (a[11] == Py_None)
            out = empty({batch, heads, dim}, type, q);
        else
            require(out = tensor(a[11], "out"), type, {batch, heads, dim}, "out");
        const bool return_lse = truth(a[13]);
        if (a[12] != Py_None)
            require(lse = tensor(a[12], "lse"), at::kFloat, {batch, heads}, "lse");
        else if (return_lse)
            lse = empty({batch, heads}, at::kFloat, q);
        const int64_t most = cache.c.page_size > 0 ? (int64_t(1) << 31) / cache.c.page_size : 0;
        size_t ws_bytes = blocks < most && pblocks < most
                              ? p_prefix_ws(batch, heads, cache.c.kv_heads, dim, prefixes, pblocks * cache.c.page_size,
                                            blocks * cache.c.page_size)
                              : 0;
        void* ws_ptr = workspace_of(a[14], &ws_bytes, q, &ws);
        const float scale = a[10] == Py_None ? (float)(1.0 / std::sqrt((double)std::max<int64_t>(dim, 1)))
                                             : (float)number(a[10], "scale");
        const int st = p_prefix(q.data_ptr(), stride, &cache.c, ptable.data_ptr<int32_t>(), pblocks,
                                plens.data_ptr<int32_t>(), cu.data_ptr<int32_t>(), prefixes, table.data_ptr<int32_t>(), blocks,
                                lens.data_ptr<int32_t>(), batch, heads, dtype, scale, out.data_ptr(),
                                lse.defined() ? lse.data_ptr<float>() : nullptr, ws_ptr, ws_bytes, current_stream(q));
        if (st != CK_OK)
            return PyLong_FromLong(st);
        PyObject* o = given_or(a[11], out);
        if (!return_lse)
            return o;
        PyObject* l = given_or(a[12], lse);
        PyObject* r = PyTuple_Pack(2, o, l);
        Py_DECREF(o);
        Py_DECREF(l);
        return r;
    });
}

// cache k, v, k_scale, v_scale, block_table, cu, total, dtype, k, v -> (k, v)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded("cache_read", n, 10, [&]() -> PyObject* {
        const Cache cache = cache_of(a[0], a[1], a[2], a[3]);
        if (!cache.there)
            type_error("cache must be a KVCache");
        const at::Tensor &of = tensor(a[0], "k"), &table = tensor(a[4], "block_table"), &cu = tensor(a[5], "cu");
        if (table.dim() != 2)
            value_error("block_table must have shape [batch, max_blocks], got " + shape_text(table.sizes()));
        const int64_t batch = table.size(0), blocks = table.size(1);
        require(table, at::kInt, {batch, blocks}, "block_table");
        require(cu, at::kInt, {batch + 1}, "cu");
        const int64_t total = integer(a[6], "total");
        if (total < 0)
            value_error("total must be >= 0, got " + std::to_string(total));
        const int dtype = (int)integer(a[7], "dtype");
        const at::ScalarType type = dtype == CK_OUT_F16 ? at::kHalf : at::kBFloat16;
        at::Tensor out[2];
        for (int i = 0; i < 2; ++i)
            if (a[8 + i] == Py_None)
                out[i] = empty({total, cache.c.kv_heads, cache.c.head_dim}, type, of);
            else
                require(out[i] = tensor(a[8 + i], i ? "v" : "k"), type, {total, cache.c.kv_heads, cache.c.head_dim}, i ? "v" : "k");
        const int st = p_cache_read(&cache.c, table.data_ptr<int32_t>(), blocks, cu.data_ptr<int32_t>(), batch, total, dtype,
                                    out[0].data_ptr(), out[1].data_ptr(), current_stream(of));
        if (st != CK_OK)
            return PyLong_FromLong(st);
        PyObject *k = given_or(a[8], out[0]), *v = given_or(a[9], out[1]);
        PyObject* r = PyTuple_Pack(2, k, v);
        Py_DECREF(k);
        Py_DECREF(v);
        return r;
    });
}

// q, k, v, cu_q, cu_k, scale, causal, window, sinks, out, lse, return_lse -> out, or (out, lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded("attention", n, 12, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const int dtype = act_type(q, "q");
        const at::ScalarType type = q.scalar_type();
        const int64_t dim = q.dim() == 3 ? q.size(2) : 0;
        const int64_t qs = token_stride(q, type, dim, "q"), ks = token_stride(k, type, dim, "k"),
                      vs = token_stride(v, type, dim, "v");
        if (k.sizes() != v.sizes())
            value_error("k and v must have one shape, got " + shape_text(k.sizes()) + " and " + shape_text(v.sizes()));
        const int64_t total_q = q.size(0), heads = q.size(1);
        const at::Tensor &cu_q = tensor(a[3], "cu_q"), &cu_k = a[4] == Py_None ? cu_q : tensor(a[4], "cu_k");
        if (cu_q.dim() != 1 || cu_q.size(0) < 1)
            value_error("cu_q must hold batch + 1 bounds, got shape " + shape_text(cu_q.sizes()));
        const int64_t batch = cu_q.size(0) - 1;
        require(cu_q, at::kInt, {batch + 1}, "cu_q");
        require(cu_k, at::kInt, {batch + 1}, "cu_k");
        at::Tensor out, lse;
        if (a[9] == Py_None)
            out = empty({total_q, heads, dim}, type, q);
        else
            require(out = tensor(a[9], "out"), type, {total_q, heads, dim}, "out");
        const bool return_lse = truth(a[11]);
        if (a[10] != Py_None)
            require(lse = tensor(a[10], "lse"), at::kFloat, {heads, total_q}, "lse");
        else if (return_lse)
            lse = empty({heads, total_q}, at::kFloat, q);
        const float scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)std::max<int64_t>(dim, 1)))
                                            : (float)number(a[5], "scale");
        const int st = p_attention(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, cu_q.data_ptr<int32_t>(),
                                   cu_k.data_ptr<int32_t>(), batch, total_q, k.size(0), heads, k.size(1), dim, dtype, scale,
                                   truth(a[6]) ? 1 : 0, integer(a[7], "window"), integer(a[8], "sinks"), out.data_ptr(),
                                   lse.defined() ? lse.data_ptr<float>() : nullptr, current_stream(q));
        if (st != CK_OK)
            return PyLong_FromLong(st);
        PyObject* o = given_or(a[9], out);
        if (!return_lse)
            return o;
        PyObject* l = given_or(a[10], lse);
        PyObject* r = PyTuple_Pack(2, o, l);
        Py_DECREF(o);
        Py_DECREF(l);
        return r;
    });
}

// x, w4, w_scale, bias, residual, y, out_dtype (a ck_dtype_t, or -1: x's) -> y
PyObject* int4_linear(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded("int4_linear", n, 7, [&]() -> PyObject* {
        const at::Tensor &x = tensor(a[0], "x"), &w4 = tensor(a[1], "w4"), &ws = tensor(a[2], "w_scale");
        const int dtype = act_type(x, "x");
        if (x.dim() != 2 || ws.dim() != 2)
            value_error("x must have shape [M, K] and w_scale [N, K / group], got " + shape_text(x.sizes()) + " and " +
                        shape_text(ws.sizes()));
        const int64_t M = x.size(0), K = x.size(1), N = ws.size(0), groups = ws.size(1);
        require(x, x.scalar_type(), {M, K}, "x");
        require(w4, at::kInt, {N, K / 8}, "w4");
        require(ws, at::kBFloat16, {N, groups}, "w_scale");
        if (groups < 1 || K % groups != 0)
            value_error("K=" + std::to_string(K) + " does not divide into " + std::to_string(groups) + " groups");
        const at::Tensor* bias = optional_tensor(a[3], "bias");
        if (bias)
            require(*bias, x.scalar_type(), {N}, "bias");
        const int64_t code = integer(a[6], "out_dtype");
        const int out_code = code < 0 ? dtype : (int)code;
        const at::ScalarType out_type = out_code == CK_OUT_BF16 ? at::kBFloat16 : out_code == CK_OUT_F16 ? at::kHalf : at::kFloat;
        const at::Tensor* residual = optional_tensor(a[4], "residual");
        if (residual)
            require(*residual, out_type, {M, N}, "residual");
        at::Tensor y;
        if (a[5] == Py_None)
            y = empty({M, N}, out_type, x);
        else
            require(y = tensor(a[5], "y"), out_type, {M, N}, "y");
        const int st = p_int4(x.data_ptr(), static_cast<const uint32_t*>(w4.data_ptr()), ws.data_ptr(), ptr(bias),
                              ptr(residual), y.data_ptr(), M, N, K, K / groups, dtype, out_code, current_stream(x));
        if (st != CK_OK)
            return PyLong_FromLong(st);
        return given_or(a[5], y);
    });
}

at::ScalarType type_of(int code)
{
    return code == CK_OUT_BF16 ? at::kBFloat16 : code == CK_OUT_F16 ? at::kHalf : at::kFloat;
}

// a ck_dtype_t, -1 for other types
int code_of(at::ScalarType t)
{
    return t == at::kBFloat16 ? CK_OUT_BF16 : t == at::kHalf ? CK_OUT_F16 : t == at::kFloat ? CK_OUT_F32 : -1;
}

// x, a, b, index, scaling, residual, y, out_dtype (a ck_dtype_t, or -1: the residual's, else x's), ws -> y
PyObject* adapter_linear(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded("adapter_linear", n, 9, [&]() -> PyObject* {
        const at::Tensor &x = tensor(a[0], "x"), &down = tensor(a[1], "a"), &up = tensor(a[2], "b"),
                         &index = tensor(a[3], "index");
        const int dtype = act_type(x, "x");
        const at::ScalarType type = x.scalar_type();
        if (x.dim() != 2 || down.dim() != 3 || up.dim() != 3)
            value_error("x must have shape [M, K], a [adapters, rank, K] and b [adapters, N, rank], got " +
                        shape_text(x.sizes()) + ", " + shape_text(down.sizes()) + " and " + shape_text(up.sizes()));
        const int64_t M = x.size(0), K = x.size(1), adapters = down.size(0), rank = down.size(1), N = up.size(1);
        require(x, type, {M, K}, "x");
        require(down, type, {adapters, rank, K}, "a");
        require(up, type, {adapters, N, rank}, "b");
        require(index, at::kInt, {M}, "index");
        const at::Tensor *scaling = optional_tensor(a[4], "scaling"), *residual = optional_tensor(a[5], "residual");
        if (scaling)
            require(*scaling, at::kFloat, {adapters}, "scaling");
        const int64_t code = integer(a[7], "out_dtype");
        const int out_code = code >= 0 ? (int)code : residual ? code_of(residual->scalar_type()) : dtype;
        if (out_code < 0)
            type_error(std::string("residual must be torch.bfloat16, torch.float16 or torch.float32, got ") +
                       type_name(residual->scalar_type()));
        if (residual)
            require(*residual, type_of(out_code), {M, N}, "residual");
        at::Tensor y, ws;
        if (a[6] == Py_None)
            y = empty({M, N}, type_of(out_code), x);
        else
            require(y = tensor(a[6], "y"), type_of(out_code), {M, N}, "y");
        size_t ws_bytes = p_adapter_ws(M, N, K, rank);
        void* ws_ptr = workspace_of(a[8], &ws_bytes, x, &ws);
        const int st = p_adapter(x.data_ptr(), down.data_ptr(), up.data_ptr(), index.data_ptr<int32_t>(),
                                 static_cast<const float*>(ptr(scaling)), ptr(residual), y.data_ptr(), M, N, K, rank, adapters,
                                 dtype, out_code, ws_ptr, ws_bytes, current_stream(x));
        if (st != CK_OK)
            return PyLong_FromLong(st);
        return given_or(a[6], y);
    });
}

// Outputs that share one allocation: a view of `of`'s memory from byte `at` on.  (Five of their own took 4 us
// more of host time.)
at::Tensor part_of(const at::Tensor& of, int64_t at, c10::IntArrayRef shape, at::ScalarType type)
{
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(of.storage()), of.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(at / (int64_t)c10::elementSize(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
}

// logits, tokens, top, scale, logprob, entropy, lse, top_logprob, top_index, ws -> the five outputs
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded("token_logprobs", n, 10, [&]() -> PyObject* {
        const at::Tensor& x = tensor(a[0], "logits");
        const int dtype = code_of(x.scalar_type());
        if (dtype < 0)
            type_error(std::string("logits must be torch.bfloat16, torch.float16 or torch.float32, got ") +
                       type_name(x.scalar_type()));
        if (x.dim() != 2 || !x.is_cuda() || (x.stride(1) != 1 && x.size(1) > 1))
            value_error("logits must be a CUDA tensor [rows, vocab] with dense rows, got " + shape_text(x.sizes()));
        const int64_t rows = x.size(0), vocab = x.size(1), top = integer(a[2], "top");
        const at::Tensor* tokens = optional_tensor(a[1], "tokens");
        if (tokens)
            require(*tokens, at::kInt, {rows}, "tokens");
        const bool wanted[5] = {tokens != nullptr, true, true, top > 0, top > 0};
        static const char* const names[5] = {"logprob", "entropy", "lse", "top", "index"};
        bool given = false;
        for (int i = 0; i < 5; ++i)
            given |= a[4 + i] != Py_None;
        at::Tensor out[5], ws, all;
        const int64_t row_bytes = (rows * 4 + 15) / 16 * 16, top_bytes = (rows * std::max<int64_t>(top, 0) * 4 + 15) / 16 * 16;
        if (!given && top <= 32)
            all = empty({3 * row_bytes + 2 * top_bytes}, at::kByte, x);
        for (int i = 0; i < 5; ++i) {
            const at::ScalarType type = i == 4 ? at::kInt : at::kFloat;
            const int64_t shape[2] = {rows, top};
            const c10::IntArrayRef sizes(shape, i < 3 ? 1 : 2);
            if (a[4 + i] != Py_None) {
                if (!wanted[i])
                    value_error(std::string(names[i]) + " is given, but not asked for");
                require(out[i] = tensor(a[4 + i], names[i]), type, sizes, names[i]);
            } else if (wanted[i] && !given && top <= 32) {
                out[i] = part_of(all, i < 3 ? i * row_bytes : 3 * row_bytes + (i - 3) * top_bytes, sizes, type);
            } else if (i >= 3 && wanted[i] && given) {
                value_error("top and index must be given where out is and top > 0");
            }
        }
        size_t ws_bytes = p_logprobs_ws(rows, vocab, top);
        void* ws_ptr = workspace_of(a[9], &ws_bytes, x, &ws);
        auto f32 = [&](int i) { return out[i].defined() ? out[i].data_ptr<float>() : nullptr; };
        const int st = p_logprobs(x.data_ptr(), rows > 1 ? x.stride(0) : vocab, tokens ? tokens->data_ptr<int32_t>() : nullptr,
                                  rows, vocab, dtype, (float)number(a[3], "scale"), top, f32(0), f32(1), f32(2), f32(3),
                                  out[4].defined() ? out[4].data_ptr<int32_t>() : nullptr, ws_ptr, ws_bytes,
                                  current_stream(x));
        if (st != CK_OK)
            return PyLong_FromLong(st);
        PyObject* r = PyTuple_New(5);
        for (int i = 0; i < 5; ++i)
            PyTuple_SET_ITEM(r, i, a[4 + i] == Py_None && !out[i].defined() ? Py_NewRef(Py_None) : given_or(a[4 + i], out[i]));
        return r;
    });
}

#define CK_FAST(fn) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn))

PyMethodDef methods[] = {{"init", CK_FAST(init), METH_FASTCALL, nullptr},
                         {"norm_rope", CK_FAST(norm_rope), METH_FASTCALL, nullptr},
                         {"paged_attention", CK_FAST(paged_attention), METH_FASTCALL, nullptr},
                         {"attention", CK_FAST(attention), METH_FASTCALL, nullptr},
                         {"int4_linear", CK_FAST(int4_linear), METH_FASTCALL, nullptr},
                         {"prefix_attention", CK_FAST(prefix_attention), METH_FASTCALL, nullptr},
                         {"cache_read", CK_FAST(cache_read), METH_FASTCALL, nullptr},
                         {"adapter_linear", CK_FAST(adapter_linear), METH_FASTCALL, nullptr},
                         {"token_logprobs", CK_FAST(token_logprobs), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ck_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ck_binding()
{
    return PyModule_Create(&module);
}
