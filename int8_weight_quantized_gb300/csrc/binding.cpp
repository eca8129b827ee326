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
    return guarded("init", n, 5, [&]() -> PyObject* {
        void* f[5];
        for (int i = 0; i < 5; ++i)
            f[i] = reinterpret_cast<void*>(static_cast<intptr_t>(integer(a[i], "address")));
        p_norm_rope = reinterpret_cast<decltype(p_norm_rope)>(f[0]);
        p_paged_ws = reinterpret_cast<decltype(p_paged_ws)>(f[1]);
        p_paged = reinterpret_cast<decltype(p_paged)>(f[2]);
        p_attention = reinterpret_cast<decltype(p_attention)>(f[3]);
        p_int4 = reinterpret_cast<decltype(p_int4)>(f[4]);
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

#define CK_FAST(fn) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn))

PyMethodDef methods[] = {{"init", CK_FAST(init), METH_FASTCALL, nullptr},
                         {"norm_rope", CK_FAST(norm_rope), METH_FASTCALL, nullptr},
                         {"paged_attention", CK_FAST(paged_attention), METH_FASTCALL, nullptr},
                         {"attention", CK_FAST(attention), METH_FASTCALL, nullptr},
                         {"int4_linear", CK_FAST(int4_linear), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ck_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ck_binding()
{
    return PyModule_Create(&module);
}
