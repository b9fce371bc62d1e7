// awq_step_module.cpp -- torch-facing side of the decoding step's operators, a Python
// module: tests the arguments, allocates outputs, passes pointers, strides and the
// current stream to the C ABI (awq_gb300.h). step.py has the public functions.
//
// A step's kernels take a few microseconds each. The same tests in Python, at a tenth
// of a microsecond an attribute, took longer: 10 us of 12 for one attention call, 13
// of 15 for one row of logits.
//
// Each function returns its result, or the status (an int) that the library gave
// instead of AWQ_OK; arguments that no library call could serve raise ValueError.
#include <Python.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "awq_gb300.h"

namespace {

using at::Tensor;

// the library that _binding.py has loaded
decltype(&awq_paged_plan) plan_entry;
decltype(&awq_kv_append) append_entry;
decltype(&awq_tree_attention) attention_entry;
decltype(&awq_process_logits) logits_entry;

struct Refused {          // becomes a ValueError
    std::string why;
};
struct Raised {};         // a Python exception is set

[[noreturn]] void refuse(const char *format, ...)
{
    char text[256];
    va_list args;
    va_start(args, format);
    std::vsnprintf(text, sizeof text, format, args);
    va_end(args);
    throw Refused{text};
}

const char *name_of(at::ScalarType t)
{
    switch (t) {
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    default: return c10::toString(t);
    }
}

const Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
        throw Raised{};
    }
    return THPVariable_Unpack(o);
}

const Tensor *tensor_or_none(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

// The device of the call: the library launches on the current one, with its scratch and
// status word, so the tensors have to be there.
int cuda_index(const Tensor &t)
{
    if (!t.is_cuda()) refuse("the AWQ library runs on CUDA tensors only");
    c10::DeviceIndex current = -1;
    if (c10::cuda::GetDevice(&current) != cudaSuccess || t.get_device() != current)
        refuse("the AWQ library works on the current CUDA device (%d), the tensors are on cuda:%d", (int)current,
               (int)t.get_device());
    return current;
}

bool on(const Tensor &t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// A contiguous tensor of this type and device, of n elements (any number if negative).
void check(const Tensor &t, const char *name, at::ScalarType type, int dev, int64_t n = -1)
{
    if (t.scalar_type() != type) refuse("%s must be %s, got %s", name, name_of(type), name_of(t.scalar_type()));
    if (!on(t, dev)) refuse("%s must be on cuda:%d, got %s", name, dev, t.device().str().c_str());
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    if (n >= 0 && t.numel() != n)
        refuse("%s must have %lld elements, got %lld", name, (long long)n, (long long)t.numel());
}

template <typename T>
T *data(const Tensor *t)
{
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}

// Data of a checked tensor, or null for none.
template <typename T>
T *checked(PyObject *o, const char *name, at::ScalarType type, int dev, int64_t n = -1)
{
    const Tensor *t = tensor_or_none(o, name);
    if (t) check(*t, name, type, dev, n);
    return data<T>(t);
}

// A block table's width and row stride.
void check_table(const Tensor &t, int64_t requests, int dev, int64_t &width, int64_t &stride)
{
    if (t.scalar_type() != at::kInt || !on(t, dev) || t.dim() != 2)
        refuse("block_table must be a torch.int32 [requests, blocks] tensor on the others' device");
    width = t.size(1);
    if (t.size(0) != requests || (t.stride(1) != 1 && width > 1))
        refuse("block_table must be [requests, blocks] with adjacent entries in a row");
    stride = requests > 1 ? t.stride(0) : width;
}

// A paged cache; the stride of an axis with one entry is never used: a valid one stands in.
awq_cache_t cache(const Tensor &t, const char *name, at::ScalarType type, int dev, const Tensor &like)
{
    if (t.scalar_type() != type || !on(t, dev) || t.dim() != 4 || t.sizes() != like.sizes() ||
        (t.stride(3) != 1 && t.size(3) > 1))
        refuse("%s must be a %s [blocks, block_size, kv_heads, head_dim] tensor with adjacent head_dim elements on the "
               "others' device, of the other's shape", name, name_of(type));
    awq_cache_t c{};
    c.data = t.data_ptr();
    c.block_stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2) * t.size(3);
    c.token_stride = t.stride(1);
    c.head_stride = t.size(2) > 1 ? t.stride(2) : t.size(3);
    return c;
}

struct Rows {
    int64_t tokens, heads, dim, token_stride, head_stride;
};

Rows rows_of(const Tensor &t, const char *name, at::ScalarType type, int dev)
{
    if (t.scalar_type() != type || !on(t, dev))
        refuse("%s must be %s on the others' device, got %s on %s", name, name_of(type), name_of(t.scalar_type()),
               t.device().str().c_str());
    if (t.dim() != 3 || (t.stride(2) != 1 && t.size(2) > 1))
        refuse("%s must be [tokens, heads, head_dim] with adjacent head_dim elements", name);
    Rows r{t.size(0), t.size(1), t.size(2), 0, 0};
    r.token_stride = r.tokens > 1 ? t.stride(0) : r.heads * r.dim;
    r.head_stride = r.heads > 1 ? t.stride(1) : r.dim;
    return r;
}

awq_stream_t stream_of(int dev)
{
    return reinterpret_cast<awq_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}

// The library call, without the interpreter's lock.
template <typename F>
int call(F entry)
{
    if (!plan_entry) refuse("the library is not bound");
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = entry();
    Py_END_ALLOW_THREADS
    return status;
}

PyObject *keep(PyObject *o)
{
    Py_INCREF(o);
    return o;
}

// ---------------------------------------------------------------------------

PyObject *paged_plan(PyObject *const *o)
{
    const Tensor &ctx = tensor(o[0], "context_lens"), &fresh = tensor(o[1], "new_lens");
    const Tensor &table = tensor(o[2], "block_table"), &free_blocks = tensor(o[3], "free_blocks");
    const int64_t block_size = integer(o[4]), T = integer(o[5]), words = integer(o[7]);
    const int dev = cuda_index(ctx);
    const int64_t B = ctx.numel();
    check(ctx, "context_lens", at::kInt, dev);
    check(fresh, "new_lens", at::kInt, dev, B);
    check(free_blocks, "free_blocks", at::kInt, dev);
    // the library's own limits, before memory of that size is asked for
    if (T < 0 || T > int64_t(1) << 30) refuse("max_tokens must be 0 to 2^30, got %lld", (long long)T);
    if (words < 0 || words > 1024) refuse("mask_words must be 0 to 1024, got %lld", (long long)words);
    const int32_t *parents = checked<int32_t>(o[6], "parents", at::kInt, dev, T);
    int64_t width, stride;
    check_table(table, B, dev, width, stride);
    // one allocation for all (six took 6 us of 10); the 64-bit numbers come first
    const Tensor area = at::empty({2 * T + (B + 1) + 2 * T + 2 + T * words},
                                  at::TensorOptions(at::kCUDA, (c10::DeviceIndex)dev).dtype(at::kInt));
    int64_t used = 0;
    auto take = [&](at::ScalarType type, at::IntArrayRef sizes) {
        Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(area.storage()),
                                                            area.key_set(), c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_storage_offset(used);     // in elements: the 64-bit ones have 0
        t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
        used += t.numel() * (type == at::kLong ? 2 : 1);
        return t;
    };
    Tensor slots = take(at::kLong, {T}), cu = take(at::kInt, {B + 1}), positions = take(at::kInt, {T});
    Tensor request = take(at::kInt, {T}), counts = take(at::kInt, {2}), mask;
    if (words > 0) mask = take(at::kInt, {T, words});
    const awq_stream_t stream = stream_of(dev);
    const int status = call([&] {
        return plan_entry(data<int32_t>(&ctx), data<int32_t>(&fresh), B, data<int32_t>(&table), width, stride,
                          data<int32_t>(&free_blocks), free_blocks.numel(), block_size, parents, T, data<int32_t>(&cu),
                          data<int64_t>(&slots), data<int32_t>(&positions), data<int32_t>(&request),
                          words > 0 ? data<int32_t>(&mask) : nullptr, words, data<int32_t>(&counts), stream);
    });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    PyObject *all = PyTuple_New(6);
    if (!all) throw Raised{};
    PyTuple_SET_ITEM(all, 0, THPVariable_Wrap(std::move(cu)));
    PyTuple_SET_ITEM(all, 1, THPVariable_Wrap(std::move(slots)));
    PyTuple_SET_ITEM(all, 2, THPVariable_Wrap(std::move(positions)));
    PyTuple_SET_ITEM(all, 3, THPVariable_Wrap(std::move(request)));
    PyTuple_SET_ITEM(all, 4, words > 0 ? THPVariable_Wrap(std::move(mask)) : keep(Py_None));
    PyTuple_SET_ITEM(all, 5, THPVariable_Wrap(std::move(counts)));
    return all;
}

PyObject *kv_append(PyObject *const *o)
{
    const Tensor &k = tensor(o[0], "k"), &v = tensor(o[1], "v"), &kc = tensor(o[2], "k_cache"), &vc = tensor(o[3], "v_cache");
    const Tensor &slots = tensor(o[4], "slot_map");
    const int dev = cuda_index(kc);
    const at::ScalarType type = kc.scalar_type();
    if (type != at::kHalf && type != at::kBFloat16) refuse("the cache must be float16 or bfloat16, got %s", name_of(type));
    const awq_cache_t k_cache = cache(kc, "k_cache", type, dev, kc), v_cache = cache(vc, "v_cache", type, dev, kc);
    const Rows kr = rows_of(k, "k", type, dev), vr = rows_of(v, "v", type, dev);
    if (kr.tokens != vr.tokens || kr.heads != vr.heads || kr.dim != vr.dim || kr.heads != kc.size(2) || kr.dim != kc.size(3))
        refuse("k, v and the two caches must agree in heads and head_dim");
    check(slots, "slot_map", at::kLong, dev, kr.tokens);
    const awq_stream_t stream = stream_of(dev);
    const int status = call([&] {
        return append_entry(k.data_ptr(), kr.token_stride, kr.head_stride, v.data_ptr(), vr.token_stride, vr.head_stride,
                            &k_cache, &v_cache, data<int64_t>(&slots), kr.tokens, kc.size(0), kc.size(1), kr.heads, kr.dim,
                            stream);
    });
    return status == AWQ_OK ? keep(Py_None) : PyLong_FromLong(status);
}

PyObject *tree_attention(PyObject *const *o)
{
    const Tensor &q = tensor(o[0], "q"), &kc = tensor(o[1], "k_cache"), &vc = tensor(o[2], "v_cache");
    const Tensor &table = tensor(o[3], "block_table"), &ctx = tensor(o[4], "context_lens"), &cu = tensor(o[5], "cu_new");
    const double scale = PyFloat_AsDouble(o[6]);
    if (scale == -1. && PyErr_Occurred()) throw Raised{};
    const Tensor *mask = tensor_or_none(o[9], "tree_mask"), *out = tensor_or_none(o[10], "out"), *lse = tensor_or_none(o[11], "lse");
    const int dev = cuda_index(q);
    const at::ScalarType type = q.scalar_type();
    if (type != at::kHalf && type != at::kBFloat16) refuse("q must be float16 or bfloat16, got %s", name_of(type));
    const Rows r = rows_of(q, "q", type, dev);
    awq_tree_attention_t a{};
    a.k_cache = cache(kc, "k_cache", type, dev, kc);
    a.v_cache = cache(vc, "v_cache", type, dev, kc);
    if (kc.size(3) != r.dim) refuse("q and the caches must agree in head_dim");
    a.B = ctx.numel();
    check(ctx, "context_lens", at::kInt, dev);
    check(cu, "cu_new", at::kInt, dev, a.B + 1);
    check_table(table, a.B, dev, a.table_width, a.table_stride);
    if (mask) {
        check(*mask, "tree_mask", at::kInt, dev);
        if (mask->dim() != 2 || mask->size(0) != r.tokens || mask->size(1) == 0) refuse("tree_mask must be [tokens, mask_words]");
        a.tree_mask = data<int32_t>(mask);
        a.mask_words = mask->size(1);
    }
    if (out) {
        check(*out, "out", type, dev);
        if (out->sizes() != q.sizes()) refuse("out must have q's shape");
    }
    if (lse) {
        check(*lse, "lse", at::kFloat, dev);
        if (lse->dim() != 2 || lse->size(0) != r.tokens || lse->size(1) != r.heads) refuse("lse must be [tokens, q_heads]");
        a.lse = data<float>(lse);
    }
    Tensor made;
    if (!out) made = at::empty(q.sizes(), q.options());
    a.q = q.data_ptr();
    a.q_token_stride = r.token_stride;
    a.q_head_stride = r.head_stride;
    a.out = out ? out->data_ptr() : made.data_ptr();
    a.block_table = data<int32_t>(&table);
    a.context_lens = data<int32_t>(&ctx);
    a.cu_new = data<int32_t>(&cu);
    a.tokens = r.tokens;
    a.q_heads = r.heads;
    a.kv_heads = kc.size(2);
    a.head_dim = r.dim;
    a.num_blocks = kc.size(0);
    a.block_size = kc.size(1);
    a.max_new = integer(o[7]);
    a.max_context = integer(o[8]);
    a.scale = (float)scale;
    a.dtype = type == at::kHalf ? AWQ_F16 : AWQ_BF16;
    const awq_stream_t stream = stream_of(dev);
    const int status = call([&] { return attention_entry(&a, stream); });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    return out ? keep(o[10]) : THPVariable_Wrap(std::move(made));
}

PyObject *process_logits(PyObject *const *o)
{
    const Tensor &x = tensor(o[0], "logits");
    const Tensor *request = tensor_or_none(o[1], "row_request");
    const Tensor *mask = tensor_or_none(o[10], "tree_mask"), *grammar = tensor_or_none(o[14], "grammar_mask");
    const Tensor *out = tensor_or_none(o[16], "out");
    const int dev = cuda_index(x);
    const at::ScalarType type = x.scalar_type();
    if (type != at::kHalf && type != at::kBFloat16 && type != at::kFloat)
        refuse("logits must be float16, bfloat16 or float32, got %s", name_of(type));
    if (x.dim() != 2 || (x.stride(1) != 1 && x.size(1) > 1)) refuse("logits must be [rows, vocab] with adjacent elements in a row");
    awq_logits_t a{};
    a.rows = x.size(0);
    a.vocab = x.size(1);
    // the requests: the rows, or as many as the per-request tensors have
    a.B = request ? (int64_t(1) << 31) - 1 : a.rows;
    if (request) {
        const int per_request[7] = {5, 6, 7, 4, 3, 13, 9};      // of which the last three have one more
        for (int i = 0; i < 7; ++i) {
            const Tensor *t = tensor_or_none(o[per_request[i]], "a per-request argument");
            if (!t) continue;
            a.B = t->numel() - (i >= 4);
            if (a.B < 0) refuse("offsets must have one element at least");
            break;
        }
    }
    a.row_request = checked<int32_t>(o[1], "row_request", at::kInt, dev, a.rows);
    a.history = checked<int32_t>(o[2], "history", at::kInt, dev);
    a.history_offsets = checked<int32_t>(o[3], "history_offsets", at::kInt, dev, a.B + 1);
    a.prompt_lens = checked<int32_t>(o[4], "prompt_lens", at::kInt, dev, a.B);
    a.repetition = checked<float>(o[5], "repetition", at::kFloat, dev, a.B);
    a.frequency = checked<float>(o[6], "frequency", at::kFloat, dev, a.B);
    a.presence = checked<float>(o[7], "presence", at::kFloat, dev, a.B);
    a.draft_tokens = checked<int32_t>(o[8], "draft_tokens", at::kInt, dev, a.rows);
    a.cu_new = checked<int32_t>(o[9], "cu_new", at::kInt, dev, a.B + 1);
    a.tree_mask = checked<int32_t>(o[10], "tree_mask", at::kInt, dev);
    a.bias_tokens = checked<int32_t>(o[11], "bias_tokens", at::kInt, dev);
    a.bias_offsets = checked<int32_t>(o[13], "bias_offsets", at::kInt, dev, a.B + 1);
    const bool biases = o[11] != Py_None;
    if (biases && (o[12] == Py_None || o[13] == Py_None)) refuse("bias_tokens, bias_values and bias_offsets go together");
    a.bias_size = biases ? THPVariable_Unpack(o[11]).numel() : 0;
    a.bias_values = checked<float>(o[12], "bias_values", at::kFloat, dev, biases ? a.bias_size : -1);
    a.grammar_mask = checked<int32_t>(o[14], "grammar_mask", at::kInt, dev);
    a.grammar_rows = checked<int32_t>(o[15], "grammar_rows", at::kInt, dev, a.rows);
    if (o[2] != Py_None) {
        if (o[3] == Py_None) refuse("history needs history_offsets");
        a.history_size = THPVariable_Unpack(o[2]).numel();
    }
    if (o[8] != Py_None && o[9] == Py_None) refuse("draft_tokens needs cu_new");
    if (mask) {
        if (mask->dim() != 2 || mask->size(0) != a.rows) refuse("tree_mask must be [rows, mask_words]");
        a.mask_words = mask->size(1);
    }
    if (grammar) {
        if (grammar->dim() != 2 || grammar->size(1) != (a.vocab + 31) / 32) refuse("grammar_mask must be [masks, ceil(vocab / 32)]");
        a.grammar_count = grammar->size(0);
    }
    Tensor made;
    if (!out) made = at::empty(x.sizes(), x.options());
    const Tensor &y = out ? *out : made;
    if (out && (y.scalar_type() != type || !on(y, dev) || y.sizes() != x.sizes() || (y.stride(1) != 1 && a.vocab > 1)))
        refuse("out must be like logits, with adjacent elements in a row");
    a.logits = x.data_ptr();
    a.out = y.data_ptr();
    a.logits_row_stride = a.rows > 1 ? x.stride(0) : a.vocab;
    a.out_row_stride = a.rows > 1 ? y.stride(0) : a.vocab;
    a.dtype = type == at::kHalf ? AWQ_F16 : type == at::kBFloat16 ? AWQ_BF16 : AWQ_F32;
    const awq_stream_t stream = stream_of(dev);
    const int status = call([&] { return logits_entry(&a, stream); });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    return out ? keep(o[16]) : THPVariable_Wrap(std::move(made));
}

// Addresses of the library's four entry points.
PyObject *bind(PyObject *const *o)
{
    const int64_t entries[4] = {integer(o[0]), integer(o[1]), integer(o[2]), integer(o[3])};
    append_entry = reinterpret_cast<decltype(append_entry)>(entries[1]);
    attention_entry = reinterpret_cast<decltype(attention_entry)>(entries[2]);
    logits_entry = reinterpret_cast<decltype(logits_entry)>(entries[3]);
    plan_entry = reinterpret_cast<decltype(plan_entry)>(entries[0]);
    return keep(Py_None);
}

template <PyObject *(*kBody)(PyObject *const *), int kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return kBody(args);
    } catch (const Refused &r) {
        PyErr_SetString(PyExc_ValueError, r.why.c_str());
    } catch (const Raised &) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*kBody)(PyObject *const *), int kArgs>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kBody, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind, 4>("bind"),
                         method<paged_plan, 8>("paged_plan"),
                         method<kv_append, 5>("kv_append"),
                         method<tree_attention, 12>("tree_attention"),
                         method<process_logits, 17>("process_logits"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "awq_step", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit_awq_step() { return PyModule_Create(&definition); }
