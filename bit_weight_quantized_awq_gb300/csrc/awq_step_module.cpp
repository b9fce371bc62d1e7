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

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <optional>
#include <string>
#include <vector>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
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
decltype(&awq_rotary) rotary_entry;
decltype(&awq_beam_select) beam_entry;
decltype(&awq_beam_select_workspace) beam_workspace_entry;
decltype(&awq_reorder_states) reorder_entry;
decltype(&awq_fork_pages) fork_entry;
decltype(&awq_copy_pages) copy_entry;
decltype(&awq_free_pages) free_entry;
decltype(&awq_compact_pages) compact_entry;
decltype(&awq_pages_workspace) pages_workspace_entry;

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
    const Tensor &t = THPVariable_Unpack(o);
    // their memory holds something else than their elements
    if (t.is_conj() || t.is_neg()) refuse("%s is conjugated or negated only when it is read: resolve_conj(), resolve_neg()", name);
    return t;
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
    if (t.size(0) != requests || (t.stride(1) != 1 && width > 1 && requests > 0))
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

// One allocation of a call for all of its results (six took 6 us of 10), in words of 4 bytes.
class Area {
public:
    Area(int dev, int64_t words)
        : area_(at::empty({words}, at::TensorOptions(at::kCUDA, (c10::DeviceIndex)dev).dtype(at::kInt)))
    {
    }
    // The next part; 64-bit ones have to lie on 8 bytes.
    Tensor take(at::ScalarType type, at::IntArrayRef sizes)
    {
        const int each = type == at::kLong ? 2 : 1;
        Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(area_.storage()),
                                                            area_.key_set(), c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_storage_offset(used_ / each);     // in elements
        t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
        used_ += t.numel() * each;
        return t;
    }

private:
    Tensor area_;
    int64_t used_ = 0;
};

// A call's workspace, apart from its results: a caller that keeps those does not keep it. It is the current
// stream's, as the call is, so that its memory serves the next one there; begins on 512 bytes.
c10::DataPtr workspace_of(int64_t bytes) { return c10::cuda::CUDACachingAllocator::get()->allocate((size_t)bytes); }

PyObject *keep(PyObject *o)
{
    Py_INCREF(o);
    return o;
}

// A tuple of tensors; one that is not defined becomes None.
template <typename... Tensors>
PyObject *tuple_of(Tensors &&...tensors)
{
    PyObject *all = PyTuple_New(sizeof...(tensors));
    if (!all) throw Raised{};
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(all, i++, tensors.defined() ? THPVariable_Wrap(std::move(tensors)) : keep(Py_None)), ...);
    return all;
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
    // the 64-bit numbers come first
    Area area(dev, 2 * T + (B + 1) + 2 * T + 2 + T * words);
    auto take = [&](at::ScalarType type, at::IntArrayRef sizes) { return area.take(type, sizes); };
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
    return tuple_of(cu, slots, positions, request, mask, counts);
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

// q or k turned, with its output (made where there is none).
struct Turned {
    Rows in, out;
    Tensor made;
    void *to;
};

Turned turned(const Tensor &x, const Tensor *out, const char *name, const char *out_name, at::ScalarType type, int dev)
{
    Turned t{rows_of(x, name, type, dev), {}, {}, nullptr};
    if (out) {
        t.out = rows_of(*out, out_name, type, dev);
        if (out->sizes() != x.sizes()) refuse("%s must have %s's shape", out_name, name);
        t.to = out->data_ptr();
    } else {
        t.made = at::empty(x.sizes(), x.options());
        t.out = {t.in.tokens, t.in.heads, t.in.dim, t.in.heads * t.in.dim, t.in.dim};
        t.to = t.made.data_ptr();
    }
    return t;
}

// Arguments that rotary and rotary_append share; returns the device.
int rotary_arguments(awq_rotary_t &a, const Tensor &q, const Tensor *q_out, PyObject *positions_o, PyObject *freq_o,
                     PyObject *axes_o, PyObject *pairs_o, Turned &tq)
{
    const Tensor &positions = tensor(positions_o, "positions"), &freq = tensor(freq_o, "inv_freq");
    const int dev = cuda_index(q);
    const at::ScalarType type = q.scalar_type();
    if (type != at::kHalf && type != at::kBFloat16) refuse("q must be float16 or bfloat16, got %s", name_of(type));
    tq = turned(q, q_out, "q", "q_out", type, dev);
    check(positions, "positions", at::kInt, dev);
    if (positions.dim() < 1 || positions.dim() > 2 || positions.size(-1) != tq.in.tokens || (positions.dim() == 2 && positions.size(0) == 0))
        refuse("positions must be [tokens] or [axes, tokens]");
    check(freq, "inv_freq", at::kFloat, dev);
    if (freq.dim() != 1 || freq.numel() == 0 || 2 * freq.numel() > tq.in.dim)
        refuse("inv_freq must be [rotary_dim / 2] with rotary_dim up to head_dim");
    a.q = q.data_ptr();
    a.q_token_stride = tq.in.token_stride;
    a.q_head_stride = tq.in.head_stride;
    a.q_out = tq.to;
    a.q_out_token_stride = tq.out.token_stride;
    a.q_out_head_stride = tq.out.head_stride;
    a.positions = data<int32_t>(&positions);
    a.inv_freq = data<float>(&freq);
    a.axes = checked<int32_t>(axes_o, "axes", at::kInt, dev, freq.numel());
    a.tokens = tq.in.tokens;
    a.q_heads = tq.in.heads;
    a.head_dim = tq.in.dim;
    a.rotary_dim = 2 * freq.numel();
    a.num_axes = positions.dim() == 2 ? positions.size(0) : 1;
    a.pairs = PyObject_IsTrue(pairs_o);
    if (a.pairs < 0) throw Raised{};
    a.dtype = type == at::kHalf ? AWQ_F16 : AWQ_BF16;
    return dev;
}

PyObject *rotary(PyObject *const *o)
{
    const Tensor &q = tensor(o[0], "q");
    const Tensor *k = tensor_or_none(o[1], "k"), *q_out = tensor_or_none(o[6], "q_out"), *k_out = tensor_or_none(o[7], "k_out");
    awq_rotary_t a{};
    Turned tq{}, tk{};
    const int dev = rotary_arguments(a, q, q_out, o[2], o[3], o[4], o[5], tq);
    if (k) {
        tk = turned(*k, k_out, "k", "k_out", q.scalar_type(), dev);
        if (tk.in.tokens != tq.in.tokens || tk.in.dim != tq.in.dim) refuse("q and k must agree in tokens and head_dim");
        a.k = k->data_ptr();
        a.k_token_stride = tk.in.token_stride;
        a.k_head_stride = tk.in.head_stride;
        a.k_out = tk.to;
        a.k_out_token_stride = tk.out.token_stride;
        a.k_out_head_stride = tk.out.head_stride;
        a.kv_heads = tk.in.heads;
    } else if (k_out) {
        refuse("k_out needs k");
    }
    const awq_stream_t stream = stream_of(dev);
    const int status = call([&] { return rotary_entry(&a, stream); });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    PyObject *all = PyTuple_New(2);
    if (!all) throw Raised{};
    PyTuple_SET_ITEM(all, 0, q_out ? keep(o[6]) : THPVariable_Wrap(std::move(tq.made)));
    PyTuple_SET_ITEM(all, 1, !k ? keep(Py_None) : k_out ? keep(o[7]) : THPVariable_Wrap(std::move(tk.made)));
    return all;
}

PyObject *rotary_append(PyObject *const *o)
{
    const Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k"), &v = tensor(o[2], "v"), &kc = tensor(o[5], "k_cache");
    const Tensor &vc = tensor(o[6], "v_cache"), &slots = tensor(o[7], "slot_map");
    const Tensor *q_out = tensor_or_none(o[10], "q_out");
    awq_rotary_t a{};
    Turned tq{};
    const int dev = rotary_arguments(a, q, q_out, o[3], o[4], o[8], o[9], tq);
    const at::ScalarType type = q.scalar_type();
    a.k_cache = cache(kc, "k_cache", type, dev, kc);
    a.v_cache = cache(vc, "v_cache", type, dev, kc);
    const Rows kr = rows_of(k, "k", type, dev), vr = rows_of(v, "v", type, dev);
    if (kr.tokens != tq.in.tokens || vr.tokens != tq.in.tokens || kr.heads != vr.heads || kr.heads != kc.size(2) ||
        kr.dim != tq.in.dim || vr.dim != tq.in.dim || kc.size(3) != tq.in.dim)
        refuse("q, k, v and the two caches must agree in tokens, heads and head_dim");
    check(slots, "slot_map", at::kLong, dev, kr.tokens);
    a.k = k.data_ptr();
    a.k_token_stride = kr.token_stride;
    a.k_head_stride = kr.head_stride;
    a.v = v.data_ptr();
    a.v_token_stride = vr.token_stride;
    a.v_head_stride = vr.head_stride;
    a.slot_map = data<int64_t>(&slots);
    a.num_blocks = kc.size(0);
    a.block_size = kc.size(1);
    a.kv_heads = kr.heads;
    const awq_stream_t stream = stream_of(dev);
    // without tokens the slots have no address, which would mean no cache
    const int status = a.tokens == 0 ? (int)AWQ_OK : call([&] { return rotary_entry(&a, stream); });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    return q_out ? keep(o[10]) : THPVariable_Wrap(std::move(tq.made));
}

PyObject *beam_select(PyObject *const *o)
{
    const Tensor &x = tensor(o[0], "logits"), &scores = tensor(o[1], "scores");
    const Tensor *ends = tensor_or_none(o[3], "end_tokens");
    const int dev = cuda_index(x);
    const at::ScalarType type = x.scalar_type();
    if (type != at::kHalf && type != at::kBFloat16 && type != at::kFloat)
        refuse("logits must be float16, bfloat16 or float32, got %s", name_of(type));
    if (x.dim() != 2 || (x.stride(1) != 1 && x.size(1) > 1)) refuse("logits must be [requests * beams, vocab] with adjacent elements in a row");
    check(scores, "scores", at::kFloat, dev);
    if (scores.dim() != 2 || scores.numel() != x.size(0) || scores.size(1) == 0)
        refuse("scores must be [requests, beams], one for every row of logits");
    awq_beam_select_t a{};
    a.logits = x.data_ptr();
    a.requests = scores.size(0);
    a.beams = scores.size(1);
    a.vocab = x.size(1);
    a.logits_row_stride = x.size(0) > 1 ? x.stride(0) : a.vocab;
    a.scores = data<float>(&scores);
    a.num_beams = integer(o[2]);
    if (ends) {
        check(*ends, "end_tokens", at::kInt, dev);
        a.end_tokens = data<int32_t>(ends);
        a.num_ends = ends->numel();
    }
    a.dtype = type == at::kHalf ? AWQ_F16 : type == at::kBFloat16 ? AWQ_BF16 : AWQ_F32;
    if (!beam_workspace_entry) refuse("the library is not bound");
    a.workspace_bytes = beam_workspace_entry(a.requests, a.beams, a.vocab, a.num_beams, a.num_ends, (awq_dtype_t)a.dtype);
    if (a.workspace_bytes < 0)
        refuse("beam_select takes up to 16384 requests, 1 to 32 beams and num_beams, up to 8 end_tokens and a vocabulary of 1 to 2^27");
    const int64_t n = a.requests * a.num_beams;
    const c10::DataPtr workspace = workspace_of(a.workspace_bytes);
    a.workspace = workspace.get();
    Area area(dev, (ends ? 6 : 3) * n);
    Tensor made[6];
    for (int i = 0; i < (ends ? 6 : 3); ++i) made[i] = area.take(i % 3 == 0 ? at::kFloat : at::kInt, {a.requests, a.num_beams});
    a.out_scores = data<float>(&made[0]);
    a.out_parents = data<int32_t>(&made[1]);
    a.out_tokens = data<int32_t>(&made[2]);
    if (ends) {
        a.ended_scores = data<float>(&made[3]);
        a.ended_parents = data<int32_t>(&made[4]);
        a.ended_tokens = data<int32_t>(&made[5]);
    }
    const awq_stream_t stream = stream_of(dev);
    const int status = call([&] { return beam_entry(&a, stream); });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    return tuple_of(made[0], made[1], made[2], made[3], made[4], made[5]);
}

// The tensors of a list or tuple.
class Tensors {
public:
    Tensors(PyObject *o, const char *name) : list_(PySequence_Fast(o, "a list of tensors is needed")), name_(name)
    {
        if (!list_) throw Raised{};
    }
    ~Tensors() { Py_DECREF(list_); }
    Tensors(const Tensors &) = delete;
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(list_); }
    const Tensor &operator[](Py_ssize_t i) const { return tensor(PySequence_Fast_GET_ITEM(list_, i), name_); }

private:
    PyObject *list_;
    const char *name_;
};

// The bytes that rows lie in: `rows` of `size`, `stride` apart.
struct Bytes {
    uintptr_t first;
    int64_t rows, stride, size;
    uintptr_t last() const { return first + (rows - 1) * stride + size; }
};

// Whether rows of one share a byte with rows of the other, which may lie between them. Both have rows and bytes.
bool overlap(const Bytes &a, const Bytes &b)
{
    if (a.last() <= b.first || b.last() <= a.first) return false;
    if (a.stride < a.size || b.stride < b.size) return true;       // not rows one after the other
    if (a.stride == b.stride) {
        const int64_t off = (int64_t)(b.first - a.first) % a.stride, behind = off < 0 ? off + a.stride : off;
        if (behind >= a.size && behind + b.size <= a.stride) return false;      // all of one in the other's gaps
    }
    // the rows of both in turn, past those that end before the other's begins
    uintptr_t x = a.first, y = b.first;
    while (x < a.last() && y < b.last()) {
        if (x + a.size <= y) x += (y - x - a.size) / a.stride * a.stride + a.stride;
        else if (y + b.size <= x) y += (x - y - b.size) / b.stride * b.stride + b.stride;
        else return true;
    }
    return false;
}

// Rows [n, ...] whose elements lie together, as an address, a stride and a size in bytes.
int64_t dense_row(const Tensor &t, const char *name)
{
    if (t.dim() < 1) refuse("%s must have a first dimension of rows", name);
    int64_t n = 1;
    for (const int64_t size : t.sizes().slice(1))
        if (size == 0) return 0;
    for (int64_t d = t.dim() - 1; d > 0; --d) {
        if (t.size(d) != 1 && t.stride(d) != n) refuse("a row of %s must be contiguous", name);
        n *= t.size(d);
    }
    return n * (int64_t)t.element_size();
}

PyObject *reorder_states(PyObject *const *o)
{
    const Tensors states(o[0], "states");
    const Tensor &parents = tensor(o[1], "parents");
    const int dev = cuda_index(parents);
    check(parents, "parents", at::kInt, dev);
    if (parents.dim() != 1) refuse("parents must be [rows]");
    const int64_t rows = parents.numel(), n = states.size();
    if (n > 4096) refuse("reorder_states takes up to 4096 states, got %lld", (long long)n);
    std::vector<awq_state_t> all(n);
    std::vector<Tensor> made;
    std::vector<Bytes> from, to;
    made.reserve(n);
    int64_t rows_in = 0;
    std::optional<Tensors> given;
    if (o[2] != Py_None) {
        given.emplace(o[2], "outs");
        if (given->size() != n) refuse("outs must have a tensor for every state");
    }
    for (int64_t i = 0; i < n; ++i) {
        const Tensor &s = states[i];
        if (!on(s, dev)) refuse("states must be on cuda:%d, got %s", dev, s.device().str().c_str());
        awq_state_t &a = all[i];
        a.row_bytes = dense_row(s, "a state");
        if (i == 0) rows_in = s.size(0);
        else if (s.size(0) != rows_in) refuse("states must have the same number of rows");
        if (given) {
            const Tensor &t = (*given)[i];
            if (t.scalar_type() != s.scalar_type() || !on(t, dev) || t.dim() != s.dim() || t.size(0) != rows ||
                t.sizes().slice(1) != s.sizes().slice(1))
                refuse("outs must be like the states, with a row for every parent");
            if (dense_row(t, "an out") != a.row_bytes) refuse("outs must be like the states");
            made.push_back(t);
        } else {
            std::vector<int64_t> sizes(s.sizes().begin(), s.sizes().end());
            sizes[0] = rows;
            made.push_back(at::empty(sizes, s.options()));
        }
        const int64_t size = s.element_size();
        a.src = s.data_ptr();
        a.dst = made[i].data_ptr();
        a.src_row_stride = rows_in > 1 ? s.stride(0) * size : a.row_bytes;
        a.dst_row_stride = rows > 1 ? made[i].stride(0) * size : a.row_bytes;
        if (rows_in > 0 && a.row_bytes > 0)
            from.push_back({reinterpret_cast<uintptr_t>(a.src), rows_in, a.src_row_stride, a.row_bytes});
        if (rows > 0 && a.row_bytes > 0)
            to.push_back({reinterpret_cast<uintptr_t>(a.dst), rows, a.dst_row_stride, a.row_bytes});
    }
    if (given)
        for (const Bytes &x : to)
            for (const Bytes &y : from)
                if (overlap(x, y)) refuse("outs must not overlap states");
    const awq_stream_t stream = stream_of(dev);
    const int status =
        call([&] { return reorder_entry(all.data(), n, data<int32_t>(&parents), rows, rows_in, stream); });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    PyObject *list = PyList_New(n);
    if (!list) throw Raised{};
    for (int64_t i = 0; i < n; ++i) PyList_SET_ITEM(list, i, THPVariable_Wrap(std::move(made[i])));
    return list;
}

PyObject *fork_pages(PyObject *const *o)
{
    const Tensor &table = tensor(o[0], "block_table"), &lens = tensor(o[1], "lens"), &parents = tensor(o[2], "parents");
    const Tensor &free_blocks = tensor(o[3], "free_blocks");
    const int64_t block_size = integer(o[4]);
    const int dev = cuda_index(table);
    check(lens, "lens", at::kInt, dev);
    const int64_t rows_in = lens.numel();
    int64_t width, stride;
    check_table(table, rows_in, dev, width, stride);
    check(parents, "parents", at::kInt, dev);
    check(free_blocks, "free_blocks", at::kInt, dev);
    const int32_t *start = checked<int32_t>(o[5], "free_start", at::kInt, dev, 1);
    const int64_t rows = parents.numel();
    if (rows > 16384) refuse("fork_pages takes up to 16384 rows, got %lld", (long long)rows);
    Area area(dev, rows * (width + 4) + 1);
    Tensor made = area.take(at::kInt, {rows, width}), made_lens = area.take(at::kInt, {rows}), src = area.take(at::kInt, {rows});
    Tensor dst = area.take(at::kInt, {rows}), tokens = area.take(at::kInt, {rows}), count = area.take(at::kInt, {1});
    const awq_stream_t stream = stream_of(dev);
    const int status = call([&] {
        return fork_entry(data<int32_t>(&table), rows_in, width, stride, data<int32_t>(&lens), data<int32_t>(&parents),
                          rows, data<int32_t>(&free_blocks), free_blocks.numel(), start, block_size, data<int32_t>(&made),
                          width, data<int32_t>(&made_lens), data<int32_t>(&src), data<int32_t>(&dst),
                          data<int32_t>(&tokens), data<int32_t>(&count), stream);
    });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    return tuple_of(made, made_lens, src, dst, tokens, count);
}

PyObject *copy_pages(PyObject *const *o)
{
    const Tensors caches(o[0], "caches");
    const Tensor &src = tensor(o[1], "src"), &dst = tensor(o[2], "dst");
    const int dev = cuda_index(src);
    check(src, "src", at::kInt, dev);
    check(dst, "dst", at::kInt, dev, src.numel());
    const int32_t *tokens = checked<int32_t>(o[3], "tokens", at::kInt, dev, src.numel());
    const int32_t *count = checked<int32_t>(o[4], "count", at::kInt, dev, 1);
    const int64_t n = caches.size();
    if (n == 0) return keep(Py_None);
    const Tensor &like = caches[0];
    const at::ScalarType type = like.scalar_type();
    if (type != at::kHalf && type != at::kBFloat16) refuse("the caches must be float16 or bfloat16, got %s", name_of(type));
    const awq_cache_t layout = cache(like, "a cache", type, dev, like);
    std::vector<void *> data_of(n);
    for (int64_t i = 0; i < n; ++i) {
        // an axis with one entry has no stride to differ in
        const awq_cache_t c = cache(caches[i], "a cache", type, dev, like);
        if (c.block_stride != layout.block_stride || c.token_stride != layout.token_stride ||
            c.head_stride != layout.head_stride)
            refuse("the caches must have the same strides");
        data_of[i] = c.data;
    }
    const awq_stream_t stream = stream_of(dev);
    const int status = call([&] {
        return copy_entry(data_of.data(), n, &layout, like.size(0), like.size(1), like.size(2), like.size(3),
                          data<int32_t>(&src), data<int32_t>(&dst), tokens, src.numel(), count, stream);
    });
    return status == AWQ_OK ? keep(Py_None) : PyLong_FromLong(status);
}

// What free_pages and compact_pages share.
struct Pages {
    const int32_t *table, *lens, *held;
    int64_t rows, width, stride, block_size, num_blocks, num_held, workspace;
    int dev;
};

Pages pages(PyObject *const *o)
{
    const Tensor &table = tensor(o[0], "block_table"), &lens = tensor(o[1], "lens");
    const Tensor *held = tensor_or_none(o[4], "held");
    Pages p{};
    p.block_size = integer(o[2]);
    p.num_blocks = integer(o[3]);
    p.dev = cuda_index(table);
    check(lens, "lens", at::kInt, p.dev);
    p.rows = lens.numel();
    check_table(table, p.rows, p.dev, p.width, p.stride);
    if (held) {
        check(*held, "held", at::kInt, p.dev);
        p.num_held = held->numel();
    }
    p.table = data<int32_t>(&table);
    p.lens = data<int32_t>(&lens);
    p.held = data<int32_t>(held);
    if (!pages_workspace_entry) refuse("the library is not bound");
    // the library's own limit, before memory of that size is asked for
    p.workspace = pages_workspace_entry(p.num_blocks);
    if (p.workspace < 0) refuse("num_blocks must be 1 to 2^28, got %lld", (long long)p.num_blocks);
    // Where the bitmap is in it, not among the allocator's blocks of up to 1 MB, which lie in segments of their own: free
    // pages of 2.5 million blocks 26.8 us, and 27.1 to 28 there
    if (p.workspace > 64 << 10) p.workspace = std::max<int64_t>(p.workspace, 2 << 20);
    return p;
}

PyObject *free_pages(PyObject *const *o)
{
    const Pages p = pages(o);
    const c10::DataPtr workspace = workspace_of(p.workspace);
    Area area(p.dev, p.num_blocks + 2);
    Tensor list = area.take(at::kInt, {p.num_blocks}), counts = area.take(at::kInt, {2});
    const awq_stream_t stream = stream_of(p.dev);
    const int status = call([&] {
        return free_entry(p.table, p.rows, p.width, p.stride, p.lens, p.block_size, p.num_blocks, p.held, p.num_held,
                          data<int32_t>(&list), data<int32_t>(&counts), workspace.get(), stream);
    });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    return tuple_of(list, counts);
}

PyObject *compact_pages(PyObject *const *o)
{
    const Pages p = pages(o);
    const int64_t half = p.num_blocks / 2;
    const c10::DataPtr workspace = workspace_of(p.workspace);
    Area area(p.dev, p.rows * p.width + p.num_blocks + 2 * half + 1);
    Tensor table = area.take(at::kInt, {p.rows, p.width}), map = area.take(at::kInt, {p.num_blocks});
    Tensor src = area.take(at::kInt, {half}), dst = area.take(at::kInt, {half}), count = area.take(at::kInt, {1});
    const awq_stream_t stream = stream_of(p.dev);
    const int status = call([&] {
        return compact_entry(p.table, p.rows, p.width, p.stride, p.lens, p.block_size, p.num_blocks, p.held, p.num_held,
                             data<int32_t>(&table), p.width, data<int32_t>(&map), data<int32_t>(&src),
                             data<int32_t>(&dst), data<int32_t>(&count), workspace.get(), stream);
    });
    if (status != AWQ_OK) return PyLong_FromLong(status);
    return tuple_of(table, map, src, dst, count);
}

template <typename F>
void set(F &entry, PyObject *address)
{
    entry = reinterpret_cast<F>(integer(address));
}

// Addresses of the library's entry points.
PyObject *bind(PyObject *const *o)
{
    set(append_entry, o[1]);
    set(attention_entry, o[2]);
    set(logits_entry, o[3]);
    set(rotary_entry, o[4]);
    set(beam_entry, o[5]);
    set(beam_workspace_entry, o[6]);
    set(reorder_entry, o[7]);
    set(fork_entry, o[8]);
    set(copy_entry, o[9]);
    set(free_entry, o[10]);
    set(compact_entry, o[11]);
    set(pages_workspace_entry, o[12]);
    set(plan_entry, o[0]);      // call() asks for this one
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

PyMethodDef methods[] = {method<bind, 13>("bind"),
                         method<paged_plan, 8>("paged_plan"),
                         method<kv_append, 5>("kv_append"),
                         method<tree_attention, 12>("tree_attention"),
                         method<process_logits, 17>("process_logits"),
                         method<rotary, 8>("rotary"),
                         method<rotary_append, 11>("rotary_append"),
                         method<beam_select, 4>("beam_select"),
                         method<reorder_states, 3>("reorder_states"),
                         method<fork_pages, 6>("fork_pages"),
                         method<copy_pages, 5>("copy_pages"),
                         method<free_pages, 5>("free_pages"),
                         method<compact_pages, 5>("compact_pages"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "awq_step", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit_awq_step() { return PyModule_Create(&definition); }
