// PyTorch binding of the cache, ragged-run and page-selection calls: checks the tensors and hands
// their pointers, the current stream and the sizes to the C library.  A decode step makes these
// calls once per layer, and each kernel takes a few microseconds: the same checks in Python took
// 10 to 40 microseconds a call, longer than the kernels.
//
// Every function takes positional arguments, raises ValueError for tensors that the call does not
// take, and returns the library's status (with the outputs that it allocated); the Python wrappers
// turn a status into an error.

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/mla_decode.h"

namespace {

constexpr int64_t kLatent = 512, kRope = 64, kFp8Row = 656;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string shape_text(std::initializer_list<int64_t> shape)
{
    std::string s = "[";
    for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
    return s + "]";
}

const at::Tensor& tensor_of(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

bool has_shape(const at::Tensor& t, std::initializer_list<int64_t> shape)
{
    if (t.dim() != static_cast<int64_t>(shape.size())) return false;
    int64_t i = 0;
    for (int64_t n : shape)
        if (t.size(i++) != n) return false;
    return true;
}

// A contiguous tensor of this type and shape on `dev`.
void need(const at::Tensor& t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, c10::Device dev)
{
    if (t.scalar_type() != type || !has_shape(t, shape) || !t.is_contiguous() || t.device() != dev)
        throw Refused(std::string(name) + " must be contiguous " + c10::toString(type) + " " + shape_text(shape) + " on " + dev.str());
}

// Rows of a 16-bit tensor that may be strided but for the last dimension.
void need_rows(const at::Tensor& t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, c10::Device dev)
{
    if (t.scalar_type() != type || !has_shape(t, shape) || t.device() != dev || t.stride(-1) != 1)
        throw Refused(std::string(name) + " must be " + c10::toString(type) + " " + shape_text(shape) + " on " + dev.str() +
                      " with a contiguous last dimension");
}

void need_ints(const at::Tensor& t, const char* name, int64_t dim, c10::Device dev)
{
    if (t.scalar_type() != at::kInt || t.dim() != dim || !t.is_contiguous() || t.device() != dev)
        throw Refused(std::string(name) + " must be a contiguous int32 tensor of " + std::to_string(dim) + " dimension(s) on " + dev.str());
}

// Stride of a dimension, 0 where it has one entry (and its stride says nothing).
int64_t stride_of(const at::Tensor& t, int64_t dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

int32_t* status_of(PyObject* o, c10::Device dev)
{
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor_of(o, "status");
    if (t.scalar_type() != at::kInt || t.numel() != 1 || t.device() != dev)
        throw Refused("status must be an int32 tensor of one value on " + dev.str());
    return t.data_ptr<int32_t>();
}

int as_int(int64_t v, const char* name)
{
    if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " does not fit 32 bits");
    return static_cast<int>(v);
}

int64_t int64_arg(PyObject* o, const char* name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + " must be an integer");
    }
    return v;
}

int int_arg(PyObject* o, const char* name) { return as_int(int64_arg(o, name), name); }

double float_arg(PyObject* o, const char* name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + " must be a number");
    }
    return v;
}

// A paged cache: 16-bit rows, or "FP8 with scale" bytes.
struct Cache {
    const at::Tensor& t;
    c10::Device dev;
    int dtype, d_qk, num_blocks, page, h_kv;
    at::ScalarType type;  // of the 16-bit tensors that go with it

    Cache(PyObject* o, bool fp8) : t(tensor_of(o, "kvcache")), dev(t.device())
    {
        if (!t.is_cuda() || !t.is_contiguous() || t.dim() != 4)
            throw Refused("kvcache must be a contiguous CUDA tensor [num_blocks, 64, h_kv, row]");
        if (fp8) {
            if (t.scalar_type() != at::kByte || t.size(3) != kFp8Row) throw Refused("an FP8 cache is a uint8 kvcache of 656-byte rows");
            dtype = MLA_BF16_FP8KV, d_qk = 576, type = at::kBFloat16;
        } else {
            type = t.scalar_type();
            if (type != at::kBFloat16 && type != at::kHalf)
                throw Refused("kvcache must be bfloat16 or float16 (or uint8 with is_fp8_kvcache)");
            dtype = type == at::kHalf ? MLA_FP16 : MLA_BF16, d_qk = as_int(t.size(3), "d_qk");
        }
        num_blocks = as_int(t.size(0), "num_blocks"), page = as_int(t.size(1), "page size"), h_kv = as_int(t.size(2), "h_kv");
    }
};

const void* ptr_or_null(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// append(latent, k_pe, positions, cos_sin, slots, kvcache, norm_weight, norm_eps, q_pe, q, interleaved, fp8, status)
PyObject* do_append(PyObject* const* a)
{
    const Cache c(a[5], a[11] == Py_True);
    const at::Tensor& slots = tensor_of(a[4], "slots");
    need_ints(slots, "slots", 1, c.dev);
    const int64_t tokens = slots.size(0);
    const bool rope = c.d_qk == 576;
    const at::Tensor& latent = tensor_of(a[0], "latent");
    need_rows(latent, "latent", c.type, {tokens, kLatent}, c.dev);
    const at::Tensor *k_pe = nullptr, *positions = nullptr, *cos_sin = nullptr, *weight = nullptr, *q_pe = nullptr, *q = nullptr;
    if (a[6] != Py_None) {
        weight = &tensor_of(a[6], "norm_weight");
        need(*weight, "norm_weight", c.type, {kLatent}, c.dev);
    }
    if (rope) {
        if (a[1] == Py_None || a[2] == Py_None || a[3] == Py_None) throw Refused("rows of 576 need k_pe, positions and cos_sin");
        k_pe = &tensor_of(a[1], "k_pe"), positions = &tensor_of(a[2], "positions"), cos_sin = &tensor_of(a[3], "cos_sin");
        need_rows(*k_pe, "k_pe", c.type, {tokens, kRope}, c.dev);
        need(*positions, "positions", at::kInt, {tokens}, c.dev);
        need(*cos_sin, "cos_sin", at::kFloat, {cos_sin->dim() == 2 ? cos_sin->size(0) : 0, kRope}, c.dev);
    } else if (a[1] != Py_None || a[8] != Py_None || a[9] != Py_None) {
        throw Refused("rows of 512 have no position columns");
    }
    if ((a[8] == Py_None) != (a[9] == Py_None)) throw Refused("q_pe and q come together");
    int64_t h_q = 0;
    if (a[9] != Py_None) {
        q_pe = &tensor_of(a[8], "q_pe"), q = &tensor_of(a[9], "q");
        if (q->dim() != 3 || (h_q = q->size(1)) == 0) throw Refused("q must be [tokens, h_q, 576] with at least one head");
        need_rows(*q, "q", c.type, {tokens, h_q, 576}, c.dev);
        need_rows(*q_pe, "q_pe", c.type, {tokens, h_q, kRope}, c.dev);
    }
    int32_t* status = status_of(a[12], c.dev);
    const double eps = float_arg(a[7], "norm_eps");
    if (tokens == 0) return PyLong_FromLong(MLA_OK);
    const c10::cuda::CUDAGuard guard(c.dev);
    return PyLong_FromLong(mla_append_kvcache(
        latent.data_ptr(), stride_of(latent, 0), ptr_or_null(k_pe), k_pe ? stride_of(*k_pe, 0) : 0, ptr_or_null(weight),
        static_cast<float>(eps), rope ? positions->data_ptr<int32_t>() : nullptr, rope ? cos_sin->data_ptr<float>() : nullptr,
        rope ? as_int(cos_sin->size(0), "max_position") : 0, slots.data_ptr<int32_t>(), as_int(tokens, "tokens"), c.t.data_ptr(),
        c.num_blocks, c.page, c.h_kv, c.d_qk, c.dtype, a[10] == Py_True, ptr_or_null(q_pe), q_pe ? stride_of(*q_pe, 0) : 0,
        q_pe ? stride_of(*q_pe, 1) : 0, const_cast<void*>(ptr_or_null(q)), q ? stride_of(*q, 0) : 0, q ? stride_of(*q, 1) : 0,
        as_int(h_q, "h_q"), status, stream_of(c.dev)));
}

void need_keys(const at::Tensor& keys, const at::Tensor& scales, int64_t num_blocks, int64_t d_qk, c10::Device dev)
{
    need(keys, "page_keys", at::kChar, {num_blocks, d_qk}, dev);
    need(scales, "page_scales", at::kFloat, {num_blocks}, dev);
}

// summarize(kvcache, block_table, prev_seqlens, cache_seqlens, page_keys, page_scales, fp8, status)
PyObject* do_summarize(PyObject* const* a)
{
    const Cache c(a[0], a[6] == Py_True);
    const at::Tensor &table = tensor_of(a[1], "block_table"), &prev = tensor_of(a[2], "prev_seqlens"),
                     &lens = tensor_of(a[3], "cache_seqlens"), &keys = tensor_of(a[4], "page_keys"),
                     &scales = tensor_of(a[5], "page_scales");
    need_ints(table, "block_table", 2, c.dev);
    const int64_t batch = table.size(0);
    need(prev, "prev_seqlens", at::kInt, {batch}, c.dev);
    need(lens, "cache_seqlens", at::kInt, {batch}, c.dev);
    need_keys(keys, scales, c.num_blocks, c.d_qk, c.dev);
    int32_t* status = status_of(a[7], c.dev);
    if (batch == 0 || table.size(1) == 0) return PyLong_FromLong(MLA_OK);
    const c10::cuda::CUDAGuard guard(c.dev);
    return PyLong_FromLong(mla_summarize_pages(c.t.data_ptr(), c.num_blocks, c.page, c.h_kv, c.d_qk, c.dtype, table.data_ptr<int32_t>(),
                                               as_int(table.size(1), "max_blocks"), prev.data_ptr<int32_t>(), lens.data_ptr<int32_t>(),
                                               as_int(batch, "batch"), keys.data_ptr<int8_t>(), scales.data_ptr<float>(), status,
                                               stream_of(c.dev)));
}

// select(q, page_keys, page_scales, block_table, cache_seqlens, topn, n_first, n_last, causal, status)
//   -> (status, page_table, page_seqlens)
PyObject* do_select(PyObject* const* a)
{
    const at::Tensor &q = tensor_of(a[0], "q"), &keys = tensor_of(a[1], "page_keys"), &scales = tensor_of(a[2], "page_scales"),
                     &table = tensor_of(a[3], "block_table"), &lens = tensor_of(a[4], "cache_seqlens");
    const c10::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    if (!q.is_cuda() || (type != at::kBFloat16 && type != at::kHalf) || q.dim() != 4 || !q.is_contiguous())
        throw Refused("q must be contiguous bfloat16 or float16 [b, s_q, h_q, d_qk] on a CUDA device");
    const int b = as_int(q.size(0), "b"), s_q = as_int(q.size(1), "s_q"), h_q = as_int(q.size(2), "h_q"), d_qk = as_int(q.size(3), "d_qk");
    if (keys.dim() != 2) throw Refused("page_keys must be int8 [num_blocks, d_qk]");
    need_keys(keys, scales, keys.size(0), d_qk, dev);
    need_ints(table, "block_table", 2, dev);
    if (table.size(0) != b) throw Refused("block_table must have one row per request");
    need(lens, "cache_seqlens", at::kInt, {b}, dev);
    const int max_blocks = as_int(table.size(1), "max_blocks");
    const int topn = int_arg(a[5], "topn"), first = int_arg(a[6], "n_first"), last = int_arg(a[7], "n_last");
    int32_t* status = status_of(a[9], dev);
    const size_t bytes = mla_select_workspace_bytes(b, s_q, h_q, d_qk, max_blocks);
    if (bytes == 0) throw Refused("invalid or unsupported sizes for the selection");
    const c10::cuda::CUDAGuard guard(dev);
    const int64_t tokens = static_cast<int64_t>(b) * s_q;
    at::Tensor out = at::empty({tokens, topn > 0 ? topn : 0}, table.options());
    at::Tensor out_lens = at::empty({tokens}, table.options());
    at::Tensor ws = at::empty({static_cast<int64_t>(bytes / 4 + 1)}, scales.options());
    const int st = mla_select_pages(q.data_ptr(), b, s_q, h_q, d_qk, type == at::kHalf ? MLA_FP16 : MLA_BF16, keys.data_ptr<int8_t>(),
                                    scales.data_ptr<float>(), as_int(keys.size(0), "num_blocks"), table.data_ptr<int32_t>(), max_blocks,
                                    lens.data_ptr<int32_t>(), a[8] == Py_True, topn, first, last, out.data_ptr<int32_t>(),
                                    out_lens.data_ptr<int32_t>(), ws.data_ptr(), ws.numel() * 4, status, stream_of(dev));
    return Py_BuildValue("(iNN)", st, THPVariable_Wrap(out), THPVariable_Wrap(out_lens));
}

// varlen_plan(cu_seqlens_q, cache_seqlens, total_q, h_q, h_kv, causal, fp8, num_parts, out) -> (status, num_parts, plan)
PyObject* do_varlen_plan(PyObject* const* a)
{
    const at::Tensor &cu = tensor_of(a[0], "cu_seqlens_q"), &lens = tensor_of(a[1], "cache_seqlens");
    const c10::Device dev = cu.device();
    if (!cu.is_cuda()) throw Refused("cu_seqlens_q must be on a CUDA device");
    need_ints(lens, "cache_seqlens", 1, dev);
    const int64_t batch = lens.size(0);
    need(cu, "cu_seqlens_q", at::kInt, {batch + 1}, dev);
    const int total_q = int_arg(a[2], "total_q"), h_q = int_arg(a[3], "h_q"), h_kv = int_arg(a[4], "h_kv");
    int parts = 0;
    if (a[7] != Py_None)
        parts = int_arg(a[7], "num_parts");
    else if (mla_num_sm_parts(dev.index(), &parts) != MLA_OK)
        return Py_BuildValue("(iOO)", MLA_ERR_CUDA, Py_None, Py_None);
    const int b = as_int(batch, "batch");
    const size_t ints = mla_varlen_plan_ints(b, total_q, h_q, h_kv, parts);
    if (ints == 0) throw Refused("invalid or unsupported sizes for the schedule");
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor plan;
    if (a[8] != Py_None) {
        plan = tensor_of(a[8], "out");
        need(plan, "out", at::kInt, {static_cast<int64_t>(ints)}, dev);
    } else {
        plan = at::empty({static_cast<int64_t>(ints)}, cu.options());
    }
    const int st = mla_get_metadata_varlen(cu.data_ptr<int32_t>(), lens.data_ptr<int32_t>(), b, total_q, h_q, h_kv, a[5] == Py_True, parts,
                                           a[6] == Py_True, plan.data_ptr<int32_t>(), stream_of(dev));
    return Py_BuildValue("(iiN)", st, parts, THPVariable_Wrap(plan));
}

// varlen(q, kvcache, block_table, cu_seqlens_q, cache_seqlens, dv, plan, num_parts, softmax_scale, fp8, workspace, out, lse, status,
//        max_scratch_bytes)
//   -> (status, out, lse)
PyObject* do_varlen(PyObject* const* a)
{
    const Cache c(a[1], a[9] == Py_True);
    const at::Tensor &q = tensor_of(a[0], "q"), &table = tensor_of(a[2], "block_table"), &cu = tensor_of(a[3], "cu_seqlens_q"),
                     &lens = tensor_of(a[4], "cache_seqlens"), &plan = tensor_of(a[6], "plan"), &ws = tensor_of(a[10], "workspace");
    if (q.dim() != 3) throw Refused("q must be [total_q, h_q, d_qk]");
    const int64_t total_q = q.size(0), h_q = q.size(1);
    need(q, "q", c.type, {total_q, h_q, c.d_qk}, c.dev);
    need_ints(table, "block_table", 2, c.dev);
    const int64_t batch = table.size(0);
    need(lens, "cache_seqlens", at::kInt, {batch}, c.dev);
    need(cu, "cu_seqlens_q", at::kInt, {batch + 1}, c.dev);
    const int dv = int_arg(a[5], "dv"), parts = int_arg(a[7], "num_parts");
    const size_t ints = mla_varlen_plan_ints(as_int(batch, "batch"), as_int(total_q, "total_q"), as_int(h_q, "h_q"), c.h_kv, parts);
    if (ints == 0) return Py_BuildValue("(iOO)", MLA_ERR_UNSUPPORTED, Py_None, Py_None);
    need(plan, "plan", at::kInt, {static_cast<int64_t>(ints)}, c.dev);
    int32_t* status = status_of(a[13], c.dev);
    if (ws.device() != c.dev || !ws.is_contiguous()) throw Refused("workspace must be contiguous and on " + c.dev.str());
    const c10::cuda::CUDAGuard guard(c.dev);
    at::Tensor out, lse;
    if (a[11] != Py_None) {
        out = tensor_of(a[11], "out");
        need(out, "out", c.type, {total_q, h_q, dv}, c.dev);
    } else {
        out = at::empty({total_q, h_q, dv > 0 ? dv : 0}, q.options());
    }
    if (a[12] != Py_None) {
        lse = tensor_of(a[12], "lse");
        need(lse, "lse", at::kFloat, {total_q, h_q}, c.dev);
    } else {
        lse = at::empty({total_q, h_q}, q.options().dtype(at::kFloat));
    }
    // FP8 pages that several groups read are dequantized once, into memory of this call alone, or, where the
    // caller or the device has not that much to give, at every read
    size_t scratch_bytes = c.dtype != MLA_BF16_FP8KV ? 0
        : mla_decode_varlen_scratch_bytes(static_cast<int>(batch), static_cast<int>(total_q), static_cast<int>(h_q),
                                          as_int(table.size(1), "max_blocks"), c.dtype);
    if (a[14] != Py_None) {
        const int64_t most = int64_arg(a[14], "max_scratch_bytes");
        if (most < 0) throw Refused("max_scratch_bytes must not be negative");
        if (scratch_bytes > static_cast<size_t>(most)) scratch_bytes = 0;
    }
    at::Tensor scratch;
    if (scratch_bytes) {
        try {
            scratch = at::empty({static_cast<int64_t>(scratch_bytes)}, c.t.options());
        } catch (const c10::OutOfMemoryError&) {
            scratch_bytes = 0;
        }
    }
    int st = MLA_OK;
    if (batch != 0 && total_q != 0)
        st = mla_decode_varlen_status(q.data_ptr(), static_cast<int>(total_q), static_cast<int>(h_q), c.d_qk, c.t.data_ptr(), c.num_blocks, c.page,
                               c.h_kv, table.data_ptr<int32_t>(), static_cast<int>(batch), as_int(table.size(1), "max_blocks"),
                               lens.data_ptr<int32_t>(), dv, c.dtype,
                               plan.data_ptr<int32_t>(), parts, static_cast<float>(float_arg(a[8], "softmax_scale")), out.data_ptr(),
                               lse.data_ptr<float>(), ws.data_ptr(), ws.numel() * ws.element_size(),
                               scratch_bytes ? scratch.data_ptr() : nullptr, scratch_bytes, status, stream_of(c.dev));
    return Py_BuildValue("(iNN)", st, THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// No C++ exception leaves an entry point.
template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != kArgs) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return kFn(args);
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {  // torch: out of memory and the like
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kFn, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<do_append, 13>("append"),
    method<do_summarize, 8>("summarize"),
    method<do_select, 10>("select"),
    method<do_varlen_plan, 9>("varlen_plan"),
    method<do_varlen, 15>("varlen"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_mla_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_torch() { return PyModule_Create(&module_def); }
