// kv_binding.cpp -- the Python side of the paged cache's calls of a step:
// argument checks, output tensors, one call of the C ABI each.
//
// A decode step makes these calls in every layer, and on the kernels' few
// microseconds the checks and allocations of a Python function weigh more than
// the kernels themselves (block tables of 8 requests: 24 us a call with the
// checks in Python, the kernel 3 us).  The entry points of the library are handed
// in as addresses, so this module links against torch alone.
#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "../../include/nvfp4_kv.h"

namespace {

using at::Tensor;

decltype(&nvfp4_kv_tables) fn_tables = nullptr;
decltype(&nvfp4_kv_append) fn_append = nullptr;
decltype(&nvfp4_kv_attention) fn_attention = nullptr;
decltype(&nvfp4_kv_append_rotary) fn_rotary = nullptr;
decltype(&nvfp4_kv_cross_attention) fn_cross = nullptr;
decltype(&nvfp4_kv_attention_shared) fn_shared = nullptr;
decltype(&nvfp4_kv_shared_scratch_size) fn_scratch = nullptr;
PyObject* error_class = nullptr;  // Nvfp4Error(function, status)

// A failed check: a ValueError with this text.
[[noreturn]] void refuse(const std::string& text)
{
    PyErr_SetString(PyExc_ValueError, text.c_str());
    throw python_error();
}

const Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o))
        refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

void on_device(const Tensor& t, const char* name, int64_t dev)
{
    if (!t.is_cuda() || (dev >= 0 && t.get_device() != dev))
        refuse(std::string(name) + " must be a CUDA tensor" +
               (dev >= 0 ? " on device " + std::to_string(dev) : ""));
}

// A contiguous vector of n elements (any number if n < 0).
template <typename T>
T* vector(const Tensor& t, at::ScalarType type, const char* name, int64_t dev, int64_t n = -1)
{
    on_device(t, name, dev);
    if (t.scalar_type() != type)
        refuse(std::string(name) + " must be " + at::toString(type) + ", got " +
               at::toString(t.scalar_type()));
    if (t.dim() != 1 || !t.is_contiguous() || (n >= 0 && t.size(0) != n))
        refuse(std::string(name) + " must be a contiguous vector" +
               (n >= 0 ? " of " + std::to_string(n) : ""));
    return static_cast<T*>(t.data_ptr());
}

struct Table {
    int32_t* p;
    int64_t stride, blocks;
};

// A block table [rows][blocks] with contiguous rows.
Table table(const Tensor& t, int64_t rows, int64_t dev, const char* name = "block_table")
{
    on_device(t, name, dev);
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != rows ||
        (t.size(1) > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < t.size(1)))
        refuse(std::string(name) + " must be int32 [" + std::to_string(rows) +
               ", blocks] with contiguous rows");
    return {static_cast<int32_t*>(t.data_ptr()), rows > 1 ? t.stride(0) : t.size(1), t.size(1)};
}

// Token stride of [tokens][heads][dim] whose token rows are contiguous.
int64_t heads_stride(const Tensor& t, const char* name, int64_t dev, int64_t dim)
{
    on_device(t, name, dev);
    if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
        refuse(std::string(name) + " must be float32 or bfloat16, got " +
               at::toString(t.scalar_type()));
    if (t.dim() != 3 || t.size(2) != dim)
        refuse(std::string(name) + " must be [tokens, heads, " + std::to_string(dim) + "]");
    const int64_t row = t.size(1) * dim;
    if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != dim) ||
        (t.size(0) > 1 && t.stride(0) < row))
        refuse(std::string(name) + ": the heads of a token must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : row;
}

// An uninitialised tensor on like's device, from the allocator that like came from (the way over
// the dispatcher takes 1.4 us, a third of a small call).
Tensor new_tensor(const Tensor& like, at::IntArrayRef sizes, at::ScalarType type)
{
    c10::Allocator* from = like.storage().allocator();
    if (!from)
        return at::empty(sizes, like.options().dtype(type));
    return at::detail::empty_generic(sizes, from, c10::DispatchKeySet(c10::DispatchKey::CUDA), type,
                                     std::nullopt);
}

bool failed(const char* name, int status)
{
    if (status == NVFP4_OK)
        return false;
    PyObject* args = Py_BuildValue("(si)", name, status);
    PyObject* e = args ? PyObject_CallObject(error_class, args) : nullptr;
    if (e)
        PyErr_SetObject(error_class, e);
    Py_XDECREF(e);
    Py_XDECREF(args);
    return true;
}

int64_t integer(PyObject* o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}

void* address(PyObject* o)
{
    return reinterpret_cast<void*>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(o)));
}

// The cache's descriptor as the caller keeps it (bytes).
const nvfp4_kv_cache* cache_of(PyObject* o)
{
    if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != (Py_ssize_t)sizeof(nvfp4_kv_cache))
        refuse("not a cache descriptor");
    return reinterpret_cast<const nvfp4_kv_cache*>(PyBytes_AS_STRING(o));
}

// New vectors of these sizes on like's device, the third int64 and the others int32,
// as parts of one allocation, each from a 16-byte boundary on (five allocations: 12 us
// a call, one: 7).
void make_vectors(const Tensor& like, const int64_t (&sizes)[5], Tensor (&out)[5])
{
    int64_t at[6] = {0};
    for (int i = 0; i < 5; ++i)
        at[i + 1] = at[i] + (sizes[i] * (i == 2 ? 8 : 4) + 15) / 16 * 16;
    const Tensor all = at::empty({at[5]}, like.options().dtype(at::kByte));
    for (int i = 0; i < 5; ++i) {
        const at::ScalarType type = i == 2 ? at::kLong : at::kInt;
        out[i] = at::detail::make_tensor<c10::TensorImpl>(
            c10::Storage(all.storage()), all.key_set(), at::scalarTypeToTypeMeta(type));
        c10::TensorImpl* impl = out[i].unsafeGetTensorImpl();
        impl->set_storage_offset(at[i] / (i == 2 ? 8 : 4));
        impl->set_sizes_contiguous({&sizes[i], 1});
    }
}

// tables(kv_len, q_len, free_pages, free_head, block_table, page_size, tokens, out or
// None, options, stream) -> (seq_len, q_start, slots, positions, free_head)
PyObject* tables(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 10)
        refuse("tables takes 10 arguments");
    const Tensor& kv_len = tensor(a[0], "kv_len");
    const int32_t* p_len = vector<int32_t>(kv_len, at::kInt, "kv_len", -1);
    const int64_t dev = kv_len.get_device(), reqs = kv_len.size(0);
    const int32_t* p_new = vector<int32_t>(tensor(a[1], "q_len"), at::kInt, "q_len", dev, reqs);
    const Tensor& free_pages = tensor(a[2], "free_pages");
    const int32_t* p_free = vector<int32_t>(free_pages, at::kInt, "free_pages", dev);
    const int32_t* p_head = vector<int32_t>(tensor(a[3], "free_head"), at::kInt, "free_head", dev, 1);
    const Table t = table(tensor(a[4], "block_table"), reqs, dev);
    const int64_t page_size = integer(a[5]), tokens = integer(a[6]);
    if (tokens < 0)
        refuse("tokens must not be negative");
    PyObject* result;
    Tensor out[5];
    static const char* const names[5] = {"seq_len", "q_start", "slots", "positions", "free_head"};
    const int64_t sizes[5] = {reqs, reqs + 1, tokens, tokens, 1};
    if (a[7] == Py_None) {
        make_vectors(kv_len, sizes, out);
        result = PyTuple_New(5);
        for (int i = 0; i < 5; ++i)
            PyTuple_SET_ITEM(result, i, THPVariable_Wrap(out[i]));
    } else {
        if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 5)
            refuse("out must be a KVTables");
        for (int i = 0; i < 5; ++i) {
            out[i] = tensor(PyTuple_GET_ITEM(a[7], i), names[i]);
            vector<void>(out[i], i == 2 ? at::kLong : at::kInt, names[i], dev, sizes[i]);
        }
        result = a[7];
        Py_INCREF(result);
    }
    const int status = fn_tables(
        p_len, p_new, reqs, page_size, p_free, free_pages.size(0), p_head, t.p, t.stride, t.blocks,
        static_cast<int32_t*>(out[0].data_ptr()), static_cast<int32_t*>(out[1].data_ptr()),
        static_cast<int64_t*>(out[2].data_ptr()), static_cast<int32_t*>(out[3].data_ptr()), tokens,
        static_cast<int32_t*>(out[4].data_ptr()), (uint32_t)integer(a[8]), address(a[9]));
    if (failed("nvfp4_kv_tables", status)) {
        Py_DECREF(result);
        return nullptr;
    }
    return result;
    END_HANDLE_TH_ERRORS
}

// append(cache, device, k, v, slots, options, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 7)
        refuse("append takes 7 arguments");
    const nvfp4_kv_cache* c = cache_of(a[0]);
    const int64_t dev = integer(a[1]);
    const Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
    const int64_t ks = heads_stride(k, "k", dev, c->head_dim);
    const int64_t vs = heads_stride(v, "v", dev, c->head_dim);
    if (k.size(1) != c->num_kv_heads || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
        refuse("k and v must be [tokens, " + std::to_string(c->num_kv_heads) + ", " +
               std::to_string(c->head_dim) + "] of one dtype");
    const int64_t* slots =
        vector<int64_t>(tensor(a[4], "slots"), at::kLong, "slots", dev, k.size(0));
    const uint32_t options = (uint32_t)integer(a[5]) |
                             (k.scalar_type() == at::kBFloat16 ? NVFP4_FLAG_X_BF16 : 0u);
    if (failed("nvfp4_kv_append", fn_append(c, k.data_ptr(), ks, v.data_ptr(), vs, k.size(0), slots,
                                            options, address(a[6]))))
        return nullptr;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// append_rotary(cache, device, q or None, k, v, slots, positions, rotary, interleaved, out or None,
// options, stream) -> the turned queries, or None
PyObject* append_rotary(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 12)
        refuse("append_rotary takes 12 arguments");
    const nvfp4_kv_cache* c = cache_of(a[0]);
    const int64_t dev = integer(a[1]), dim = c->head_dim;
    const Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
    nvfp4_kv_rotary_args r = {};
    r.k_stride = heads_stride(k, "k", dev, dim);
    r.v_stride = heads_stride(v, "v", dev, dim);
    if (k.size(1) != c->num_kv_heads || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
        refuse("k and v must be [tokens, " + std::to_string(c->num_kv_heads) + ", " + std::to_string(dim) +
               "] of one dtype");
    r.k = k.data_ptr();
    r.v = v.data_ptr();
    r.tokens = k.size(0);
    r.slots = vector<int64_t>(tensor(a[5], "slots"), at::kLong, "slots", dev, r.tokens);
    r.positions = vector<int32_t>(tensor(a[6], "positions"), at::kInt, "positions", dev, r.tokens);
    const Tensor& rotary = tensor(a[7], "rotary");
    on_device(rotary, "rotary", dev);
    if (rotary.scalar_type() != at::kFloat || rotary.dim() != 2 || rotary.size(1) < 1 || rotary.size(1) > dim ||
        (rotary.size(1) > 1 && rotary.stride(1) != 1) ||
        (rotary.size(0) > 1 && rotary.stride(0) < rotary.size(1)))
        refuse("rotary must be float32 [positions, elements of a head that are turned] with contiguous rows");
    r.rotary = static_cast<const float*>(rotary.data_ptr());
    r.rotary_rows = rotary.size(0);
    r.rotary_stride = r.rotary_rows > 1 ? rotary.stride(0) : rotary.size(1);
    r.rotary_dim = (int32_t)rotary.size(1);
    const int interleaved = PyObject_IsTrue(a[8]);
    if (interleaved < 0)
        throw python_error();
    r.interleaved = interleaved;
    Tensor out;
    if (a[2] != Py_None) {
        const Tensor& q = tensor(a[2], "q");
        r.q_stride = heads_stride(q, "q", dev, dim);
        if (q.size(0) != r.tokens || q.scalar_type() != k.scalar_type())
            refuse("q must have the tokens and the dtype of k");
        if (a[9] == Py_None) {
            out = new_tensor(q, q.sizes(), q.scalar_type());
            r.q_out_stride = q.size(1) * dim;
        } else {
            out = tensor(a[9], "out");
            r.q_out_stride = heads_stride(out, "out", dev, dim);
            if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type())
                refuse("out must have q's shape and dtype");
        }
        r.q = q.data_ptr();
        r.q_out = out.data_ptr();
        r.num_q_heads = q.size(1);
    } else if (a[9] != Py_None) {
        refuse("out is for the turned queries: there are none");
    }
    const uint32_t options = (uint32_t)integer(a[10]) |
                             (k.scalar_type() == at::kBFloat16 ? NVFP4_FLAG_X_BF16 : 0u);
    if (failed("nvfp4_kv_append_rotary", fn_rotary(c, &r, options, address(a[11]))))
        return nullptr;
    if (!out.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// The operands that every attention call has, checked; its outputs.
struct Attention {
    nvfp4_kv_attention_args r = {};
    Tensor out, lse;
    uint32_t options = 0;

    // q, block_table, seq_len, q_start or None, max_q or None, scale or None, window or None (none),
    // out or None, output dtype (0: q's, 1: float32, 2: bfloat16), with lse, options
    Attention(const nvfp4_kv_cache* c, int64_t dev, PyObject* q_, PyObject* table_, PyObject* seq_len_,
              PyObject* q_start_, PyObject* max_q_, PyObject* scale_, PyObject* window_, PyObject* out_,
              PyObject* type_, PyObject* lse_, PyObject* options_)
    {
        const int64_t dim = c->head_dim;
        const Tensor& q = tensor(q_, "q");
        r.q_stride = heads_stride(q, "q", dev, dim);
        r.q = q.data_ptr();
        r.tokens = q.size(0);
        r.num_q_heads = q.size(1);
        const Tensor& seq_len = tensor(seq_len_, "seq_len");
        r.seq_len = vector<int32_t>(seq_len, at::kInt, "seq_len", dev);
        r.reqs = seq_len.size(0);
        if (q_start_ != Py_None)
            r.q_start = vector<int32_t>(tensor(q_start_, "q_start"), at::kInt, "q_start", dev, r.reqs + 1);
        else if (r.reqs && r.tokens % r.reqs)
            refuse("without q_start every request has the same number of rows");
        if (r.num_q_heads % c->num_kv_heads)
            refuse(std::to_string(r.num_q_heads) + " query heads do not share " +
                   std::to_string(c->num_kv_heads) + " kv heads");
        const Table t = table(tensor(table_, "block_table"), r.reqs, dev);
        r.block_table = t.p;
        r.table_stride = t.stride;
        r.max_blocks = t.blocks;
        r.max_q = max_q_ != Py_None ? integer(max_q_)
                  : r.q_start       ? r.tokens
                                    : (r.reqs ? r.tokens / r.reqs : 0);
        r.scale = scale_ != Py_None ? (float)number(scale_) : 1.0f / std::sqrt((float)dim);
        r.window = window_ ? integer(window_) : 0;
        // rows of no request are written where the memory is new, left alone in a given output
        const bool new_out = out_ == Py_None;
        if (new_out) {
            const int64_t type = integer(type_);
            out = new_tensor(q, {r.tokens, r.num_q_heads, dim},
                             type == 0 ? q.scalar_type() : type == 1 ? at::kFloat : at::kBFloat16);
            r.out_stride = r.num_q_heads * dim;
        } else {
            out = tensor(out_, "out");
            if (out.sizes() != q.sizes())
                refuse("out must have q's shape");
            r.out_stride = heads_stride(out, "out", dev, dim);
        }
        r.out = out.data_ptr();
        if (PyObject_IsTrue(lse_) == 1) {
            lse = new_out ? new_tensor(q, {r.tokens, r.num_q_heads}, at::kFloat)
                          : at::full({r.tokens, r.num_q_heads}, -INFINITY, q.options().dtype(at::kFloat));
            r.lse = static_cast<float*>(lse.data_ptr());
        }
        options = (uint32_t)integer(options_) |
                  (q.scalar_type() == at::kBFloat16 ? NVFP4_FLAG_X_BF16 : 0u) |
                  (out.scalar_type() == at::kBFloat16 ? NVFP4_FLAG_Y_BF16 : 0u) |
                  (new_out ? NVFP4_FLAG_ALL_ROWS : 0u);
    }

    // out, or (out, lse)
    PyObject* result() const
    {
        if (!lse.defined())
            return THPVariable_Wrap(out);
        PyObject* pair = PyTuple_New(2);
        PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
        PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(lse));
        return pair;
    }
};

// attention(cache, device, q, block_table, seq_len, q_start or None, max_q or None,
// scale or None, window, out or None, output dtype, with lse, options, workspace, workspace
// bytes, stream) -> out, or (out, lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 16)
        refuse("attention takes 16 arguments");
    const nvfp4_kv_cache* c = cache_of(a[0]);
    const Attention t(c, integer(a[1]), a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12]);
    if (failed("nvfp4_kv_attention", fn_attention(c, &t.r, t.options, address(a[13]),
                                                  (size_t)integer(a[14]), address(a[15]))))
        return nullptr;
    return t.result();
    END_HANDLE_TH_ERRORS
}

// cross_attention(cache, device, q, block_table, seq_len, q_start or None, max_q or None, scale or
// None, out or None, output dtype, with lse, options, workspace, workspace bytes, stream)
PyObject* cross_attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 15)
        refuse("cross_attention takes 15 arguments");
    const nvfp4_kv_cache* c = cache_of(a[0]);
    const Attention t(c, integer(a[1]), a[2], a[3], a[4], a[5], a[6], a[7], nullptr, a[8], a[9], a[10], a[11]);
    if (failed("nvfp4_kv_cross_attention", fn_cross(c, &t.r, t.options, address(a[12]),
                                                    (size_t)integer(a[13]), address(a[14]))))
        return nullptr;
    return t.result();
    END_HANDLE_TH_ERRORS
}

// attention_shared(cache, device, q, prefix_table, prefix_len, group_start or None, block_table,
// seq_len, q_start or None, max_q or None, scale or None, out or None, output dtype, with lse,
// options, workspace, workspace bytes, stream)
PyObject* attention_shared(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 18)
        refuse("attention_shared takes 18 arguments");
    const nvfp4_kv_cache* c = cache_of(a[0]);
    const int64_t dev = integer(a[1]);
    const Attention t(c, dev, a[2], a[6], a[7], a[8], a[9], a[10], nullptr, a[11], a[12], a[13], a[14]);
    nvfp4_kv_prefixes p = {};
    const Tensor& prefix_len = tensor(a[4], "prefix_len");
    p.prefix_len = vector<int32_t>(prefix_len, at::kInt, "prefix_len", dev);
    p.groups = prefix_len.size(0);
    if (a[5] != Py_None)
        p.group_start = vector<int32_t>(tensor(a[5], "group_start"), at::kInt, "group_start", dev, p.groups + 1);
    else if (p.groups > 1)
        refuse("without group_start there is one group of all requests");
    const Table s = table(tensor(a[3], "prefix_table"), p.groups, dev, "prefix_table");
    p.block_table = s.p;
    p.table_stride = s.stride;
    p.max_blocks = s.blocks;
    Tensor scratch;
    if (p.groups) {
        const int64_t size = fn_scratch(t.r.tokens, t.r.num_q_heads, c->head_dim);
        if (size < 0) {
            failed("nvfp4_kv_shared_scratch_size", (int)-size);
            return nullptr;
        }
        scratch = new_tensor(tensor(a[2], "q"), {size}, at::kByte);
        p.scratch = scratch.data_ptr();
        p.scratch_bytes = (size_t)size;
    }
    if (failed("nvfp4_kv_attention_shared", fn_shared(c, &t.r, &p, t.options, address(a[15]),
                                                      (size_t)integer(a[16]), address(a[17]))))
        return nullptr;
    return t.result();
    END_HANDLE_TH_ERRORS
}

// bind(the addresses of nvfp4_kv_tables, _append, _attention, _append_rotary, _cross_attention,
// _attention_shared and _shared_scratch_size, Nvfp4Error)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 8)
        refuse("bind takes 8 arguments");
    fn_tables = reinterpret_cast<decltype(fn_tables)>(address(a[0]));
    fn_append = reinterpret_cast<decltype(fn_append)>(address(a[1]));
    fn_attention = reinterpret_cast<decltype(fn_attention)>(address(a[2]));
    fn_rotary = reinterpret_cast<decltype(fn_rotary)>(address(a[3]));
    fn_cross = reinterpret_cast<decltype(fn_cross)>(address(a[4]));
    fn_shared = reinterpret_cast<decltype(fn_shared)>(address(a[5]));
    fn_scratch = reinterpret_cast<decltype(fn_scratch)>(address(a[6]));
    Py_INCREF(a[7]);
    Py_XDECREF(error_class);
    error_class = a[7];
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    {"tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&tables)), METH_FASTCALL,
     nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&append)), METH_FASTCALL,
     nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&attention)),
     METH_FASTCALL, nullptr},
    {"append_rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&append_rotary)),
     METH_FASTCALL, nullptr},
    {"cross_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&cross_attention)),
     METH_FASTCALL, nullptr},
    {"attention_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&attention_shared)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_binding()
{
    return PyModule_Create(&module);
}
