// kv_binding.cpp -- the Python side of the paged cache's three calls of a step:
// argument checks, output tensors, one call of the C ABI each.
//
// A decode step makes these calls in every layer, and on the kernels' few
// microseconds the checks and allocations of a Python function weigh more than
// the kernels themselves (block tables of 8 requests: 24 us a call with the
// checks in Python, the kernel 3 us).  The entry points of the library are handed
// in as addresses, so this module links against torch alone.
#include <ATen/ATen.h>
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
Table table(const Tensor& t, int64_t rows, int64_t dev)
{
    on_device(t, "block_table", dev);
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != rows ||
        (t.size(1) > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < t.size(1)))
        refuse("block_table must be int32 [" + std::to_string(rows) +
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

// attention(cache, device, q, block_table, seq_len, q_start or None, max_q or None,
// scale or None, window, out or None, output dtype (0: q's, 1: float32, 2: bfloat16),
// with lse, options, workspace, workspace bytes, stream) -> out, or (out, lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 16)
        refuse("attention takes 16 arguments");
    const nvfp4_kv_cache* c = cache_of(a[0]);
    const int64_t dev = integer(a[1]), dim = c->head_dim;
    const Tensor& q = tensor(a[2], "q");
    nvfp4_kv_attention_args r = {};
    r.q_stride = heads_stride(q, "q", dev, dim);
    r.q = q.data_ptr();
    r.tokens = q.size(0);
    r.num_q_heads = q.size(1);
    const Tensor& seq_len = tensor(a[4], "seq_len");
    r.seq_len = vector<int32_t>(seq_len, at::kInt, "seq_len", dev);
    r.reqs = seq_len.size(0);
    if (a[5] != Py_None)
        r.q_start = vector<int32_t>(tensor(a[5], "q_start"), at::kInt, "q_start", dev, r.reqs + 1);
    else if (r.reqs && r.tokens % r.reqs)
        refuse("without q_start every request has the same number of rows");
    if (r.num_q_heads % c->num_kv_heads)
        refuse(std::to_string(r.num_q_heads) + " query heads do not share " +
               std::to_string(c->num_kv_heads) + " kv heads");
    const Table t = table(tensor(a[3], "block_table"), r.reqs, dev);
    r.block_table = t.p;
    r.table_stride = t.stride;
    r.max_blocks = t.blocks;
    r.max_q = a[6] != Py_None ? integer(a[6])
              : r.q_start     ? r.tokens
                              : (r.reqs ? r.tokens / r.reqs : 0);
    r.scale = a[7] != Py_None ? (float)number(a[7]) : 1.0f / std::sqrt((float)dim);
    r.window = integer(a[8]);
    Tensor out, lse;
    // rows of no request are written where the memory is new, left alone in a given output
    const bool new_out = a[9] == Py_None;
    if (new_out) {
        const int64_t type = integer(a[10]);
        out = at::empty({r.tokens, r.num_q_heads, dim},
                        q.options().dtype(type == 0   ? q.scalar_type()
                                          : type == 1 ? at::kFloat
                                                      : at::kBFloat16));
        r.out_stride = r.num_q_heads * dim;
    } else {
        out = tensor(a[9], "out");
        if (out.sizes() != q.sizes())
            refuse("out must have q's shape");
        r.out_stride = heads_stride(out, "out", dev, dim);
    }
    r.out = out.data_ptr();
    const bool with_lse = PyObject_IsTrue(a[11]) == 1;
    if (with_lse) {
        const auto lse_options = q.options().dtype(at::kFloat);
        lse = new_out ? at::empty({r.tokens, r.num_q_heads}, lse_options)
                      : at::full({r.tokens, r.num_q_heads}, -INFINITY, lse_options);
        r.lse = static_cast<float*>(lse.data_ptr());
    }
    const uint32_t options = (uint32_t)integer(a[12]) |
                             (q.scalar_type() == at::kBFloat16 ? NVFP4_FLAG_X_BF16 : 0u) |
                             (out.scalar_type() == at::kBFloat16 ? NVFP4_FLAG_Y_BF16 : 0u) |
                             (new_out ? NVFP4_FLAG_ALL_ROWS : 0u);
    if (failed("nvfp4_kv_attention", fn_attention(c, &r, options, address(a[13]),
                                                  (size_t)integer(a[14]), address(a[15]))))
        return nullptr;
    if (!with_lse)
        return THPVariable_Wrap(out);
    PyObject* pair = PyTuple_New(2);
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(lse));
    return pair;
    END_HANDLE_TH_ERRORS
}

// bind(address of nvfp4_kv_tables, of nvfp4_kv_append, of nvfp4_kv_attention, Nvfp4Error)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 4)
        refuse("bind takes 4 arguments");
    fn_tables = reinterpret_cast<decltype(fn_tables)>(address(a[0]));
    fn_append = reinterpret_cast<decltype(fn_append)>(address(a[1]));
    fn_attention = reinterpret_cast<decltype(fn_attention)>(address(a[2]));
    Py_INCREF(a[3]);
    Py_XDECREF(error_class);
    error_class = a[3];
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
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_binding()
{
    return PyModule_Create(&module);
}
