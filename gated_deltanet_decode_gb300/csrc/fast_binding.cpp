// The Python binding's calls of the attention layers, in C++: the same checks
// and the same C ABI as the functions of the package, without a Python call for
// every property of every tensor.  A decode step makes these calls per layer,
// and each took 10 to 12 us of host time, as much as its kernels on the GPU.
//
// A call that the checks here do not pass gets None, and the package goes its
// own way, which says what is wrong.  A call that the C ABI refuses gets the
// status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gdn_decode.h"

namespace {

decltype(&attn_prologue) c_prologue;
decltype(&paged_attention_workspace_bytes) c_workspace;
decltype(&paged_attention) c_attention;
decltype(&kv_pages_fork) c_fork;
decltype(&kv_pages_free) c_free;
decltype(&kv_pages_copy) c_copy;

struct Pool {
    kv_page_pool *handle;
    int hkv, d, code, device;
    at::ScalarType type;
};

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool plain(const at::Tensor &t, at::ScalarType type, int device)
{
    return t.scalar_type() == type && t.is_cuda() && t.get_device() == device && t.is_contiguous();
}

enum Takes { kExactly, kOrNone, kOrMore };

// A contiguous tensor of n elements; also None (a null pointer), or more elements, where that is taken.
struct Arg {
    const void *p = nullptr;
    bool ok = false;
    Arg(PyObject *o, int64_t n, at::ScalarType type, int device, Takes takes = kExactly)
    {
        if (takes == kOrNone && o == Py_None) {
            ok = true;
            return;
        }
        const at::Tensor *t = tensor(o);
        if (t && (t->numel() == n || (takes == kOrMore && t->numel() > n)) && plain(*t, type, device))
            p = t->const_data_ptr(), ok = true;
    }
    template <typename T> T *as() const { return static_cast<T *>(const_cast<void *>(p)); }
};

// [tokens][heads][d] whose tokens may be apart
struct Tokens {
    const void *p = nullptr;
    int64_t tokens = 0, heads = 0, stride = 0;
    bool ok = false;
    Tokens(PyObject *o, const Pool &pool)
    {
        const at::Tensor *t = tensor(o);
        if (!t || t->dim() != 3 || t->scalar_type() != pool.type || !t->is_cuda() || t->get_device() != pool.device)
            return;
        const auto size = t->sizes(), step = t->strides();
        tokens = size[0], heads = size[1];
        stride = tokens > 1 ? step[0] : heads * pool.d;
        ok = size[2] == pool.d && step[2] == 1 && (step[1] == pool.d || heads == 1);
        p = t->const_data_ptr();
    }
};

struct Table {
    int32_t *p = nullptr;
    int rows = 0, width = 0, device = -1;
    bool ok = false;
    explicit Table(PyObject *o)
    {
        const at::Tensor *t = tensor(o);
        if (!t || t->dim() != 2 || !t->is_cuda() || !plain(*t, at::kInt, t->get_device()))
            return;
        p = t->mutable_data_ptr<int32_t>();
        rows = (int)t->size(0), width = (int)t->size(1), device = t->get_device();
        ok = true;
    }
};

Pool *pool_of(PyObject *o) { return static_cast<Pool *>(PyLong_AsVoidPtr(o)); }

// A launch goes to the current device where the stream's handle does not name one (0, PyTorch's default stream).  Tensors
// of another device are left to the package, which changes over for the call.
bool current(int device) { return c10::cuda::current_device() == device; }

void *stream_of(int device) { return c10::cuda::getCurrentCUDAStream(device).stream(); }

at::Tensor cuda_empty(at::IntArrayRef size, at::ScalarType type, int device)
{
    return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, device)));
}

// q k v pool rope table seq_len cu_seqlens layer q_norm k_norm eps interleaved out
PyObject *prologue(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 14)
        Py_RETURN_NONE;
    const Pool &pool = *pool_of(a[3]);
    const int dev = pool.device;
    const Tokens q(a[0], pool), k(a[1], pool), v(a[2], pool);
    const Table table(a[5]);
    const at::Tensor *rope = a[4] == Py_None ? nullptr : tensor(a[4]);
    if (!current(dev) || !q.ok || !k.ok || !v.ok || !table.ok || table.device != dev || k.tokens != q.tokens || v.tokens != q.tokens ||
        k.heads != pool.hkv || v.heads != pool.hkv ||
        (a[4] != Py_None && (!rope || rope->dim() != 2 || !plain(*rope, at::kFloat, dev))))
        Py_RETURN_NONE;
    const Arg seq(a[6], table.rows, at::kInt, dev), cu(a[7], table.rows + 1, at::kInt, dev);
    const Arg qn(a[9], pool.d, at::kFloat, dev, kOrNone), kn(a[10], pool.d, at::kFloat, dev, kOrNone);
    const long layer = PyLong_AsLong(a[8]);
    const double eps = PyFloat_AsDouble(a[11]);
    const int interleaved = PyObject_IsTrue(a[12]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const int64_t size[3] = {q.tokens, q.heads, pool.d};
    const Arg given(a[13], q.tokens * q.heads * pool.d, pool.type, dev, kOrNone);
    if (!seq.ok || !cu.ok || !qn.ok || !kn.ok || !given.ok)
        Py_RETURN_NONE;
    at::Tensor made;
    void *out = given.as<void>();
    if (a[13] == Py_None) {
        made = cuda_empty(size, pool.type, dev);
        out = made.mutable_data_ptr();
    }
    const int rc = c_prologue(q.p, q.stride, k.p, k.stride, v.p, v.stride, pool.handle, (int)layer,
                   rope ? rope->const_data_ptr<float>() : nullptr, rope ? (int)rope->size(0) : 0,
                   rope ? (int)rope->size(1) : 0, interleaved, qn.as<float>(), kn.as<float>(), (float)eps, table.p,
                   table.width, seq.as<int32_t>(), cu.as<int32_t>(), out, (int)q.heads, table.rows, (int)q.tokens,
                   pool.code, stream_of(dev));
    if (rc != GDN_OK)
        return PyLong_FromLong(rc);
    if (a[13] == Py_None)
        return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[13]);
    return a[13];
}

// q pool table seq_len cu_seqlens layer scale out workspace
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 9)
        Py_RETURN_NONE;
    const Pool &pool = *pool_of(a[1]);
    const int dev = pool.device;
    const Tokens q(a[0], pool);
    const Table table(a[2]);
    if (!current(dev) || !q.ok || !table.ok || table.device != dev)
        Py_RETURN_NONE;
    const Arg seq(a[3], table.rows, at::kInt, dev), cu(a[4], table.rows + 1, at::kInt, dev);
    const Arg given(a[7], q.tokens * q.heads * pool.d, pool.type, dev, kOrNone);
    const long layer = PyLong_AsLong(a[5]);
    const double scale = PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (!seq.ok || !cu.ok || !given.ok)
        Py_RETURN_NONE;
    const int64_t size[3] = {q.tokens, q.heads, pool.d};
    at::Tensor made, room;
    void *out = given.as<void>(), *work = nullptr;
    size_t bytes = 0;
    if (a[7] == Py_None) {
        made = cuda_empty(size, pool.type, dev);
        out = made.mutable_data_ptr();
    }
    if (a[8] == Py_None) {
        bytes = c_workspace(pool.handle, (int)q.heads, table.rows, (int)q.tokens);
        const int64_t length = (int64_t)bytes;
        room = cuda_empty(at::IntArrayRef(&length, 1), at::kByte, dev);
        work = room.mutable_data_ptr();
    } else {
        const at::Tensor *w = tensor(a[8]);
        if (!w || !plain(*w, w->scalar_type(), dev))
            Py_RETURN_NONE;
        work = w->mutable_data_ptr();
        bytes = w->nbytes();
    }
    const int rc = c_attention(q.p, q.stride, pool.handle, (int)layer, table.p, table.width, seq.as<int32_t>(), cu.as<int32_t>(),
                    (float)scale, out, (int)q.heads, table.rows, (int)q.tokens, work, bytes, pool.code,
                    stream_of(dev));
    if (rc != GDN_OK)
        return PyLong_FromLong(rc);
    if (a[7] == Py_None)
        return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[7]);
    return a[7];
}

// table seq_len refs src_rows dst_rows page_size move_src move_dst move_count status
PyObject *fork_rows(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 10)
        Py_RETURN_NONE;
    const Table table(a[0]);
    const at::Tensor *refs = tensor(a[2]), *src = tensor(a[3]);
    if (!table.ok || !current(table.device) || !refs || !src || !plain(*refs, at::kInt, table.device) || !plain(*src, at::kInt, table.device))
        Py_RETURN_NONE;
    const int dev = table.device;
    const int64_t rows = src->numel();
    const Arg seq(a[1], table.rows, at::kInt, dev), dst(a[4], rows, at::kInt, dev), ms(a[6], rows, at::kInt, dev, kOrMore),
        md(a[7], rows, at::kInt, dev, kOrMore), mc(a[8], 1, at::kInt, dev), st(a[9], rows, at::kInt, dev, kOrMore);
    const long page = PyLong_AsLong(a[5]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (!seq.ok || !dst.ok || !ms.ok || !md.ok || !mc.ok || !st.ok)
        Py_RETURN_NONE;
    return PyLong_FromLong(c_fork(table.p, table.rows, table.width, seq.as<int32_t>(), refs->mutable_data_ptr<int32_t>(),
                                  (int)refs->numel(), (int)page, src->const_data_ptr<int32_t>(), dst.as<int32_t>(),
                                  (int)rows, ms.as<int32_t>(), md.as<int32_t>(), mc.as<int32_t>(), st.as<int32_t>(),
                                  stream_of(dev)));
}

// table seq_len refs rows
PyObject *free_rows(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 4)
        Py_RETURN_NONE;
    const Table table(a[0]);
    const at::Tensor *refs = tensor(a[2]), *rows = tensor(a[3]);
    if (!table.ok || !current(table.device) || !refs || !rows || !plain(*refs, at::kInt, table.device) || !plain(*rows, at::kInt, table.device))
        Py_RETURN_NONE;
    const Arg seq(a[1], table.rows, at::kInt, table.device);
    if (!seq.ok)
        Py_RETURN_NONE;
    return PyLong_FromLong(c_free(table.p, table.rows, table.width, seq.as<int32_t>(), refs->mutable_data_ptr<int32_t>(),
                                  (int)refs->numel(), rows->const_data_ptr<int32_t>(), (int)rows->numel(),
                                  stream_of(table.device)));
}

// pool src dst count
PyObject *copy_pages(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 4)
        Py_RETURN_NONE;
    const Pool &pool = *pool_of(a[0]);
    const at::Tensor *src = tensor(a[1]);
    if (!current(pool.device) || !src || !plain(*src, at::kInt, pool.device))
        Py_RETURN_NONE;
    const Arg dst(a[2], src->numel(), at::kInt, pool.device), count(a[3], 1, at::kInt, pool.device);
    if (!dst.ok || !count.ok)
        Py_RETURN_NONE;
    return PyLong_FromLong(c_copy(pool.handle, src->const_data_ptr<int32_t>(), dst.as<int32_t>(), (int)src->numel(),
                                  count.as<int32_t>(), stream_of(pool.device)));
}

// handle hkv d dtype_code device -> the pool as the calls above take it
PyObject *make_pool(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 5)
        Py_RETURN_NONE;
    Pool *p = new (std::nothrow) Pool;
    if (!p)
        return PyErr_NoMemory();
    p->handle = static_cast<kv_page_pool *>(PyLong_AsVoidPtr(a[0]));
    p->hkv = (int)PyLong_AsLong(a[1]);
    p->d = (int)PyLong_AsLong(a[2]);
    p->code = (int)PyLong_AsLong(a[3]);
    p->device = (int)PyLong_AsLong(a[4]);
    p->type = p->code == GDN_BF16 ? at::kBFloat16 : at::kFloat;
    if (PyErr_Occurred()) {
        delete p;
        return nullptr;
    }
    return PyLong_FromVoidPtr(p);
}

PyObject *drop_pool(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n == 1)
        delete pool_of(a[0]);
    Py_RETURN_NONE;
}

// the addresses of the C ABI's functions, in the order of the variables above
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void **to[] = {reinterpret_cast<void **>(&c_prologue),  reinterpret_cast<void **>(&c_workspace),
                   reinterpret_cast<void **>(&c_attention), reinterpret_cast<void **>(&c_fork),
                   reinterpret_cast<void **>(&c_free),      reinterpret_cast<void **>(&c_copy)};
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "six addresses are needed");
        return nullptr;
    }
    for (int i = 0; i < 6; ++i)
        *to[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred())
        return nullptr;
    Py_RETURN_NONE;
}

// C++ exceptions (an allocation that fails) end at the C entry: the package's own way meets and reports them.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    try {
        return F(self, a, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

#define METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("bind", bind),           METHOD("make_pool", make_pool),
                         METHOD("drop_pool", drop_pool), METHOD("attn_prologue", prologue),
                         METHOD("paged_attention", attention), METHOD("kv_pages_fork", fork_rows),
                         METHOD("kv_pages_free", free_rows),   METHOD("kv_pages_copy", copy_pages),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__fast_binding(void) { return PyModule_Create(&module); }
