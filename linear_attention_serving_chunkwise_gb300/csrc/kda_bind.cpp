// The Python binding's checks and marshalling for the calls of the attention layers' prompt path and of the cache's upkeep
// (include/kda.h; the functions of _lib.py that carry their names call these).  The calls take a few microseconds on the
// GPU: one for 64 tokens' norms and rotations cost the host 18 us with its checks in Python, of which the launch was 5.
//
// Each function takes the Python call's arguments in order, tensors or None, and `stream`: None for the current one of
// the tensors' GPU, or a raw handle that belongs to that GPU.  The C calls know pointers only: a wrong type, shape, layout or device is found
// here, before anything is launched.  A function returns the C call's status and the tensors that it made.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <limits>

#include "../../include/kda.h"

namespace {

using at::Tensor;
using Shape = at::IntArrayRef;

std::string type_name(at::ScalarType t)
{
    switch (t) {
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    default: return std::string("torch.") + c10::toString(t);
    }
}

const Tensor& tensor(PyObject* o, const char* name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// an integer of the C calls' 32 bits
int32_t number(PyObject* o, const char* name)
{
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &over);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(!over && x >= std::numeric_limits<int32_t>::min() && x <= std::numeric_limits<int32_t>::max(), name, " is out of range");
    return (int32_t)x;
}

int32_t small(int64_t n, const char* name)
{
    TORCH_CHECK_VALUE(n <= std::numeric_limits<int32_t>::max(), name, " has too many elements");
    return (int32_t)n;
}

double real(PyObject* o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

int32_t code_of(const Tensor& t, const char* name)
{
    if (t.scalar_type() == at::kBFloat16) return KDA_BF16;
    TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, name, " must be float32 or bfloat16, got ", type_name(t.scalar_type()));
    return KDA_F32;
}

// type, shape and device; the layout is the caller's to look at
void look(const Tensor& t, const char* name, at::ScalarType type, Shape shape, int64_t device)
{
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type_name(type), ", got ", type_name(t.scalar_type()));
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
    TORCH_CHECK_VALUE(t.get_device() == device, name, " is on ", t.device(), ", not on the device of the other tensors");
}

void* address(PyObject* o, const char* name, at::ScalarType type, Shape shape, int64_t device)
{
    const Tensor& t = tensor(o, name);
    look(t, name, type, shape, device);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    return t.data_ptr();
}

// Whether what follows the first `lead` dimensions lies without gaps.
bool packed(const Tensor& t, int64_t lead)
{
    int64_t want = 1;
    for (int64_t i = t.dim() - 1; i >= lead; --i) {
        if (t.size(i) != 1 && t.stride(i) != want) return t.numel() == 0;
        want *= t.size(i);
    }
    return true;
}

// a cache [pages, page_size, heads, dim] whose pages are contiguous each: its address, and the elements from page to page
void* cache(PyObject* o, const char* name, at::ScalarType type, Shape shape, int64_t device, int64_t& stride)
{
    const Tensor& t = tensor(o, name);
    look(t, name, type, shape, device);
    TORCH_CHECK_VALUE(packed(t, 1), name, ": each page must be contiguous");
    stride = shape[0] > 1 ? t.stride(0) : shape[1] * shape[2] * shape[3];
    return t.data_ptr();
}

// tokens [T, heads, dim] whose heads are contiguous each: the address, and the elements from token to token
void* tokens(PyObject* o, const char* name, at::ScalarType type, Shape shape, int64_t device, int64_t& stride)
{
    const Tensor& t = tensor(o, name);
    look(t, name, type, shape, device);
    TORCH_CHECK_VALUE(packed(t, 1), name, ": the heads of a token must be contiguous");
    stride = shape[0] > 1 ? t.stride(0) : shape[1] * shape[2];
    return t.data_ptr();
}

// The queue for tensors on `device`, which has to be the GPU that the library will use: the current one.
void* queue_on(PyObject* stream, int64_t device)
{
    TORCH_CHECK_VALUE(device >= 0, "the tensors must be on a CUDA device");
    const int current = c10::cuda::current_device();
    TORCH_CHECK_VALUE(device == current, "the tensors are on cuda:", device, ", the current device is cuda:", current);
    if (stream == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    void* const handle = PyLong_AsVoidPtr(stream);
    if (!handle && PyErr_Occurred()) throw python_error();
    return handle;
}

Tensor fresh(Shape shape, at::ScalarType type, const Tensor& beside)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(beside.device()));
}

template <typename F>
kda_status without_gil(F call)
{
    kda_status st;
    Py_BEGIN_ALLOW_THREADS
    st = call();
    Py_END_ALLOW_THREADS
    return st;
}

template <typename... T>
PyObject* answer(kda_status st, const T&... made)
{
    PyObject* const t = PyTuple_New(1 + sizeof...(T));
    if (!t) throw python_error();
    PyTuple_SET_ITEM(t, 0, PyLong_FromLong(st));
    Py_ssize_t i = 1;
    ((PyTuple_SET_ITEM(t, i, THPVariable_Wrap(made)), ++i), ...);
    return t;
}

void arity(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, want, " arguments expected, got ", n); }

// q, k_cache, v_cache, block_table, context_lens, cu_seqlens, out, scale, workspace, stream -> status, out, workspace
PyObject* chunk_attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 10);
    const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &table = tensor(a[3], "block_table");
    const int32_t code = code_of(q, "q");
    TORCH_CHECK_VALUE(q.dim() == 3 && kc.dim() == 4 && table.dim() == 2, "q must have 3 dimensions, the caches 4 and block_table 2");
    const auto type = q.scalar_type();
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), P = kc.size(0), ps = kc.size(1), Hk = kc.size(2), B = table.size(0), cols = table.size(1);
    const int64_t at = q.get_device();
    int64_t ks, vs;
    void* const qp = address(a[0], "q", type, {T, H, D}, at);
    void* const kp = cache(a[1], "k_cache", type, {P, ps, Hk, D}, at, ks);
    void* const vp = cache(a[2], "v_cache", type, {P, ps, Hk, D}, at, vs);
    const auto tp = (const int32_t*)address(a[3], "block_table", at::kInt, {B, cols}, at);
    const auto cp = (const int32_t*)address(a[4], "context_lens", at::kInt, {B}, at);
    const auto up = (const int32_t*)address(a[5], "cu_seqlens", at::kInt, {B + 1}, at);
    const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)real(a[7]);
    const kda_chunk_attention_desc d = {small(B, "block_table"), small(T, "q"), small(H, "q"), small(Hk, "k_cache"), small(D, "q"), code,
                                        small(P, "k_cache"), small(ps, "k_cache"), small(cols, "block_table"), scale, ks, vs};
    Tensor out, ws;
    void* wp;
    size_t bytes = kda_chunk_attention_workspace_bytes(&d);
    if (a[8] != Py_None) {
        ws = tensor(a[8], "workspace");
        TORCH_CHECK_VALUE(ws.get_device() == at && ws.is_contiguous(), "workspace must be contiguous and on the device of the other tensors");
        bytes = ws.nbytes();
    }
    if (a[6] != Py_None) {
        address(a[6], "out", type, {T, H, D}, at);
        out = tensor(a[6], "out");
    }
    void* const queue = queue_on(a[9], at);
    if (!out.defined()) out = fresh({T, H, D}, type, q);
    if (!ws.defined()) ws = fresh({(int64_t)bytes}, at::kByte, q);
    wp = ws.data_ptr();
    void* const op = out.data_ptr();
    const kda_status st = without_gil([&] { return kda_chunk_attention(&d, qp, kp, vp, tp, cp, up, op, wp, bytes, queue); });
    return answer(st, out, ws);
    END_HANDLE_TH_ERRORS
}

// q, k, v, positions, inv_freq, slots, k_cache, v_cache, out, q_weight, k_weight, eps, flags, stream -> status, out
PyObject* norm_rotate(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 14);
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &freq = tensor(a[4], "inv_freq"), &kc = tensor(a[6], "k_cache");
    const int32_t code = code_of(q, "q");
    TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 3 && kc.dim() == 4, "q, k and v must have 3 dimensions, the caches 4");
    const auto type = q.scalar_type();
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), Hk = k.size(1), P = kc.size(0), ps = kc.size(1), half = freq.numel(), at = q.get_device();
    int64_t qs, ks, vs, kps, vps;
    void* const qp = tokens(a[0], "q", type, {T, H, D}, at, qs);
    void* const kp = tokens(a[1], "k", type, {T, Hk, D}, at, ks);
    void* const vp = tokens(a[2], "v", type, {T, Hk, D}, at, vs);
    void* const kcp = cache(a[6], "k_cache", type, {P, ps, Hk, D}, at, kps);
    void* const vcp = cache(a[7], "v_cache", type, {P, ps, Hk, D}, at, vps);
    const auto pos = (const int32_t*)address(a[3], "positions", at::kInt, {T}, at);
    const auto fp = (const float*)address(a[4], "inv_freq", at::kFloat, {half}, at);
    const auto slot = (const int64_t*)address(a[5], "slots", at::kLong, {T}, at);
    const auto wq = a[9] == Py_None ? nullptr : (const float*)address(a[9], "q_weight", at::kFloat, {D}, at);
    const auto wk = a[10] == Py_None ? nullptr : (const float*)address(a[10], "k_weight", at::kFloat, {D}, at);
    const kda_norm_rotate_desc d = {small(T, "q"), small(H, "q"), small(Hk, "k"), small(D, "q"), code, small(2 * half, "inv_freq"), number(a[12], "flags"),
                                    small(P, "k_cache"), small(ps, "k_cache"), (float)real(a[11]), qs, ks, vs, kps, vps};
    Tensor out;
    if (a[8] != Py_None) {
        address(a[8], "out", type, {T, H, D}, at);
        out = tensor(a[8], "out");
    }
    void* const queue = queue_on(a[13], at);
    if (!out.defined()) out = fresh({T, H, D}, type, q);
    void* const op = out.data_ptr();
    const kda_status st = without_gil([&] { return kda_norm_rotate(&d, qp, kp, vp, wq, wk, fp, pos, slot, op, kcp, vcp, queue); });
    return answer(st, out);
    END_HANDLE_TH_ERRORS
}

// parents, children, lens, pages_held, block_table, shares, free_pages, page_size, stream -> status, pages_held, copies, pages_taken
PyObject* page_fork(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 9);
    const Tensor& table = tensor(a[4], "block_table");
    TORCH_CHECK_VALUE(table.dim() == 2, "block_table must have 2 dimensions");
    const int64_t R = table.size(0), cols = table.size(1), at = table.get_device();
    const int64_t N = tensor(a[0], "parents").numel(), F = tensor(a[6], "free_pages").numel(), P = tensor(a[5], "shares").numel();
    const auto par = (const int32_t*)address(a[0], "parents", at::kInt, {N}, at);
    const auto chi = (const int32_t*)address(a[1], "children", at::kInt, {N}, at);
    const auto len = (const int32_t*)address(a[2], "lens", at::kInt, {N}, at);
    const auto had = (const int32_t*)address(a[3], "pages_held", at::kInt, {R}, at);
    const auto tp = (int32_t*)address(a[4], "block_table", at::kInt, {R, cols}, at);
    const auto sp = (int32_t*)address(a[5], "shares", at::kInt, {P}, at);
    const auto fp = (const int32_t*)address(a[6], "free_pages", at::kInt, {F}, at);
    const int32_t page = number(a[7], "page_size"), forks = small(N, "parents"), rows = small(R, "block_table"), width = small(cols, "block_table"),
                  pages = small(P, "shares"), frees = small(F, "free_pages");
    void* const queue = queue_on(a[8], at);
    Tensor held = fresh({R}, at::kInt, table), copies = fresh({N, 3}, at::kInt, table), taken = fresh({1}, at::kInt, table);
    const auto hp = (int32_t*)held.data_ptr(), cp = (int32_t*)copies.data_ptr(), kp = (int32_t*)taken.data_ptr();
    const kda_status st = without_gil([&] { return kda_page_fork(forks, rows, width, pages, frees, page, par, chi, len, had, tp, sp, fp, hp, cp, kp, queue); });
    return answer(st, held, copies, taken);
    END_HANDLE_TH_ERRORS
}

// keep_lens, pages_held, block_table, shares, page_size, stream -> status, pages_held, freed, num_freed
PyObject* page_release(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 6);
    const Tensor& table = tensor(a[2], "block_table");
    TORCH_CHECK_VALUE(table.dim() == 2, "block_table must have 2 dimensions");
    const int64_t R = table.size(0), cols = table.size(1), at = table.get_device(), P = tensor(a[3], "shares").numel();
    const auto keep = (const int32_t*)address(a[0], "keep_lens", at::kInt, {R}, at);
    const auto had = (const int32_t*)address(a[1], "pages_held", at::kInt, {R}, at);
    const auto tp = (const int32_t*)address(a[2], "block_table", at::kInt, {R, cols}, at);
    const auto sp = (int32_t*)address(a[3], "shares", at::kInt, {P}, at);
    const int32_t page = number(a[4], "page_size"), rows = small(R, "block_table"), width = small(cols, "block_table"), pages = small(P, "shares");
    void* const queue = queue_on(a[5], at);
    Tensor held = fresh({R}, at::kInt, table), freed = fresh({P}, at::kInt, table), count = fresh({1}, at::kInt, table);
    const auto hp = (int32_t*)held.data_ptr(), fp = (int32_t*)freed.data_ptr(), np = (int32_t*)count.data_ptr();
    const kda_status st = without_gil([&] { return kda_page_release(rows, width, pages, page, keep, had, tp, sp, hp, fp, np, queue); });
    return answer(st, held, freed, count);
    END_HANDLE_TH_ERRORS
}

// The caches of all layers, [layers, pages, page_size, heads, dim], or of one, without the first.
struct Layers {
    kda_cache_desc d;
    void *k, *v;
};

Layers layers(PyObject* ko, PyObject* vo, int64_t device)
{
    const Tensor& k = tensor(ko, "k_cache");
    const int32_t code = code_of(k, "k_cache");
    const int64_t dims = k.dim(), first = dims - 4;
    TORCH_CHECK_VALUE(dims == 4 || dims == 5, "k_cache must be [pages, page_size, heads, dim], or that for each layer");
    Layers c = {};
    int64_t layer[2], page[2];
    for (int i = 0; i < 2; ++i) {
        const char* const name = i ? "v_cache" : "k_cache";
        const Tensor& t = tensor(i ? vo : ko, name);
        look(t, name, k.scalar_type(), k.sizes(), device);
        TORCH_CHECK_VALUE(packed(t, first + 1), name, ": each page must be contiguous");
        layer[i] = dims == 5 ? t.stride(0) : 0;
        page[i] = t.stride(first);
        (i ? c.v : c.k) = t.data_ptr();
    }
    c.d = {dims == 5 ? small(k.size(0), "k_cache") : 1, small(k.size(first), "k_cache"), small(k.size(first + 1), "k_cache"), small(k.size(first + 2), "k_cache"),
           small(k.size(first + 3), "k_cache"), code, layer[0], layer[1], page[0], page[1]};
    return c;
}

// copies, k_cache, v_cache, stream -> status
PyObject* cache_copy(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 4);
    const Tensor& list = tensor(a[0], "copies");
    TORCH_CHECK_VALUE(list.dim() == 2, "copies must have 2 dimensions");
    const int64_t at = list.get_device();
    const auto lp = (const int32_t*)address(a[0], "copies", at::kInt, {list.size(0), 3}, at);
    const Layers c = layers(a[1], a[2], at);
    const int32_t count = small(list.size(0), "copies");
    void* const queue = queue_on(a[3], at);
    return answer(without_gil([&] { return kda_cache_copy(&c.d, count, lp, c.k, c.v, queue); }));
    END_HANDLE_TH_ERRORS
}

// slots, path, n_accept, k_cache, v_cache, stream -> status
PyObject* cache_keep_path(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 6);
    const Tensor& slots = tensor(a[0], "slots");
    TORCH_CHECK_VALUE(slots.dim() == 2, "slots must have 2 dimensions");
    const int64_t B = slots.size(0), K = slots.size(1), at = slots.get_device();
    const auto sp = (const int64_t*)address(a[0], "slots", at::kLong, {B, K}, at);
    const auto pp = (const int32_t*)address(a[1], "path", at::kInt, {B, K}, at);
    const auto np = (const int32_t*)address(a[2], "n_accept", at::kInt, {B}, at);
    const Layers c = layers(a[3], a[4], at);
    const int32_t batch = small(B, "slots"), nodes = small(K, "slots");
    void* const queue = queue_on(a[5], at);
    return answer(without_gil([&] { return kda_cache_keep_path(&c.d, batch, nodes, sp, pp, np, c.k, c.v, queue); }));
    END_HANDLE_TH_ERRORS
}

#define KDA_BOUND(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_BOUND(chunk_attention), KDA_BOUND(norm_rotate), KDA_BOUND(page_fork), KDA_BOUND(page_release),
                         KDA_BOUND(cache_copy),      KDA_BOUND(cache_keep_path), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
