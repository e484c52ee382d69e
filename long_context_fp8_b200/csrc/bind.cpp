// Python binding of the speculative-decoding entry points: reads the tensors,
// checks them, and calls the C library.  A step of speculative decoding is a
// run of short kernels (4 to 15 us each), and one call through ctypes with its
// checks in Python costs 14 to 25 us of the host; here it is about 3.
#include <Python.h>

#include <dlfcn.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dsa.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject *g_error = nullptr;           // DSAError

struct Lib {
    decltype(&dsa_rope) rope;
    decltype(&dsa_blocks_extend) blocks_extend;
    decltype(&dsa_blocks_trim) blocks_trim;
    decltype(&dsa_tree_attn_workspace_size) tree_attn_workspace_size;
    decltype(&dsa_tree_attn) tree_attn;
    decltype(&dsa_verify_tree) verify_tree;
    decltype(&dsa_cache_compact) cache_compact;
} g_lib;

// Something the arguments may not be: a ValueError.
struct Bad : std::runtime_error { using std::runtime_error::runtime_error; };
// A Python exception that is set already.
struct Raised {};

int64_t as_int(PyObject *o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

int as_int32(PyObject *o)
{
    const int64_t v = as_int(o);
    if (v != (int)v) throw Bad("an argument does not fit 32 bits");
    return (int)v;
}

double as_double(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

bool as_bool(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

const Tensor &as_tensor(PyObject *o)
{
    if (!THPVariable_Check(o)) throw Bad("DSA entry points take tensors");
    return THPVariable_Unpack(o);
}

// The tensor whose device the call runs on.
const Tensor &reference(PyObject *o)
{
    const Tensor &t = as_tensor(o);
    if (!t.is_cuda()) throw Bad("DSA entry points take CUDA tensors");
    return t;
}

std::string text(at::IntArrayRef s)
{
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

void check(const Tensor &t, ScalarType type, const Tensor &ref)
{
    if (t.scalar_type() != type) throw Bad(std::string("expected ") + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.device() != ref.device()) throw Bad("tensors on " + t.device().str() + " and " + ref.device().str());
    if (!t.is_contiguous()) throw Bad("DSA entry points take contiguous tensors");
}

// Address of a contiguous tensor of that type on ref's device.
void *address(PyObject *o, ScalarType type, const Tensor &ref)
{
    const Tensor &t = as_tensor(o);
    check(t, type, ref);
    return t.data_ptr();
}

// ... and of that shape.
void *address(PyObject *o, ScalarType type, const Tensor &ref, at::IntArrayRef shape)
{
    const Tensor &t = as_tensor(o);
    check(t, type, ref);
    if (t.sizes() != shape) throw Bad("expected shape " + text(shape) + ", got " + text(t.sizes()));
    return t.data_ptr();
}

void *optional(PyObject *o, ScalarType type, const Tensor &ref, at::IntArrayRef shape)
{
    return o == Py_None ? nullptr : address(o, type, ref, shape);
}

uint32_t *status_word(PyObject *o, const Tensor &ref)
{
    return o == Py_None ? nullptr : (uint32_t *)address(o, at::kInt, ref);
}

// The device and stream of a call: a stream object's, or with None the current
// one.  What the call allocates belongs to that stream: memory from another
// stream's pool may still be in use there, and a workspace would go back to that
// pool while the call runs.  Outputs go to the caller, whose current stream is
// told of them.
struct Run {
    c10::cuda::CUDAGuard device;
    c10::cuda::CUDAStream caller;
    c10::cuda::OptionalCUDAStreamGuard other;
    void *stream;

    Run(PyObject *o, const Tensor &ref)
        : device(ref.device()), caller(c10::cuda::getCurrentCUDAStream(ref.get_device())), stream(caller.stream())
    {
        if (o == Py_None) return;
        PyObject *v = PyObject_GetAttrString(o, "cuda_stream");
        if (!v) throw Raised{};
        stream = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (!stream && PyErr_Occurred()) throw Raised{};
        if (stream != caller.stream())
            other.reset_stream(c10::cuda::getStreamFromExternal((cudaStream_t)stream, ref.get_device()));
    }

    Tensor output(at::IntArrayRef sizes, const at::TensorOptions &options) const
    {
        Tensor t = at::empty(sizes, options);
        if (other.current_stream()) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), caller);
        return t;
    }
};

void done(const char *fn, dsa_status st)
{
    if (st == DSA_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "si", fn, (int)st);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }

PyObject *keep(PyObject *given, const Tensor &t)
{
    if (given == Py_None) return wrap(t);
    Py_INCREF(given);
    return given;
}

template <typename F> PyObject *guarded(F &&f)
{
    try {
        return f();
    } catch (const Raised &) {
    } catch (const Bad &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

void arguments(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) throw Bad("wrong number of arguments");
}

// ---------------------------------------------------------------- entry points

// Row stride of [rows, H, d] with dense heads.
int64_t rope_stride(const Tensor &x, const Tensor *like)
{
    if (x.dim() != 3 || (x.size(2) > 1 && x.stride(2) != 1) || (x.size(1) > 1 && x.stride(1) != x.size(2)))
        throw Bad("dsa_rope takes [rows, H, d] with dense heads");
    if (like && (x.sizes() != like->sizes() || x.scalar_type() != like->scalar_type() || x.device() != like->device()))
        throw Bad("dsa_rope's tensors must agree in shape, type and device");
    // a single row's stride says nothing
    return x.size(0) > 1 ? x.stride(0) : x.size(1) * x.size(2);
}

// q, k, positions, turns, rot_dim, rot_begin, interleaved, attn_factor, inverse, q_out, k_out, stream
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        arguments(n, 12);
        const Tensor &q = reference(a[0]);
        const Run run(a[11], q);
        const ScalarType type = q.scalar_type();
        if (type != at::kBFloat16 && type != at::kFloat) throw Bad("dsa_rope takes bf16 or fp32");
        const int64_t qs = rope_stride(q, nullptr);
        const int64_t rows = q.size(0), d = q.size(2);
        const Tensor q_out = a[9] == Py_None ? run.output(q.sizes(), q.options()) : as_tensor(a[9]);
        const int64_t qos = rope_stride(q_out, &q);
        Tensor k_out;
        const void *kp = nullptr;
        void *kop = nullptr;
        int64_t ks = 0, kos = 0, H_k = 0;
        if (a[1] != Py_None) {
            const Tensor &k = as_tensor(a[1]);
            ks = rope_stride(k, nullptr);
            H_k = k.size(1);
            if (k.size(0) != rows || k.size(2) != d || k.scalar_type() != type || k.device() != q.device())
                throw Bad("q and k must agree in rows, head dimension, type and device");
            k_out = a[10] == Py_None ? run.output(k.sizes(), k.options()) : as_tensor(a[10]);
            kos = rope_stride(k_out, &k);
            kp = k.data_ptr();
            kop = k_out.data_ptr();
        }
        if (d > INT32_MAX || q.size(1) > INT32_MAX || H_k > INT32_MAX) throw Bad("dsa_rope: a size is out of range");
        done("dsa_rope", g_lib.rope(q.data_ptr(), qs, (int)q.size(1), kp, ks, (int)H_k,
                                    (const int32_t *)address(a[2], at::kInt, q, {rows}), rows, (int)d, as_int32(a[5]),
                                    as_int32(a[4]), as_bool(a[6]), (const uint64_t *)as_int(a[3]), (float)as_double(a[7]),
                                    as_bool(a[8]), q_out.data_ptr(), qos, kop, kos,
                                    type == at::kBFloat16 ? DSA_BF16 : DSA_F32, run.stream));
        return Py_BuildValue("NN", keep(a[9], q_out), a[1] == Py_None ? Py_NewRef(Py_None) : keep(a[10], k_out));
    });
}

struct Pool {
    const Tensor &table;
    int64_t B, width, capacity;
    int32_t *block_table, *context_lens, *pages_held, *free_pages, *free_count;
    // block_table, context_lens, pages_held, free_pages, free_count
    explicit Pool(PyObject *const *a) : table(reference(a[0]))
    {
        if (table.dim() != 2) throw Bad("expected block_table [B, max_pages]");
        B = table.size(0);
        width = table.size(1);
        if (B > INT32_MAX || width > INT32_MAX) throw Bad("block_table is too large");
        block_table = (int32_t *)address(a[0], at::kInt, table);
        context_lens = (int32_t *)address(a[1], at::kInt, table, {B});
        pages_held = (int32_t *)address(a[2], at::kInt, table, {B});
        free_pages = (int32_t *)address(a[3], at::kInt, table);
        capacity = as_tensor(a[3]).numel();
        free_count = (int32_t *)address(a[4], at::kInt, table, {1});
    }
};

// pool (5), new_lens, page_size, num_pages, max_tokens, token_start, seq_ids, positions, slots, status, stream
PyObject *blocks_extend(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        arguments(n, 15);
        const Pool p(a);
        const Run run(a[14], p.table);
        const int64_t m = as_int(a[8]);
        done("dsa_blocks_extend",
             g_lib.blocks_extend((const int32_t *)address(a[5], at::kInt, p.table, {p.B}), p.context_lens, p.pages_held,
                                 p.block_table, p.free_pages, p.capacity, p.free_count, (int)p.B, (int)p.width,
                                 as_int(a[7]), as_int32(a[6]), m, (int32_t *)address(a[9], at::kInt, p.table, {p.B + 1}),
                                 (int32_t *)address(a[10], at::kInt, p.table, {m}),
                                 (int32_t *)address(a[11], at::kInt, p.table, {m}),
                                 (int64_t *)optional(a[12], at::kLong, p.table, {m}), status_word(a[13], p.table),
                                 run.stream));
        Py_RETURN_NONE;
    });
}

// pool (5), keep_lens, page_size, num_pages, status, stream
PyObject *blocks_trim(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        arguments(n, 10);
        const Pool p(a);
        const Run run(a[9], p.table);
        done("dsa_blocks_trim",
             g_lib.blocks_trim((const int32_t *)address(a[5], at::kInt, p.table, {p.B}), p.context_lens, p.pages_held,
                               p.block_table, p.free_pages, p.capacity, p.free_count, (int)p.B, (int)p.width, as_int(a[7]),
                               as_int32(a[6]), status_word(a[8], p.table), run.stream));
        Py_RETURN_NONE;
    });
}

// q, k_cache, k_scale, v_cache, v_scale, block_table, context_lens, token_start, parents, max_tree, max_context,
// sm_scale (None: 1 / sqrt(d)), out, lse, ws, stream
PyObject *tree_attn(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        arguments(n, 16);
        const Tensor &q = reference(a[0]), &kc = as_tensor(a[1]), &bt = as_tensor(a[5]);
        const Run run(a[15], q);
        if (q.dim() != 3 || bt.dim() != 2 || (kc.dim() != 3 && kc.dim() != 4))
            throw Bad("expected q [N, H_q, d], block_table [B, max_pages] and caches [P, page_size(, H_kv), d]");
        const int64_t N = q.size(0), H = q.size(1), d = q.size(2), B = bt.size(0);
        const int64_t Hkv = kc.dim() == 4 ? kc.size(2) : 1;
        if (kc.sizes().back() != d) throw Bad("expected cache rows of " + std::to_string(d) + " values");
        if (H > INT32_MAX || d > INT32_MAX || B > INT32_MAX || Hkv > INT32_MAX || bt.size(1) > INT32_MAX ||
            kc.size(1) > INT32_MAX)
            throw Bad("dsa_tree_attn: a size is out of range");
        const bool kv8 = a[2] != Py_None;
        const ScalarType code = kv8 ? at::kByte : at::kBFloat16;
        const at::IntArrayRef scales = kc.sizes().slice(0, kc.dim() - 1);
        const Tensor out = a[12] == Py_None ? run.output(q.sizes(), q.options()) : as_tensor(a[12]);
        const Tensor lse = a[13] == Py_None ? run.output({N, H}, q.options().dtype(at::kFloat)) : as_tensor(a[13]);
        Tensor ws = a[14] == Py_None ? Tensor() : as_tensor(a[14]);
        if (!ws.defined())
            ws = at::empty({(int64_t)g_lib.tree_attn_workspace_size((int)B, N, (int)H, (int)Hkv, (int)d) + 256},
                           q.options().dtype(at::kByte));
        check(q, at::kBFloat16, q);
        check(out, at::kBFloat16, q);
        check(lse, at::kFloat, q);
        check(ws, at::kByte, q);
        if (out.sizes() != q.sizes() || lse.dim() != 2 || lse.size(0) != N || lse.size(1) != H)
            throw Bad("expected out " + text(q.sizes()) + " and lse " + text({N, H}));
        const float sm = a[11] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : (float)as_double(a[11]);
        done("dsa_tree_attn",
             g_lib.tree_attn(q.data_ptr(), address(a[1], code, q), (const float *)optional(a[2], at::kFloat, q, scales),
                             address(a[3], code, q, kc.sizes()), (const float *)optional(a[4], at::kFloat, q, scales),
                             (const int32_t *)address(a[5], at::kInt, q),
                             (const int32_t *)address(a[6], at::kInt, q, {B}),
                             (const int32_t *)address(a[7], at::kInt, q, {B + 1}),
                             (const int32_t *)address(a[8], at::kInt, q, {N}), kc.size(0), (int)bt.size(1),
                             (int)kc.size(1), (int)B, N, as_int32(a[9]), as_int(a[10]), (int)H, (int)Hkv, (int)d, sm,
                             out.data_ptr(), (float *)lse.data_ptr(), ws.data_ptr(), (size_t)ws.numel(),
                             run.stream));
        return Py_BuildValue("NN", keep(a[12], out), keep(a[13], lse));
    });
}

// target, draft, tokens, parents, token_start, u_accept, u_sample, max_path, path, accept_len, next_token, status, stream
PyObject *verify_tree(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        arguments(n, 13);
        const Tensor &p = reference(a[0]), &us = as_tensor(a[6]);
        const Run run(a[12], p);
        if (p.dim() != 2 || us.dim() != 1) throw Bad("expected target_probs [N, V] and u_sample [B]");
        const int64_t N = p.size(0), V = p.size(1), B = us.size(0);
        if (B > INT32_MAX) throw Bad("dsa_verify_tree: a size is out of range");
        const auto ints = p.options().dtype(at::kInt);
        const Tensor path = a[8] == Py_None ? run.output({B, a[7] == Py_None ? DSA_MAX_TREE : as_int(a[7])}, ints)
                                            : as_tensor(a[8]);
        if (path.dim() != 2 || path.size(0) != B || path.size(1) > INT32_MAX) throw Bad("expected path [B, max_path]");
        if (a[8] != Py_None && a[7] != Py_None && as_int(a[7]) != path.size(1)) throw Bad("path's width is max_path");
        const Tensor len = a[9] == Py_None ? run.output({B}, ints) : as_tensor(a[9]);
        const Tensor next = a[10] == Py_None ? run.output({B}, ints) : as_tensor(a[10]);
        for (const Tensor *t : {&path, &len, &next}) check(*t, at::kInt, p);
        if (len.numel() != B || next.numel() != B) throw Bad("expected accept_len and next_token [B]");
        done("dsa_verify_tree",
             g_lib.verify_tree((const float *)address(a[0], at::kFloat, p),
                               (const float *)optional(a[1], at::kFloat, p, p.sizes()),
                               (const int32_t *)address(a[2], at::kInt, p, {N}),
                               (const int32_t *)address(a[3], at::kInt, p, {N}),
                               (const int32_t *)address(a[4], at::kInt, p, {B + 1}),
                               (const float *)address(a[5], at::kFloat, p, {N}),
                               (const float *)address(a[6], at::kFloat, p), (int)B, N, V, (int)path.size(1),
                               (int32_t *)path.data_ptr(), (int32_t *)len.data_ptr(), (int32_t *)next.data_ptr(),
                               status_word(a[11], p), run.stream));
        return Py_BuildValue("NNN", keep(a[8], path), keep(a[9], len), keep(a[10], next));
    });
}

// kidx, kscale, k, k_scale, v, v_scale, block_table, context_lens, token_start, path, accept_len, N (None: any),
// keep_lens, status, stream
PyObject *cache_compact(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        arguments(n, 15);
        const Tensor &bt = reference(a[6]), &kc = as_tensor(a[2]), &path = as_tensor(a[9]);
        const Run run(a[14], bt);
        if (bt.dim() != 2 || (kc.dim() != 3 && kc.dim() != 4) || path.dim() != 2)
            throw Bad("expected block_table [B, max_pages], caches [P, page_size(, H_kv), d] and path [B, max_path]");
        // the K/V heads of a position are one row to the library, which knows one scale a row
        const int64_t heads = kc.dim() == 4 ? kc.size(2) : 1;
        if (a[3] != Py_None && heads != 1) throw Bad("dsa_cache_compact takes FP8 caches of one K/V head");
        const at::IntArrayRef scales = kc.sizes().slice(0, kc.dim() - 1);
        const int64_t B = bt.size(0), P = kc.size(0), ps = kc.size(1), d = heads * kc.sizes().back(), m = path.size(1);
        int64_t d_I = 0;
        if (a[0] != Py_None) {
            const Tensor &ki = as_tensor(a[0]);
            if (ki.dim() != 3) throw Bad("expected kidx_cache [P, page_size, d_I]");
            d_I = ki.size(2);
        }
        if (B > INT32_MAX || bt.size(1) > INT32_MAX || ps > INT32_MAX || d > INT32_MAX || m > INT32_MAX || d_I > INT32_MAX)
            throw Bad("dsa_cache_compact: a size is out of range");
        const ScalarType code = a[3] == Py_None ? at::kBFloat16 : at::kByte;
        const Tensor lens = a[12] == Py_None ? run.output({B}, bt.options()) : as_tensor(a[12]);
        check(lens, at::kInt, bt);
        if (lens.numel() != B) throw Bad("expected keep_lens [B]");
        done("dsa_cache_compact",
             g_lib.cache_compact((const int32_t *)address(a[6], at::kInt, bt),
                                 (const int32_t *)address(a[7], at::kInt, bt, {B}),
                                 (const int32_t *)address(a[8], at::kInt, bt, {B + 1}),
                                 (const int32_t *)address(a[9], at::kInt, bt, {B, m}),
                                 (const int32_t *)address(a[10], at::kInt, bt, {B}), (int)B,
                                 a[11] == Py_None ? INT32_MAX : as_int(a[11]), (int)m, (int)bt.size(1), P, (int)ps,
                                 (int)d_I, (int)d, optional(a[0], at::kByte, bt, {P, ps, d_I}),
                                 (float *)optional(a[1], at::kFloat, bt, {P, ps}), address(a[2], code, bt),
                                 (float *)optional(a[3], at::kFloat, bt, scales), address(a[4], code, bt, kc.sizes()),
                                 (float *)optional(a[5], at::kFloat, bt, scales), (int32_t *)lens.data_ptr(),
                                 status_word(a[13], bt), run.stream));
        return keep(a[12], lens);
    });
}

// library path, DSAError
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        arguments(n, 2);
        const char *path = PyUnicode_AsUTF8(a[0]);
        if (!path) throw Raised{};
        void *h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
        if (!h) throw std::runtime_error(dlerror());
        auto find = [&](auto &f, const char *name) {
            f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
            if (!f) throw std::runtime_error(std::string("no symbol ") + name + " in " + path);
        };
        find(g_lib.rope, "dsa_rope");
        find(g_lib.blocks_extend, "dsa_blocks_extend");
        find(g_lib.blocks_trim, "dsa_blocks_trim");
        find(g_lib.tree_attn_workspace_size, "dsa_tree_attn_workspace_size");
        find(g_lib.tree_attn, "dsa_tree_attn");
        find(g_lib.verify_tree, "dsa_verify_tree");
        find(g_lib.cache_compact, "dsa_cache_compact");
        Py_INCREF(a[1]);
        Py_XDECREF(g_error);
        g_error = a[1];
        Py_RETURN_NONE;
    });
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(init), METHOD(rope), METHOD(blocks_extend), METHOD(blocks_trim), METHOD(tree_attn),
                         METHOD(verify_tree), METHOD(cache_compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module_def); }
