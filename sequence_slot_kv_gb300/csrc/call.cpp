// call.cpp -- the Python module _slotkv_call: the scored, shared, tree and
// request-length calls and those on pages of include/slotkv.h made straight
// from torch tensors.
//
// A small step's kernels take a few microseconds, and checking a dozen tensors
// and marshalling them attribute by attribute in Python takes as long (3.5 us
// of a 6.8 us slot_kv_token_map).  Each function here takes the call's
// arguments in the order of the C declaration, checks every tensor (type,
// current device, contiguous, shape) and makes the call: an int status, or
// None when some argument is not as the fast path wants it, without having
// done anything -- the Python binding then looks again and says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/slotkv.h"

namespace {

constexpr auto F32 = at::ScalarType::Float;
constexpr auto I32 = at::ScalarType::Int;

struct Unlike {};  // an argument the fast path does not take

const at::Tensor& tensor(PyObject* o, at::ScalarType type, int dev) {
    if (!THPVariable_Check(o)) throw Unlike{};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
        throw Unlike{};
    return t;
}

template <typename T>
T* address(PyObject* o, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
    const at::Tensor& t = tensor(o, type, dev);
    if (t.sizes() != at::IntArrayRef(shape)) throw Unlike{};
    return static_cast<T*>(t.data_ptr());
}

const float* floats(PyObject* o, int dev, std::initializer_list<int64_t> shape) {
    return address<const float>(o, F32, dev, shape);
}
uint32_t* ints(PyObject* o, int dev, std::initializer_list<int64_t> shape) {
    return address<uint32_t>(o, I32, dev, shape);
}
const float* floats_or_null(PyObject* o, int dev, std::initializer_list<int64_t> shape) {
    return o == Py_None ? nullptr : floats(o, dev, shape);
}
const uint32_t* ints_or_null(PyObject* o, int dev, std::initializer_list<int64_t> shape) {
    return o == Py_None ? nullptr : ints(o, dev, shape);
}

void* pointer(PyObject* o) {  // an int, or None for NULL
    if (o == Py_None) return nullptr;
    if (!PyLong_Check(o)) throw Unlike{};
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unlike{};
    }
    return p;
}

double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unlike{};
    }
    return x;
}

int64_t integer(PyObject* o) {
    if (!PyLong_Check(o)) throw Unlike{};
    const int64_t x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unlike{};
    }
    return x;
}

slotkv_stream_t stream_of(PyObject* o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    return pointer(o);
}

// (cap, window, slopes, doc_start, prefix_end) or None; rows: what doc_start and
// prefix_end have an entry for
const slotkv_scores* scores_of(PyObject* o, slotkv_scores& s, int dev, int64_t rows,
                               int64_t n_head) {
    if (o == Py_None) return nullptr;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) throw Unlike{};
    s.cap = static_cast<float>(number(PyTuple_GET_ITEM(o, 0)));
    s.window = static_cast<uint32_t>(integer(PyTuple_GET_ITEM(o, 1)));
    s.slopes = floats_or_null(PyTuple_GET_ITEM(o, 2), dev, {n_head});
    s.doc_start = ints_or_null(PyTuple_GET_ITEM(o, 3), dev, {rows});
    s.prefix_end = ints_or_null(PyTuple_GET_ITEM(o, 4), dev, {rows});
    return &s;
}

// What every step takes; a[0..] = handle, n_kv_head, head_dim, q, k_new,
// v_new, positions.
struct Step {
    slotkv_t h;
    int64_t B, n_head, hd;
    uint32_t b, nh;
    const float *q, *k_new, *v_new;
    const uint32_t* positions;
    int dev;
    explicit Step(PyObject* const* a) {
        dev = static_cast<int>(c10::cuda::current_device());
        h = static_cast<slotkv_t>(pointer(a[0]));
        const int64_t n_kv = integer(a[1]);
        const at::Tensor& tq = tensor(a[3], F32, dev);
        if (tq.dim() != 3) throw Unlike{};
        B = tq.size(0);
        n_head = tq.size(1);
        hd = tq.size(2);
        if (hd != integer(a[2]) || B > UINT32_MAX || n_head > UINT32_MAX) throw Unlike{};
        b = static_cast<uint32_t>(B);
        nh = static_cast<uint32_t>(n_head);
        q = static_cast<const float*>(tq.data_ptr());
        k_new = floats(a[4], dev, {B, n_kv, hd});
        v_new = floats(a[5], dev, {B, n_kv, hd});
        positions = ints(a[6], dev, {B});
    }
};

// And the rest; a[0..] = q_norm_w, k_norm_w, inv_freq, sinks, scores, out,
// eps, scale, stream.
struct Rest {
    const float *qw, *kw, *inv, *sinks;
    slotkv_scores store;
    const slotkv_scores* scores;
    float* out;
    float eps, scale;
    slotkv_stream_t stream;
    Rest(PyObject* const* a, const Step& s) : Rest(a, s, s.B) {}
    template <typename S>
    Rest(PyObject* const* a, const S& s, int64_t rule_rows) {
        qw = floats(a[0], s.dev, {s.hd});
        kw = floats(a[1], s.dev, {s.hd});
        inv = floats(a[2], s.dev, {s.hd / 2});
        sinks = floats_or_null(a[3], s.dev, {s.n_head});
        scores = scores_of(a[4], store, s.dev, rule_rows, s.n_head);
        out = address<float>(a[5], F32, s.dev, {s.B, s.n_head, s.hd});
        eps = static_cast<float>(number(a[6]));
        scale = static_cast<float>(number(a[7]));
        stream = stream_of(a[8], s.dev);
    }
};

// Runs body (which returns a status) and turns its outcome into Python's.
template <typename Body>
PyObject* run(Py_ssize_t n, Py_ssize_t want, Body body) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(body());
    } catch (const Unlike&) {
        Py_RETURN_NONE;
    } catch (const std::exception&) {  // (torch's own, say without a device)
        Py_RETURN_NONE;
    }
}

template <typename Call>
int without_gil(Call call) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return rc;
}

PyObject* slot_step(PyObject* const* a, Py_ssize_t n, decltype(&decode_batch_attn_scored) fn) {
    return run(n, 17, [&] {
        const Step s(a);
        const uint32_t* slots = ints(a[7], s.dev, {s.B});
        const Rest r(a + 8, s);
        return without_gil([&] {
            return fn(s.h, s.b, s.nh, s.q, s.k_new, s.v_new, s.positions, slots, r.qw, r.kw, r.inv,
                      r.sinks, r.scores, r.out, r.eps, r.scale, r.stream);
        });
    });
}

PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return slot_step(a, n, decode_batch_attn_scored);
}
PyObject* py_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return slot_step(a, n, prefill_batch_attn_scored);
}

PyObject* py_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return run(n, 17, [&] {
        const Step s(a);
        const at::Tensor& tab = tensor(a[7], I32, s.dev);
        if (tab.dim() != 2 || tab.size(0) != s.B || tab.size(1) > UINT32_MAX) throw Unlike{};
        const Rest r(a + 8, s);
        return without_gil([&] {
            return decode_batch_attn_paged_scored(
                s.h, s.b, s.nh, s.q, s.k_new, s.v_new, s.positions,
                static_cast<const uint32_t*>(tab.data_ptr()), static_cast<uint32_t>(tab.size(1)),
                r.qw, r.kw, r.inv, r.sinks, r.scores, r.out, r.eps, r.scale, r.stream);
        });
    });
}

PyObject* py_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return run(n, 20, [&] {
        const Step s(a);
        const uint32_t* slots = ints(a[7], s.dev, {s.B});
        slotkv_t prefix = static_cast<slotkv_t>(pointer(a[8]));
        const uint32_t* pslots = ints(a[9], s.dev, {s.B});
        const uint32_t* plens = ints(a[10], s.dev, {s.B});
        const Rest r(a + 11, s);
        return without_gil([&] {
            return decode_batch_attn_shared(s.h, s.b, s.nh, s.q, s.k_new, s.v_new, s.positions,
                                            slots, prefix, pslots, plens, r.qw, r.kw, r.inv,
                                            r.sinks, r.scores, r.out, r.eps, r.scale, r.stream);
        });
    });
}

PyObject* py_token_map(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return run(n, 8, [&] {
        const int dev = static_cast<int>(c10::cuda::current_device());
        slotkv_t h = static_cast<slotkv_t>(pointer(a[0]));
        const at::Tensor& slots = tensor(a[1], I32, dev);
        const at::Tensor& ts = tensor(a[5], I32, dev);
        const int64_t R = slots.numel(), T = ts.numel();
        if (slots.dim() != 1 || ts.dim() != 1 || R >= UINT32_MAX || T > UINT32_MAX) throw Unlike{};
        const uint32_t* past = ints(a[2], dev, {R});
        const uint32_t* fresh = ints(a[3], dev, {R});
        uint32_t* starts = ints(a[4], dev, {R + 1});
        uint32_t* tp = ints(a[6], dev, {T});
        slotkv_stream_t stream = stream_of(a[7], dev);
        return without_gil([&] {
            return slot_kv_token_map(h, static_cast<uint32_t>(R),
                                     static_cast<const uint32_t*>(slots.data_ptr()), past, fresh,
                                     static_cast<uint32_t>(T), starts,
                                     static_cast<uint32_t*>(ts.data_ptr()), tp, stream);
        });
    });
}

PyObject* py_extend_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return run(n, 8, [&] {
        const int dev = static_cast<int>(c10::cuda::current_device());
        slotkv_t h = static_cast<slotkv_t>(pointer(a[0]));
        const at::Tensor& past = tensor(a[1], I32, dev);
        const at::Tensor& tab = tensor(a[3], I32, dev);
        const at::Tensor& free_ids = tensor(a[4], I32, dev);
        const int64_t R = past.numel();
        if (past.dim() != 1 || tab.dim() != 2 || tab.size(0) != R || free_ids.dim() != 1 ||
            R > UINT32_MAX || tab.size(1) > UINT32_MAX || free_ids.size(0) > UINT32_MAX)
            throw Unlike{};
        const uint32_t* fresh = ints(a[2], dev, {R});
        const uint32_t* head = ints(a[5], dev, {1});
        uint32_t* head_out = ints(a[6], dev, {1});
        slotkv_stream_t stream = stream_of(a[7], dev);
        return without_gil([&] {
            return slot_kv_extend_tables(
                h, static_cast<uint32_t>(R), static_cast<const uint32_t*>(past.data_ptr()), fresh,
                static_cast<uint32_t*>(tab.data_ptr()), static_cast<uint32_t>(tab.size(1)),
                static_cast<const uint32_t*>(free_ids.data_ptr()),
                static_cast<uint32_t>(free_ids.size(0)), head, head_out, stream);
        });
    });
}

// A tree call's; a[0..] = handle, n_kv_head, head_dim, q, k_new, v_new, slots or
// block tables, past, starts, parents.
struct TreeStep {
    slotkv_t h;
    int64_t B, n_head, hd, R, stride = 0;
    const float *q, *k_new, *v_new;
    const uint32_t *idx, *past, *starts, *parents;
    int dev;
    TreeStep(PyObject* const* a, bool paged) {
        dev = static_cast<int>(c10::cuda::current_device());
        h = static_cast<slotkv_t>(pointer(a[0]));
        const int64_t n_kv = integer(a[1]);
        const at::Tensor& tq = tensor(a[3], F32, dev);
        if (tq.dim() != 3) throw Unlike{};
        B = tq.size(0);
        n_head = tq.size(1);
        hd = tq.size(2);
        if (hd != integer(a[2]) || B > UINT32_MAX || n_head > UINT32_MAX) throw Unlike{};
        q = static_cast<const float*>(tq.data_ptr());
        k_new = floats(a[4], dev, {B, n_kv, hd});
        v_new = floats(a[5], dev, {B, n_kv, hd});
        const at::Tensor& tp = tensor(a[7], I32, dev);
        if (tp.dim() != 1 || tp.size(0) >= UINT32_MAX) throw Unlike{};
        R = tp.size(0);
        past = static_cast<const uint32_t*>(tp.data_ptr());
        if (paged) {
            const at::Tensor& tab = tensor(a[6], I32, dev);
            if (tab.dim() != 2 || tab.size(0) != R || tab.size(1) > UINT32_MAX) throw Unlike{};
            stride = tab.size(1);
            idx = static_cast<const uint32_t*>(tab.data_ptr());
        } else {
            idx = ints(a[6], dev, {R});
        }
        starts = ints(a[8], dev, {R + 1});
        parents = ints(a[9], dev, {B});
    }
};

PyObject* py_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return run(n, 19, [&] {
        const TreeStep s(a, false);
        const Rest r(a + 10, s, s.R);
        return without_gil([&] {
            return tree_batch_attn(s.h, static_cast<uint32_t>(s.R), static_cast<uint32_t>(s.B),
                                   static_cast<uint32_t>(s.n_head), s.q, s.k_new, s.v_new, s.idx,
                                   s.past, s.starts, s.parents, r.qw, r.kw, r.inv, r.sinks,
                                   r.scores, r.out, r.eps, r.scale, r.stream);
        });
    });
}

PyObject* py_tree_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return run(n, 19, [&] {
        const TreeStep s(a, true);
        const Rest r(a + 10, s, s.R);
        return without_gil([&] {
            return tree_batch_attn_paged(
                s.h, static_cast<uint32_t>(s.R), static_cast<uint32_t>(s.B),
                static_cast<uint32_t>(s.n_head), s.q, s.k_new, s.v_new, s.idx,
                static_cast<uint32_t>(s.stride), s.past, s.starts, s.parents, r.qw, r.kw, r.inv,
                r.sinks, r.scores, r.out, r.eps, r.scale, r.stream);
        });
    });
}

// handle, slots or block tables, past, starts, n_keep, path, stream
PyObject* keep_path(PyObject* const* a, Py_ssize_t n, bool paged) {
    return run(n, 7, [&] {
        const int dev = static_cast<int>(c10::cuda::current_device());
        slotkv_t h = static_cast<slotkv_t>(pointer(a[0]));
        const at::Tensor& tp = tensor(a[2], I32, dev);
        const at::Tensor& path = tensor(a[5], I32, dev);
        if (tp.dim() != 1 || path.dim() != 1 || tp.size(0) >= UINT32_MAX ||
            path.size(0) > UINT32_MAX)
            throw Unlike{};
        const int64_t R = tp.size(0);
        const at::Tensor& idx = tensor(a[1], I32, dev);
        if (idx.dim() != (paged ? 2 : 1) || idx.size(0) != R ||
            (paged && idx.size(1) > UINT32_MAX))
            throw Unlike{};
        const uint32_t* past = static_cast<const uint32_t*>(tp.data_ptr());
        const uint32_t* where = static_cast<const uint32_t*>(idx.data_ptr());
        const uint32_t* starts = ints(a[3], dev, {R + 1});
        const uint32_t* n_keep = ints(a[4], dev, {R});
        const uint32_t* p = static_cast<const uint32_t*>(path.data_ptr());
        const uint32_t r = static_cast<uint32_t>(R), t = static_cast<uint32_t>(path.size(0));
        slotkv_stream_t stream = stream_of(a[6], dev);
        return without_gil([&] {
            return paged ? slot_kv_keep_path_paged(h, r, t, where,
                                                   static_cast<uint32_t>(idx.size(1)), past,
                                                   starts, n_keep, p, stream)
                         : slot_kv_keep_path(h, r, t, where, past, starts, n_keep, p, stream);
        });
    });
}
PyObject* py_keep(PyObject*, PyObject* const* a, Py_ssize_t n) { return keep_path(a, n, false); }
PyObject* py_keep_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return keep_path(a, n, true);
}

// The arguments that the calls on pages share: past [rows], block tables
// [rows][stride], shares (or None), free list, head.
struct Pages {
    slotkv_t h;
    int dev;
    uint32_t rows, stride, n_free;
    uint32_t *past, *tables, *shares, *free_ids, *head;
    int64_t shape1;
    Pages(PyObject* handle, PyObject* n_blocks, PyObject* o_past, PyObject* o_tables,
          PyObject* o_shares, PyObject* o_free, PyObject* o_head) {
        dev = static_cast<int>(c10::cuda::current_device());
        h = static_cast<slotkv_t>(pointer(handle));
        const at::Tensor& tab = tensor(o_tables, I32, dev);
        const at::Tensor& f = tensor(o_free, I32, dev);
        if (tab.dim() != 2 || f.dim() != 1 || tab.size(0) > UINT32_MAX ||
            tab.size(1) > UINT32_MAX || f.size(0) > UINT32_MAX)
            throw Unlike{};
        shape1 = tab.size(1);
        rows = static_cast<uint32_t>(tab.size(0));
        stride = static_cast<uint32_t>(shape1);
        n_free = static_cast<uint32_t>(f.size(0));
        past = ints(o_past, dev, {tab.size(0)});
        tables = static_cast<uint32_t*>(tab.data_ptr());
        shares = o_shares == Py_None ? nullptr : ints(o_shares, dev, {integer(n_blocks)});
        free_ids = static_cast<uint32_t*>(f.data_ptr());
        head = ints(o_head, dev, {1});
    }
};

// handle, n_blocks, src, past, block tables, out tables, shares, free list, head,
// head out, stream
PyObject* py_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return run(n, 11, [&] {
        const Pages p(a[0], a[1], a[3], a[4], a[6], a[7], a[8]);
        const at::Tensor& src = tensor(a[2], I32, p.dev);
        if (src.dim() != 1 || src.size(0) > UINT32_MAX || !p.shares) throw Unlike{};
        uint32_t* out = ints(a[5], p.dev, {src.size(0), p.shape1});
        uint32_t* head_out = ints(a[9], p.dev, {1});
        slotkv_stream_t stream = stream_of(a[10], p.dev);
        return without_gil([&] {
            return slot_kv_fork_tables(p.h, static_cast<uint32_t>(src.size(0)),
                                       static_cast<const uint32_t*>(src.data_ptr()), p.rows,
                                       p.past, p.tables, p.stride, out, p.shares, p.free_ids,
                                       p.n_free, p.head, head_out, stream);
        });
    });
}

// handle, n_blocks, past, keep, block tables, shares, free list, head, head out, stream
PyObject* py_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return run(n, 10, [&] {
        const Pages p(a[0], a[1], a[2], a[4], a[5], a[6], a[7]);
        const uint32_t* keep = ints_or_null(a[3], p.dev, {static_cast<int64_t>(p.rows)});
        uint32_t* head_out = ints(a[8], p.dev, {1});
        slotkv_stream_t stream = stream_of(a[9], p.dev);
        return without_gil([&] {
            return slot_kv_free_tables(p.h, p.rows, p.past, keep, p.tables, p.stride, p.shares,
                                       p.free_ids, p.n_free, p.head, head_out, stream);
        });
    });
}

// handle, n_blocks, past, block tables, shares, free list, head, stream
PyObject* py_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return run(n, 8, [&] {
        const Pages p(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
        slotkv_stream_t stream = stream_of(a[7], p.dev);
        return without_gil([&] {
            return slot_kv_compact_pool(p.h, p.rows, p.past, p.tables, p.stride, p.shares,
                                        p.free_ids, p.n_free, p.head, stream);
        });
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<py_decode>("decode_batch_attn_scored"),
                         method<py_prefill>("prefill_batch_attn_scored"),
                         method<py_paged>("decode_batch_attn_paged_scored"),
                         method<py_shared>("decode_batch_attn_shared"),
                         method<py_token_map>("slot_kv_token_map"),
                         method<py_extend_tables>("slot_kv_extend_tables"),
                         method<py_tree>("tree_batch_attn"),
                         method<py_tree_paged>("tree_batch_attn_paged"),
                         method<py_keep>("slot_kv_keep_path"),
                         method<py_keep_paged>("slot_kv_keep_path_paged"),
                         method<py_fork>("slot_kv_fork_tables"),
                         method<py_free>("slot_kv_free_tables"),
                         method<py_compact>("slot_kv_compact_pool"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_slotkv_call", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__slotkv_call() { return PyModule_Create(&module); }
