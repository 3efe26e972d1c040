// binding.cpp — the torch side of the calls around the verify step (beam
// selection, state reordering, slot planning, path commit): checks of the
// tensors, then the C-ABI of libspecdec.so.
//
// Their kernels take a few microseconds, and a dozen tensors checked from
// Python take ten; read here they take half of one.  The Python functions keep
// the defaults, the allocation of outputs and the errors of the C-ABI; each
// function below returns its status.  Arguments are positional, as the Python
// side passes them; `stream` is a handle, or None for the current stream of
// device `cur`, the current device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include "../../include/specdec.h"

namespace {

decltype(&specdec_beam_select) f_beam_select = nullptr;
decltype(&specdec_reorder_states) f_reorder_states = nullptr;
decltype(&specdec_commit_path) f_commit_path = nullptr;
decltype(&specdec_plan_slots) f_plan_slots = nullptr;

struct Refused : std::runtime_error {  // becomes a ValueError
    using std::runtime_error::runtime_error;
};
struct WrongType : std::runtime_error {  // becomes a TypeError
    using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python error is set

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw WrongType(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

void on(const at::Tensor& t, int cur, const char* name) {
    if (!t.is_cuda())
        throw Refused(std::string("verifier arrays must be CUDA device tensors, got ") + name + " on " + t.device().str());
    if (t.get_device() != cur)
        throw Refused("arguments must be on the current device cuda:" + std::to_string(cur) + ", got " + name + " on " +
                      t.device().str());
}

// Address of a contiguous tensor of that type and shape.
void* want(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, int cur, const char* name) {
    const at::Tensor& t = tensor(o, name);
    on(t, cur, name);
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous()) {
        std::string s;
        for (int64_t d : shape) s += (s.empty() ? "" : ", ") + std::to_string(d);
        throw Refused(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape [" + s + "]");
    }
    return t.data_ptr();
}
void* want_or_null(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, int cur, const char* name) {
    return o == Py_None ? nullptr : want(o, type, shape, cur, name);
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
int small(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    if (v < INT_MIN || v > INT_MAX) throw Refused(std::string(name) + " is out of range");
    return static_cast<int>(v);
}

CUstream_st* stream_of(PyObject* o, int cur) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(cur)).stream();
    return reinterpret_cast<CUstream_st*>(static_cast<uintptr_t>(integer(o)));
}

// The bytes a tensor's elements lie in.
bool overlap(const at::Tensor& a, const at::Tensor& b) {
    auto last = [](const at::Tensor& t) {
        int64_t n = 1;
        for (int64_t d = 0; d < t.dim(); ++d) n += (t.size(d) - 1) * t.stride(d);
        return static_cast<char*>(t.data_ptr()) + n * static_cast<int64_t>(t.element_size());
    };
    return static_cast<char*>(a.data_ptr()) < last(b) && static_cast<char*>(b.data_ptr()) < last(a);
}

// Elements of a row: the dimensions from `lead` on, which must lie one behind
// the other.
int64_t row_elems(const at::Tensor& t, int64_t lead, const char* name) {
    int64_t n = 1;
    for (int64_t d = t.dim() - 1; d >= lead; --d) {
        if (t.stride(d) != n && t.size(d) != 1)
            throw Refused(std::string(name) + ": the dimensions of a row must be contiguous");
        n *= t.size(d);
    }
    return n;
}

// Rows that are written (`row` elements each, over the first `lead` dimensions)
// must not share memory: from the smallest stride on, each has to pass what lies
// within it.
void rows_apart(const at::Tensor& t, int64_t lead, int64_t row) {
    std::vector<std::pair<int64_t, int64_t>> d;  // stride, size
    for (int64_t i = 0; i < lead; ++i)
        if (t.size(i) > 1) d.emplace_back(t.stride(i), t.size(i));
    std::sort(d.begin(), d.end());
    int64_t extent = row;
    for (const auto& [stride, size] : d) {
        if (stride < extent) throw Refused("the rows written must not share memory");
        extent += stride * (size - 1);
    }
}

template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want_n, F f) {
    if (got != want_n) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want_n, got);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Raised&) {
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const WrongType& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// logits, beam_scores, num_beams, finished, eos_token, (scores, parents,
// tokens), workspace or None, its bytes, stream, cur
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> int {
        const int cur = small(a[9], "device");
        const at::Tensor& x = tensor(a[0], "logits");
        on(x, cur, "logits");
        if (x.scalar_type() != at::kBFloat16 && x.scalar_type() != at::kFloat)
            throw WrongType(std::string("logits must be bfloat16 or float32, got ") + c10::toString(x.scalar_type()));
        if (x.dim() != 3 || x.stride(2) != 1)
            throw Refused("logits must be a 3-D tensor with a contiguous last dimension");
        const int64_t B = x.size(0), W = x.size(1), V = x.size(2);
        int64_t rs = V;
        if (W > 1) {
            rs = x.stride(1);
            if (B > 1 && x.stride(0) != W * rs) throw Refused("logits: rows are not evenly spaced");
        } else if (B > 1) {
            rs = x.stride(0);
        }
        if (rs < V) throw Refused("logits: overlapping rows");
        if (B > INT_MAX || W > INT_MAX || V > INT_MAX) return SPECDEC_ERR_INVALID_ARG;
        const int K = small(a[2], "num_beams"), eos = small(a[4], "eos_token");
        const int64_t k = K > 0 ? K : 0;
        const void* scores = want(a[1], at::kFloat, {B, W}, cur, "beam_scores");
        const void* finished = want_or_null(a[3], at::kInt, {B, W}, cur, "finished");
        if (!PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 3) throw Refused("out must be (scores, parents, tokens)");
        void* os = want(PyTuple_GET_ITEM(a[5], 0), at::kFloat, {B, k}, cur, "out: scores");
        void* op = want(PyTuple_GET_ITEM(a[5], 1), at::kInt, {B, k}, cur, "out: parents");
        void* ot = want(PyTuple_GET_ITEM(a[5], 2), at::kInt, {B, k}, cur, "out: tokens");
        void* ws = nullptr;
        if (a[6] != Py_None) {
            const at::Tensor& w = tensor(a[6], "workspace");
            on(w, cur, "workspace");
            ws = w.data_ptr();
        }
        return f_beam_select(x.data_ptr(), x.scalar_type() == at::kFloat ? SPECDEC_F32 : SPECDEC_BF16, rs,
                             static_cast<const float*>(scores), static_cast<const int32_t*>(finished), eos,
                             static_cast<int>(B), static_cast<int>(W), K, static_cast<int>(V), static_cast<float*>(os),
                             static_cast<int32_t*>(op), static_cast<int32_t*>(ot), ws,
                             static_cast<size_t>(integer(a[7])), stream_of(a[8], cur));
    });
}

// states, parents, lengths, time_dim, out or None, stream, cur
PyObject* reorder_states(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> int {
        const int cur = small(a[6], "device");
        const at::Tensor& x = tensor(a[0], "states");
        const at::Tensor& to = a[4] == Py_None ? x : tensor(a[4], "out");
        const int td = small(a[3], "time_dim");
        if ((td != 3 && td != 4) || x.dim() <= td)
            throw Refused("states must be [G, B, W, T, ...] (time_dim 3) or [G, B, W, H, T, ...] (time_dim 4)");
        on(x, cur, "states");
        on(to, cur, "out");
        if (to.sizes() != x.sizes() || to.scalar_type() != x.scalar_type())
            throw Refused("out must have the shape and type of states");
        const int64_t G = x.size(0), B = x.size(1), W = x.size(2), H = td == 4 ? x.size(3) : 1, T = x.size(td);
        const void* parents = want(a[1], at::kInt, {B, W}, cur, "parents");
        const void* lengths = want_or_null(a[2], at::kInt, {B}, cur, "lengths");
        const int64_t row = row_elems(x, td + 1, "states");
        row_elems(to, td + 1, "out");
        if (x.numel() == 0) return SPECDEC_OK;
        if (!(to.data_ptr() == x.data_ptr() && to.strides() == x.strides()) && overlap(x, to))
            throw Refused("out overlaps states: pass none to reorder in place");
        const int64_t es = static_cast<int64_t>(x.element_size());
        int64_t ss[5], ds[5];
        for (int i = 0; i < 5; ++i) {
            const int d = i < 3 ? i : i == 3 ? (td == 4 ? 3 : -1) : td;
            ss[i] = d < 0 ? 0 : x.stride(d) * es;
            ds[i] = d < 0 ? 0 : to.stride(d) * es;
        }
        rows_apart(to, td + 1, row);
        if (B > INT_MAX || W > INT_MAX) return SPECDEC_ERR_INVALID_ARG;
        return f_reorder_states(x.data_ptr(), to.data_ptr(), static_cast<const int32_t*>(parents),
                                static_cast<const int32_t*>(lengths), G, static_cast<int>(B), static_cast<int>(W), H, T,
                                row * es, ss, ds, stream_of(a[5], cur));
    });
}

struct Slots {
    const int64_t* at = nullptr;
    int64_t n = 0, stride = 0;
};
Slots slot_table(PyObject* o, int64_t B, int cur, const char* name) {
    const at::Tensor& t = tensor(o, name);
    on(t, cur, name);
    if (t.scalar_type() != at::kLong || t.dim() != 2 || t.size(0) != B || (t.stride(1) != 1 && t.size(1) != 1) ||
        (t.stride(0) < t.size(1) && B > 1))
        throw Refused(std::string(name) + " must be an int64 [B, n] tensor with contiguous rows");
    Slots s;
    s.at = static_cast<const int64_t*>(t.data_ptr());
    s.n = t.size(1);
    s.stride = t.stride(0) > s.n ? t.stride(0) : s.n;
    return s;
}

// src, accept_len, accept_nodes, dst, dst_slots, src_slots or None, stream, cur
PyObject* commit_path(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> int {
        const int cur = small(a[7], "device");
        const at::Tensor &src = tensor(a[0], "src"), &dst = tensor(a[3], "dst"), &nodes = tensor(a[2], "accept_nodes");
        on(src, cur, "src");
        on(dst, cur, "dst");
        if (nodes.dim() != 2) throw Refused("accept_nodes must be [B, max_depth]");
        const int64_t B = nodes.size(0), depth = nodes.size(1);
        const void* path = want(a[2], at::kInt, {B, depth}, cur, "accept_nodes");
        const void* len = want(a[1], at::kInt, {B}, cur, "accept_len");
        const bool paged = a[5] != Py_None;
        const int64_t lead = paged ? 2 : 3;
        if (src.dim() < lead || dst.dim() < 2 || src.scalar_type() != dst.scalar_type() ||
            src.sizes().slice(lead) != dst.sizes().slice(2) || src.size(0) != dst.size(0) ||
            (!paged && src.size(1) != B))
            throw Refused(
                "src must be [G, B, N + 1, ...] (with src_slots [G, S, ...]) and dst [G, slots, ...] of its type");
        const Slots to = slot_table(a[4], B, cur, "dst_slots");
        if (to.n < depth + 1) throw Refused("dst_slots must have max_depth + 1 columns at least");
        Slots from;
        if (paged) from = slot_table(a[5], B, cur, "src_slots");
        const int64_t row = row_elems(src, lead, "src");
        row_elems(dst, 2, "dst");
        if (src.numel() == 0 || dst.numel() == 0 || B == 0) return SPECDEC_OK;
        const bool same = paged && src.data_ptr() == dst.data_ptr() && src.strides() == dst.strides();
        if (!same && overlap(src, dst))
            throw Refused("src and dst overlap: in place both must be the same cache, with src_slots");
        rows_apart(dst, 2, row);
        const int64_t es = static_cast<int64_t>(src.element_size());
        const int64_t rows = paged ? src.size(1) : src.size(2);  // rows along the row stride
        int64_t sr = paged ? src.stride(1) : src.stride(2), dr = dst.stride(1);
        if (rows == 1 && sr < row) sr = row;
        if (dst.size(1) == 1 && dr < row) dr = row;
        const int64_t count = paged ? from.n : src.size(2);
        if (B > INT_MAX || count > INT_MAX || depth > INT_MAX) return SPECDEC_ERR_INVALID_ARG;
        return f_commit_path(src.data_ptr(), src.stride(0) * es, paged ? 0 : src.stride(1) * es, sr * es, from.at,
                             from.stride, paged ? rows : 0, dst.data_ptr(), dst.stride(0) * es, dr * es, to.at, to.stride,
                             dst.size(1), static_cast<const int32_t*>(len), static_cast<const int32_t*>(path),
                             src.size(0), static_cast<int>(B), static_cast<int>(count) - 1, static_cast<int>(depth),
                             row * es, stream_of(a[6], cur));
    });
}

// seq_lens, block_tables, held_blocks, free_ring, ring_state, block_size, k,
// draft_offsets, total_drafts, accept_len, release, (seq_lens, held_blocks,
// ring_state, positions, slots), stream, cur
PyObject* plan_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> int {
        const int cur = small(a[13], "device");
        const int64_t B = tensor(a[0], "seq_lens").numel(), ring = tensor(a[3], "free_ring").numel();
        const int block_size = small(a[5], "block_size"), k = small(a[6], "k");
        const int64_t total = integer(a[8]);
        const void* lens = want(a[0], at::kInt, {B}, cur, "seq_lens");
        const at::Tensor& tables = tensor(a[1], "block_tables");
        on(tables, cur, "block_tables");
        if (tables.scalar_type() != at::kInt || tables.dim() != 2 || tables.size(0) != B ||
            (tables.stride(1) != 1 && tables.size(1) != 1) || (B > 1 && tables.stride(0) < tables.size(1)))
            throw Refused("block_tables must be an int32 [B, max_blocks] tensor with contiguous rows");
        const int64_t cols = tables.size(1), ts = tables.stride(0) > cols ? tables.stride(0) : cols;
        const void* held = want(a[2], at::kInt, {B}, cur, "held_blocks");
        void* free_ring = want(a[3], at::kInt, {ring}, cur, "free_ring");
        const void* state = want(a[4], at::kInt, {2}, cur, "ring_state");
        const void* offsets = want_or_null(a[7], at::kInt, {B + 1}, cur, "draft_offsets");
        const void* accept = want_or_null(a[9], at::kInt, {B}, cur, "accept_len");
        const void* release = want_or_null(a[10], at::kInt, {B}, cur, "release");
        const int64_t rows = offsets ? B + total : B * (static_cast<int64_t>(k) + 1);
        if (rows < 0 || total < 0) throw Refused("k and total_drafts must not be negative");
        if (!PyTuple_Check(a[11]) || PyTuple_GET_SIZE(a[11]) != 5)
            throw Refused("out must be (seq_lens, held_blocks, ring_state, positions, slots)");
        auto out = [&](int i) { return PyTuple_GET_ITEM(a[11], i); };
        void* new_lens = want(out(0), at::kInt, {B}, cur, "out: seq_lens");
        void* new_held = want(out(1), at::kInt, {B}, cur, "out: held_blocks");
        void* new_state = want(out(2), at::kInt, {2}, cur, "out: ring_state");
        void* positions = want(out(3), at::kLong, {rows}, cur, "out: positions");
        void* slots = want(out(4), at::kLong, {rows}, cur, "out: slots");
        if (B > INT_MAX || cols > INT_MAX || ring > INT_MAX) return SPECDEC_ERR_INVALID_ARG;
        return f_plan_slots(static_cast<const int32_t*>(lens), static_cast<const int32_t*>(accept),
                            static_cast<const int32_t*>(release), static_cast<const int32_t*>(offsets),
                            static_cast<int>(B), k, total, block_size, static_cast<int32_t*>(tables.data_ptr()), ts,
                            static_cast<int>(cols), static_cast<const int32_t*>(held), static_cast<int32_t*>(free_ring),
                            static_cast<int>(ring), static_cast<const int32_t*>(state), static_cast<int32_t*>(new_lens),
                            static_cast<int32_t*>(new_held), static_cast<int32_t*>(new_state),
                            static_cast<int64_t*>(positions), static_cast<int64_t*>(slots), stream_of(a[12], cur));
    });
}

// Looks the entry points up in the library at `path`.
PyObject* load(PyObject*, PyObject* path) {
    const char* p = PyUnicode_AsUTF8(path);
    if (p == nullptr) return nullptr;
    void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
    if (h == nullptr) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    f_beam_select = reinterpret_cast<decltype(f_beam_select)>(dlsym(h, "specdec_beam_select"));
    f_reorder_states = reinterpret_cast<decltype(f_reorder_states)>(dlsym(h, "specdec_reorder_states"));
    f_commit_path = reinterpret_cast<decltype(f_commit_path)>(dlsym(h, "specdec_commit_path"));
    f_plan_slots = reinterpret_cast<decltype(f_plan_slots)>(dlsym(h, "specdec_plan_slots"));
    if (!f_beam_select || !f_reorder_states || !f_commit_path || !f_plan_slots) {
        PyErr_Format(PyExc_RuntimeError, "%s lacks an entry point: build it again", p);
        return nullptr;
    }
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef fast(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"load", load, METH_O, nullptr},
    fast<beam_select>("beam_select"),
    fast<reorder_states>("reorder_states"),
    fast<commit_path>("commit_path"),
    fast<plan_slots>("plan_slots"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the PyTorch and Python that the binding was compiled against, by
// which the build finds a stale one.
PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
