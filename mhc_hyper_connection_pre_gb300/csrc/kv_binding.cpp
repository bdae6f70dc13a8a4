// kv_binding.cpp -- Python binding of the calls in include/mhc_kv.h, as a
// CPython extension over PyTorch's tensors (module _mhc_kv; kv.py is its
// Python side).
//
// Why not ctypes, as for the seam's calls: a decode step's append and attend
// each take a dozen tensors to check and a few microseconds on the GPU, and
// checking the tensors from Python took 30 to 45 us a call.  Here it takes
// about one.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "mhc_kv.h"

namespace {

PyObject* g_error = nullptr;                  // MhcError(fn, status, message)

// Thrown as the Python exception of that type.
struct Refused {
    PyObject* type;
    std::string what;
};
[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// A contiguous tensor of `type` on CUDA device `dev`.
void check_dense(const at::Tensor& t, const char* name, at::ScalarType type, const at::Device& dev) {
    if (!t.is_cuda() || t.device() != dev)
        value_error(std::string(name) + " must be on the cache's CUDA device (got " + t.device().str() + ")");
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + c10::toString(type) + " (got " + c10::toString(t.scalar_type()) + ")");
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}

template <class T>
T* data(const at::Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

mhc_kv_cache cache_of(PyObject* const* o, at::Device& dev) {
    const at::Tensor &k = tensor(o[0], "cache['k']"), &v = tensor(o[1], "cache['v']");
    const at::Tensor &ks = tensor(o[2], "cache['k_scale']"), &vs = tensor(o[3], "cache['v_scale']");
    if (k.dim() != 4) value_error("cache['k'] must be [num_pages, heads, page_tokens, head_dim]");
    if (!v.sizes().equals(k.sizes())) value_error("cache['k'] and cache['v'] must have the same shape");
    dev = k.device();
    check_dense(k, "cache['k']", at::kFloat8_e4m3fn, dev);
    check_dense(v, "cache['v']", at::kFloat8_e4m3fn, dev);
    const int64_t pages = k.size(0), heads = k.size(1), tokens = k.size(2), dim = k.size(3);
    const std::pair<const at::Tensor*, const char*> scales[] = {{&ks, "cache['k_scale']"}, {&vs, "cache['v_scale']"}};
    for (const auto& s : scales) {
        if (s.first->dim() != 2 || s.first->size(0) != pages || s.first->size(1) != heads)
            value_error(std::string(s.second) + " must be [num_pages, heads]");
        check_dense(*s.first, s.second, at::kFloat, dev);
    }
    if (heads > 0x7fffffff || tokens > 0x7fffffff || dim > 0x7fffffff) value_error("cache['k'] is too large");
    return mhc_kv_cache{data<uint8_t>(k), data<uint8_t>(v), data<float>(ks), data<float>(vs), pages, (int)heads,
                        (int)tokens, (int)dim};
}

// bf16 [T, heads, head_dim] whose heads lie one after the other; rows may have a stride.
struct Rows {
    uint16_t* p = nullptr;
    int64_t stride = 0, tokens = 0, heads = 0;
};

Rows rows_of(const at::Tensor& t, const char* name, const mhc_kv_cache& c, const at::Device& dev) {
    if (t.dim() != 3 || t.size(2) != c.head_dim)
        value_error(std::string(name) + " must be [T, heads, " + std::to_string(c.head_dim) + "]");
    if (t.device() != dev) value_error(std::string(name) + " must be on the cache's device (got " + t.device().str() + ")");
    if (t.scalar_type() != at::kBFloat16)
        type_error(std::string(name) + " must be BFloat16 (got " + c10::toString(t.scalar_type()) + ")");
    Rows r;
    r.tokens = t.size(0);
    r.heads = t.size(1);
    if (r.tokens && ((t.stride(2) != 1 && t.size(2) > 1) || (t.stride(1) != t.size(2) && r.heads > 1)))
        value_error(std::string(name) + ": the heads of a token must be contiguous");
    r.p = data<uint16_t>(t);
    r.stride = r.tokens > 1 ? t.stride(0) : std::max<int64_t>(r.heads * t.size(2), 1);
    return r;
}

struct Seqs {
    const int32_t *table, *lens, *cu;
    int64_t width, B;
};

Seqs seqs_of(PyObject* table_o, PyObject* lens_o, PyObject* cu_o, int64_t T, const at::Device& dev) {
    const at::Tensor &table = tensor(table_o, "block_table"), &lens = tensor(lens_o, "seq_lens");
    if (table.dim() != 2 || lens.dim() != 1 || table.size(0) != lens.size(0))
        value_error("block_table must be [B, width] and seq_lens [B]");
    Seqs s{nullptr, nullptr, nullptr, table.size(1), table.size(0)};
    if (!given(cu_o)) {
        if (T != s.B) value_error("without cu_q there is one new token for each sequence");
    } else {
        const at::Tensor& cu = tensor(cu_o, "cu_q");
        if (cu.dim() != 1 || cu.size(0) != s.B + 1) value_error("cu_q must be [B + 1]");
        check_dense(cu, "cu_q", at::kInt, dev);
        s.cu = data<int32_t>(cu);
    }
    check_dense(table, "block_table", at::kInt, dev);
    check_dense(lens, "seq_lens", at::kInt, dev);
    s.table = data<int32_t>(table);
    s.lens = data<int32_t>(lens);
    return s;
}

void check_cuda(cudaError_t e, const char* what) {
    if (e != cudaSuccess) throw Refused{PyExc_RuntimeError, std::string(what) + ": " + cudaGetErrorString(e)};
}

// The workspace of captured calls (the seam's as well).  Replays write it at any time and on any
// stream, so it is the graph's alone, for as long as the graph or an
// instantiation of it lives: the graph holds a CUDA user object whose end hands
// the memory back.  The calls of one capture on one stream follow one another
// and share it.  (A buffer of the capturing allocator alone would not do: it is
// free again once the call has returned, and outside of PyTorch's own captures
// to anybody.)
enum User { kAttend, kPre, kHost, kUsers };      // of the library's calls, each has its own

struct Captured {
    at::Tensor memory;
    User user;
    cudaStream_t stream;
    unsigned long long capture;
};

std::mutex g_mutex;                                              // of what follows; never held during a CUDA call
auto* const g_kept = new std::map<std::pair<int, cudaStream_t>, at::Tensor>();    // never destroyed: outlives CUDA
auto* const g_captured = new std::vector<Captured*>();           // of graphs that live
auto* const g_gone = new std::vector<Captured*>();               // of graphs that do not

// Called by CUDA, on a thread of its own, where no CUDA function may be called.
void CUDART_CB graph_is_gone(void* p) {
    std::lock_guard<std::mutex> lock(g_mutex);
    g_captured->erase(std::remove(g_captured->begin(), g_captured->end(), p), g_captured->end());
    g_gone->push_back(static_cast<Captured*>(p));
}

at::Tensor new_workspace(size_t need, const at::Device& dev) {
    return at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(dev));
}

// The workspace for a call on a stream that is being captured; undefined if it is not.
at::Tensor captured_workspace(User user, size_t need, const at::Device& dev, cudaStream_t stream) {
    std::vector<Captured*> gone;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        gone.swap(*g_gone);
    }
    for (Captured* c : gone) delete c;
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    check_cuda(cudaStreamIsCapturing(stream, &status), "cudaStreamIsCapturing");
    if (status == cudaStreamCaptureStatusNone) return at::Tensor();
    unsigned long long capture = 0;
    cudaGraph_t graph = nullptr;
    const cudaGraphNode_t* nodes = nullptr;
    const cudaGraphEdgeData* edges = nullptr;
    size_t n = 0;
    check_cuda(cudaStreamGetCaptureInfo(stream, &status, &capture, &graph, &nodes, &edges, &n), "cudaStreamGetCaptureInfo");
    if (status != cudaStreamCaptureStatusActive) check_cuda(cudaErrorStreamCaptureInvalidated, "kv workspace");
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        for (Captured* c : *g_captured)
            if (c->user == user && c->stream == stream && c->capture == capture && (size_t)c->memory.numel() >= need)
                return c->memory;
    }
    auto* c = new Captured{new_workspace(need, dev), user, stream, capture};
    at::Tensor memory = c->memory;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        g_captured->push_back(c);
    }
    // a graph that cannot hold one leaves the memory with us, for good
    cudaUserObject_t object = nullptr;
    if (cudaUserObjectCreate(&object, c, graph_is_gone, 1, cudaUserObjectNoDestructorSync) != cudaSuccess ||
        cudaGraphRetainUserObject(graph, object, 1, cudaGraphUserObjectMove) != cudaSuccess)
        cudaGetLastError();
    return memory;
}

// The workspace of a device and stream: kept and grown, as a user's program
// would; of a stream that is being captured, the graph's.
at::Tensor workspace_for(const mhc_kv_cache& c, int64_t q_heads, int64_t B, int64_t T, const at::Device& dev,
                         const c10::cuda::CUDAStream& stream) {
    const size_t need = mhc_kv_attend_workspace_bytes(&c, (int)q_heads, B, T);
    if (need == 0) return at::Tensor();
    at::Tensor t = captured_workspace(kAttend, need, dev, stream.stream());
    if (t.defined()) return t;
    const std::pair<int, cudaStream_t> key(dev.index(), stream.stream());
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        const at::Tensor& kept = (*g_kept)[key];
        if (kept.defined() && (size_t)kept.numel() >= need) return kept;
    }
    t = new_workspace(need, dev);
    at::Tensor old = t;                       // let go of after the lock
    std::lock_guard<std::mutex> lock(g_mutex);
    std::swap((*g_kept)[key], old);
    return t;
}

void check_status(const char* fn, mhc_status st) {
    if (st == MHC_OK) return;
    PyObject* args = Py_BuildValue("(sis)", fn, (int)st, mhc_status_string(st));
    if (args) PyErr_SetObject(g_error, args);
    Py_XDECREF(args);
    throw Refused{nullptr, ""};
}

// Runs f, its C++ exceptions as Python ones.
template <class F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const Refused& r) {
        if (r.type) PyErr_SetString(r.type, r.what.c_str());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool truth(PyObject* o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw Refused{nullptr, ""};
    return t != 0;
}

void count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) type_error("wrong number of arguments");
}

// append(k codes, v codes, k_scale, v_scale, k, v, block_table, seq_lens, cu_q, q, cos, sin, interleaved, q_out)
PyObject* append(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        count(n, 14);
        at::Device dev(at::kCPU);
        const mhc_kv_cache c = cache_of(o, dev);
        const Rows k = rows_of(tensor(o[4], "k"), "k", c, dev), v = rows_of(tensor(o[5], "v"), "v", c, dev);
        if (k.tokens != v.tokens || k.heads != v.heads || k.heads != c.heads)
            value_error("k and v must be [T, heads, head_dim] with the cache's heads");
        const Seqs s = seqs_of(o[6], o[7], o[8], k.tokens, dev);
        const c10::cuda::CUDAGuard guard(dev);
        Rows q, out;
        at::Tensor q_out;
        if (given(o[9])) {
            q = rows_of(tensor(o[9], "q"), "q", c, dev);
            if (q.tokens != k.tokens) value_error("q must have as many tokens as k and v");
            if (q.heads > 0x7fffffff) value_error("q has too many heads");
            q_out = given(o[13]) ? tensor(o[13], "q_out")
                                 : at::empty({q.tokens, q.heads, c.head_dim}, at::TensorOptions().dtype(at::kBFloat16).device(dev));
            out = rows_of(q_out, "q_out", c, dev);
            if (out.tokens != q.tokens || out.heads != q.heads) value_error("q_out must have q's shape");
        } else if (given(o[13])) {
            value_error("q_out without q");
        }
        const float *cos = nullptr, *sin = nullptr;
        int64_t rows = 0, dim = 0;
        if (given(o[10]) != given(o[11])) value_error("cos and sin go together");
        if (given(o[10])) {
            const at::Tensor &ct = tensor(o[10], "cos"), &st = tensor(o[11], "sin");
            if (ct.dim() != 2 || !ct.sizes().equals(st.sizes())) value_error("cos and sin must be [positions, rotary_dim / 2]");
            check_dense(ct, "cos", at::kFloat, dev);
            check_dense(st, "sin", at::kFloat, dev);
            cos = data<float>(ct);
            sin = data<float>(st);
            rows = ct.size(0);
            dim = std::min<int64_t>(2 * ct.size(1), 1 << 20);
        }
        const bool inter = truth(o[12]);
        check_status("mhc_kv_append",
                     mhc_kv_append(&c, k.p, k.stride, v.p, v.stride, q.p, q.stride, (int)q.heads, out.p, out.stride, cos,
                                   sin, rows, (int)dim, inter, s.table, s.width, s.lens, s.cu, s.B, k.tokens,
                                   c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
        if (!q_out.defined()) Py_RETURN_NONE;
        if (given(o[13])) {
            Py_INCREF(o[13]);
            return o[13];
        }
        return THPVariable_Wrap(std::move(q_out));
    });
}

// attend(q, k codes, v codes, k_scale, v_scale, block_table, seq_lens, cu_q, softmax_scale, out, lse, return_lse,
// workspace) -> (out, lse)
PyObject* attend(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        count(n, 13);
        at::Device dev(at::kCPU);
        const mhc_kv_cache c = cache_of(o + 1, dev);
        const Rows q = rows_of(tensor(o[0], "q"), "q", c, dev);
        const Seqs s = seqs_of(o[5], o[6], o[7], q.tokens, dev);
        if (q.heads > 0x7fffffff) value_error("q has too many heads");
        double scale = 1.0 / std::sqrt((double)c.head_dim);
        if (given(o[8])) {
            scale = PyFloat_AsDouble(o[8]);
            if (PyErr_Occurred()) throw Refused{nullptr, ""};
        }
        const c10::cuda::CUDAGuard guard(dev);
        const auto stream = c10::cuda::getCurrentCUDAStream(dev.index());
        at::Tensor out, lse, ws;
        if (given(o[9])) {
            out = tensor(o[9], "out");
            check_dense(out, "out", at::kBFloat16, dev);
            if (out.dim() != 3 || out.size(0) != q.tokens || out.size(1) != q.heads || out.size(2) != c.head_dim)
                value_error("out has the wrong shape");
        } else {
            out = at::empty({q.tokens, q.heads, c.head_dim}, at::TensorOptions().dtype(at::kBFloat16).device(dev));
        }
        if (given(o[10])) {
            lse = tensor(o[10], "lse");
            check_dense(lse, "lse", at::kFloat, dev);
            if (lse.dim() != 2 || lse.size(0) != q.tokens || lse.size(1) != q.heads) value_error("lse has the wrong shape");
        } else if (truth(o[11])) {
            lse = at::empty({q.tokens, q.heads}, at::TensorOptions().dtype(at::kFloat).device(dev));
        }
        if (given(o[12])) {
            ws = tensor(o[12], "workspace");
            check_dense(ws, "workspace", at::kByte, dev);
        } else {
            ws = workspace_for(c, q.heads, s.B, q.tokens, dev, stream);
        }
        check_status("mhc_kv_attend",
                     mhc_kv_attend(&c, q.p, q.stride, (int)q.heads, s.table, s.width, s.lens, s.cu, s.B, q.tokens,
                                   (float)scale, data<uint16_t>(out), lse.defined() ? data<float>(lse) : nullptr,
                                   ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0,
                                   stream.stream()));
        PyObject* a = given(o[9]) ? o[9] : THPVariable_Wrap(std::move(out));
        if (given(o[9])) Py_INCREF(a);
        PyObject* b = given(o[10]) ? o[10] : (lse.defined() ? THPVariable_Wrap(std::move(lse)) : Py_None);
        if (b == o[10] || b == Py_None) Py_INCREF(b);
        PyObject* r = PyTuple_Pack(2, a, b);
        Py_DECREF(a);
        Py_DECREF(b);
        return r;
    });
}

// workspace(k codes, v codes, k_scale, v_scale, q_heads, B, T): the one that attend keeps for the current stream, or None
PyObject* workspace(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        count(n, 7);
        at::Device dev(at::kCPU);
        const mhc_kv_cache c = cache_of(o, dev);
        int64_t v[3];
        for (int i = 0; i < 3; ++i) {
            v[i] = PyLong_AsLongLong(o[4 + i]);
            if (PyErr_Occurred()) throw Refused{nullptr, ""};
        }
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor t = workspace_for(c, v[0], v[1], v[2], dev, c10::cuda::getCurrentCUDAStream(dev.index()));
        if (!t.defined()) Py_RETURN_NONE;
        return THPVariable_Wrap(std::move(t));
    });
}

// captured(user, bytes, device index, stream): the workspace of the capture that is under way on the stream, or None
PyObject* captured(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        count(n, 4);
        const long long user = PyLong_AsLongLong(o[0]), need = PyLong_AsLongLong(o[1]), index = PyLong_AsLongLong(o[2]);
        void* const stream = PyLong_AsVoidPtr(o[3]);
        if (PyErr_Occurred()) throw Refused{nullptr, ""};
        if (user < 0 || user >= kUsers || need < 1) value_error("no such workspace");
        const at::Device dev(at::kCUDA, (c10::DeviceIndex)index);
        const auto on = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), dev.index());
        const c10::cuda::CUDAStreamGuard guard(on);              // memory is the stream's
        at::Tensor t = captured_workspace((User)user, (size_t)need, dev, on.stream());
        if (!t.defined()) Py_RETURN_NONE;
        return THPVariable_Wrap(std::move(t));
    });
}

// set_error(MhcError)
PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, "mhc_kv_append"},
    {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, "mhc_kv_attend"},
    {"workspace", (PyCFunction)(void (*)(void))workspace, METH_FASTCALL, "a workspace for attend"},
    {"captured", (PyCFunction)(void (*)(void))captured, METH_FASTCALL, "a workspace of a capture"},
    {"set_error", set_error, METH_O, "the exception for a status that is not MHC_OK"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mhc_kv", "binding of include/mhc_kv.h", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mhc_kv(void) { return PyModule_Create(&module); }
