// torch_ops.cpp -- the binding of the serving calls: checks of the tensors, outputs and workspaces, the C entry.
//
// A step's kernel takes four to ten microseconds.  Through ctypes the call itself took 12 to 22 us on the GPU's host,
// nearly all of it attribute by attribute questions to tensors and conversions of arguments; here they are
// plain C++ on the tensors, 4 to 8 us with the launches.  Every function takes positional arguments from its Python
// wrapper, runs on the current stream and returns new references.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>
#include <string>

#include "kda.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

struct Refused {
    PyObject* type;
    std::string what;
};
struct Raised {};      // a Python error is set
[[noreturn]] void refuse(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

PyObject* g_check;     // raises for a status that is not KDA_OK: check(status, entry)
PyObject* g_scratch;   // (device, kind, stream) -> workspace

void check(kda_status st, const char* what) {
    if (st == KDA_OK) return;
    Py_XDECREF(PyObject_CallFunction(g_check, "is", (int)st, what));
    if (PyErr_Occurred()) throw Raised();
    refuse(std::string(what) + " failed");
}

std::string shape_text(IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

const Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}

void on_device(const char* name, const Tensor& t, int dev) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    if (t.get_device() != dev) refuse(std::string(name) + ": all tensors of a call must be on one CUDA device");
}

// The address of a contiguous tensor of the type and shape on the device; nullptr for None.
void* need(const char* name, PyObject* o, ScalarType type, IntArrayRef shape, int dev) {
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(name, o);
    on_device(name, t, dev);
    if (t.scalar_type() != type) refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape) refuse(std::string(name) + " must be " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
}
template <typename T> T* need_as(const char* name, PyObject* o, ScalarType type, IntArrayRef shape, int dev) {
    return static_cast<T*>(need(name, o, type, shape, dev));
}
float* need_f(const char* name, PyObject* o, IntArrayRef shape, int dev) { return need_as<float>(name, o, at::kFloat, shape, dev); }
int32_t* need_i(const char* name, PyObject* o, IntArrayRef shape, int dev) { return need_as<int32_t>(name, o, at::kInt, shape, dev); }

kda_dtype dtype_code(const Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return KDA_BF16;
    if (t.scalar_type() == at::kFloat) return KDA_FP32;
    throw Refused{PyExc_TypeError, std::string("unsupported activation dtype ") + c10::toString(t.scalar_type()) + " (bf16 or fp32)"};
}

// A call's leading tensor.
const Tensor& leading(const char* name, PyObject* o, int dims) {
    const Tensor& t = tensor(name, o);
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    if (t.dim() != dims) refuse(std::string(name) + " must have " + std::to_string(dims) + " axes, got " + shape_text(t.sizes()));
    return t;
}

int as_int(const char* name, int64_t v) {
    if (v < INT_MIN || v > INT_MAX) refuse(std::string(name) + " is out of range");
    return (int)v;
}
// Documents of a call's offsets.
int64_t documents(PyObject* cu) {
    const int64_t n = tensor("cu_seqlens", cu).numel() - 1;
    if (n < 0) refuse("cu_seqlens must hold one offset more than there are documents");
    return as_int("documents", n);
}
int64_t integer(const char* name, PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return as_int(name, v);
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}
const int32_t* host_copy(PyObject* o) {      // an address, None: none
    if (o == Py_None) return nullptr;
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised();
    return static_cast<const int32_t*>(p);
}

// Elements between neighbouring tokens of a tensor whose first `lead` axes are tokens ([B, T] or [B]) and whose other
// axes are one token's contiguous values: it may be a slice of a wider projection.  Tokens that share memory are
// refused: an expanded axis has stride 0, which is "contiguous" to the C entries.
int64_t token_stride(const char* name, const Tensor& t, int lead) {
    const IntArrayRef size = t.sizes(), stride = t.strides();
    int64_t want = 1, step = -1, span = -1;
    for (int k = (int)t.dim() - 1; k >= lead; --k) {
        if (stride[k] != want && size[k] > 1) refuse(std::string(name) + ": the values of one token must be contiguous");
        want *= size[k];
    }
    for (int k = lead - 1; k >= 0; --k)
        if (size[k] > 1) {
            if (step < 0) step = stride[k];
            else if (stride[k] != span) refuse(std::string(name) + ": tokens must be evenly spaced over the leading axes");
            span = stride[k] * size[k];
        }
    if (step >= 0 && step < want)
        refuse(std::string(name) + ": tokens must not share memory, got a stride of " + std::to_string(step) + " for " +
               std::to_string(want) + " values (expanded tensors: call contiguous())");
    return step < 0 ? want : step;
}

cudaStream_t current_stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

Tensor fresh(const Tensor& like, IntArrayRef shape, ScalarType type) { return at::empty(shape, like.options().dtype(type)); }

// The output tensor of like's shape and type, given or new.
struct Result {
    Tensor own;
    PyObject* given = nullptr;
    void* p = nullptr;
    Result(const char* name, PyObject* o, const Tensor& like, IntArrayRef shape, ScalarType type) {
        if (o == Py_None) {
            own = fresh(like, shape, type);
            p = own.data_ptr();
        } else {
            given = o;
            p = need(name, o, type, shape, (int)like.get_device());
        }
    }
    PyObject* object() const { return given ? Py_NewRef(given) : THPVariable_Wrap(own); }
};

PyObject* pair(PyObject* a, PyObject* b) {      // takes both references
    PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

// A call's workspace: one per device, kind and stream (calls on different streams may overlap), grown on demand.  While
// the stream is captured the call gets a buffer of its own, which the graph keeps: a kept one may be given up for a
// larger one later, and one made here would belong to the graph.
struct Scratch {
    Tensor own;
    void* p;
    size_t size;
    Scratch(const Tensor& like, const char* kind, cudaStream_t st, size_t bytes) {
        const int64_t want = (int64_t)(bytes > 256 ? bytes : 256);
        if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
            own = fresh(like, {want}, at::kByte);
        } else {
            PyObject* key = Py_BuildValue("(isK)", (int)like.get_device(), kind, (unsigned long long)reinterpret_cast<uintptr_t>(st));
            if (!key) throw Raised();
            PyObject* had = PyDict_GetItemWithError(g_scratch, key);
            if (had && THPVariable_Check(had) && (size_t)THPVariable_Unpack(had).numel() >= bytes) {
                Py_DECREF(key);
                own = THPVariable_Unpack(had);
            } else {
                own = fresh(like, {want}, at::kByte);
                PyObject* o = THPVariable_Wrap(own);
                const bool kept = o && PyDict_SetItem(g_scratch, key, o) == 0;
                Py_DECREF(key);
                Py_XDECREF(o);
                if (!kept) throw Raised();
            }
        }
        p = own.data_ptr();
        size = (size_t)own.numel();
    }
};

// ------------------------------------------------------------------ state space scan and step

struct SsmIn {
    const Tensor *x, *dt, *b, *c;
    int dev;
    int64_t H, N, P;
    kda_ssm_dims dims;
    const float *a_log, *dt_bias, *d_skip;
};

SsmIn ssm_in(PyObject* const* o, int lead) {
    SsmIn s;
    s.x = &leading("x", o[0], lead + 2);
    s.dt = &tensor("dt_raw", o[1]);
    s.b = &tensor("b", o[2]);
    s.c = &tensor("c", o[3]);
    s.dev = (int)s.x->get_device();
    const kda_dtype code = dtype_code(*s.x);
    const IntArrayRef xs = s.x->sizes(), bs = s.b->sizes();
    if ((int)bs.size() != lead + 2 || bs.slice(0, lead) != xs.slice(0, lead) || s.c->sizes() != bs ||
        s.dt->sizes() != xs.slice(0, lead + 1))
        refuse("x must be [..., H, P], b and c [..., G, N] and dt_raw [..., H] over the same tokens");
    const ScalarType type = s.x->scalar_type();
    if (s.b->scalar_type() != type || s.c->scalar_type() != type || s.dt->scalar_type() != type)
        refuse("x, b, c and dt_raw must have one dtype");
    on_device("b", *s.b, s.dev);
    on_device("c", *s.c, s.dev);
    on_device("dt_raw", *s.dt, s.dev);
    const int64_t G = bs[lead];
    s.H = xs[lead];
    s.P = xs[lead + 1];
    s.N = bs[lead + 1];
    if (G < 1 || s.H % G) refuse("heads (" + std::to_string(s.H) + ") must be a multiple of the groups of b and c (" + std::to_string(G) + ")");
    memset(&s.dims, 0, sizeof(s.dims));
    s.dims.B = as_int("B", xs[0]);
    s.dims.T = lead == 2 ? as_int("T", xs[1]) : 1;
    s.dims.H = as_int("H", s.H);
    s.dims.G = as_int("G", G);
    s.dims.N = as_int("N", s.N);
    s.dims.P = as_int("P", s.P);
    s.dims.dtype = code;
    s.dims.x_stride = token_stride("x", *s.x, lead);
    s.dims.b_stride = token_stride("b", *s.b, lead);
    s.dims.c_stride = token_stride("c", *s.c, lead);
    s.dims.dt_stride = token_stride("dt_raw", *s.dt, lead);
    s.a_log = need_f("a_log", o[4], {s.H}, s.dev);
    s.dt_bias = need_f("dt_bias", o[5], {s.H}, s.dev);
    s.d_skip = need_f("d_skip", o[6], {s.H}, s.dev);
    return s;
}

// The scan's workspace by its dimensions (it takes a microsecond of schedules).
size_t ssm_workspace(const kda_ssm_dims& d) {
    struct Entry { kda_ssm_dims d; size_t bytes; };
    static Entry seen[64];
    uint64_t h = 0;
    int32_t w[sizeof(d) / 4];
    memcpy(w, &d, sizeof(w));
    for (int32_t v : w) h = (h ^ (uint32_t)v) * 0x9e3779b97f4a7c15ull;
    Entry& e = seen[h >> 58];
    if (!e.bytes || memcmp(&e.d, &d, sizeof(d))) {
        e.d = d;
        e.bytes = kda_ssm_fwd_workspace_size(&d);
    }
    return e.bytes;
}

// (x, dt_raw, b, c, a_log, dt_bias, d_skip, cu_seqlens, host offsets' address, initial_state, output_final_state, out,
// final_state)
PyObject* ssm_scan(PyObject* const* o) {
    SsmIn s = ssm_in(o, 2);
    int64_t rows = s.dims.B;
    const int32_t* cu = nullptr;
    if (o[7] != Py_None) {
        rows = documents(o[7]);
        cu = need_i("cu_seqlens", o[7], {rows + 1}, s.dev);
        s.dims.num_seqs = (int)rows;
    }
    const int64_t state[4] = {rows, s.H, s.N, s.P};
    const float* s0 = need_f("initial_state", o[9], state, s.dev);
    const cudaStream_t st = current_stream(s.dev);
    const Result out("out", o[11], *s.x, s.x->sizes(), s.x->scalar_type());
    const int wants = PyObject_IsTrue(o[10]);
    if (wants < 0) throw Raised();
    PyObject* last = Py_None;
    void* pf = nullptr;
    Tensor own;
    if (wants) {
        const Result f("final_state", o[12], *s.x, state, at::kFloat);
        own = f.own;
        last = f.given;
        pf = f.p;
    }
    const Scratch ws(*s.x, "ssm", st, ssm_workspace(s.dims));
    check(kda_ssm_fwd(&s.dims, s.x->data_ptr(), s.dt->data_ptr(), s.b->data_ptr(), s.c->data_ptr(), s.a_log, s.dt_bias,
                      s.d_skip, cu, host_copy(o[8]), s0, out.p, static_cast<float*>(pf), ws.p, ws.size, st), "kda_ssm_fwd");
    return pair(out.object(), last ? Py_NewRef(last) : THPVariable_Wrap(own));
}

// A slot pool [slots, *cell] and where it is written.
struct Pool {
    int n;
    const int32_t* slots;
    void *in, *out;
    PyObject* written;
    Pool(const char* name, PyObject* pool, PyObject* slot, PyObject* pool_out, int64_t B, std::initializer_list<int64_t> cell,
         ScalarType type, int dev) {
        const Tensor& t = tensor(name, pool);
        int64_t shape[4] = {t.dim() ? t.size(0) : 0};
        size_t k = 1;
        for (int64_t c : cell) shape[k++] = c;
        written = pool_out == Py_None ? pool : pool_out;
        slots = need_i("slots", slot, {B}, dev);
        n = as_int("slots", shape[0]);
        in = need(name, pool, type, IntArrayRef(shape, k), dev);
        out = need((std::string(name) + "_out").c_str(), written, type, IntArrayRef(shape, k), dev);
    }
};

// (x, dt_raw, b, c, a_log, dt_bias, d_skip, state, slots, state_out, out)
PyObject* ssm_step(PyObject* const* o) {
    const SsmIn s = ssm_in(o, 1);
    const Pool pool("state", o[7], o[8], o[9], s.dims.B, {s.H, s.N, s.P}, at::kFloat, s.dev);
    const Result out("out", o[10], *s.x, s.x->sizes(), s.x->scalar_type());
    check(kda_ssm_step(&s.dims, s.x->data_ptr(), s.dt->data_ptr(), s.b->data_ptr(), s.c->data_ptr(), s.a_log, s.dt_bias,
                       s.d_skip, pool.slots, pool.n, static_cast<const float*>(pool.in), static_cast<float*>(pool.out), out.p,
                       current_stream(s.dev)), "kda_ssm_step");
    return pair(out.object(), Py_NewRef(pool.written));
}

// ------------------------------------------------------------------ the delta rule's step

// (q, k, v, g_raw, beta_raw, a_log, dt_bias, scale, lower_bound, gate code, state, slots, state_out, out)
PyObject* decode_step(PyObject* const* o) {
    const Tensor &q = leading("q", o[0], 3), &v = tensor("v", o[2]);
    if (v.dim() != 3) refuse("v must be [B, H, V]");
    const int dev = (int)q.get_device();
    const int64_t B = q.size(0), Hk = q.size(1), K = q.size(2), H = v.size(1), V = v.size(2);
    kda_dims d;
    memset(&d, 0, sizeof(d));
    d.dtype = dtype_code(q);
    d.B = as_int("B", B); d.T = 1; d.H = as_int("H", H); d.K = as_int("K", K); d.V = as_int("V", V); d.Hk = as_int("Hk", Hk);
    d.gate = (kda_gate)integer("gate", o[9]);
    const ScalarType type = q.scalar_type();
    const int64_t key[3] = {B, Hk, K}, value[3] = {B, H, V}, gates[3] = {B, H, K};
    const void *pq = need("q", o[0], type, key, dev), *pk = need("k", o[1], type, key, dev), *pv = need("v", o[2], type, value, dev);
    const void *pg = need("g_raw", o[3], type, gates, dev), *pb = need("beta_raw", o[4], type, {B, H}, dev);
    const float *al = need_f("a_log", o[5], {H}, dev), *db = need_f("dt_bias", o[6], {H * K}, dev);
    const Pool pool("state", o[10], o[11], o[12], B, {H, K, V}, at::kFloat, dev);
    const Result out("out", o[13], v, value, type);
    check(kda_decode_step(&d, pq, pk, pv, pg, pb, al, db, (float)number(o[7]), (float)number(o[8]), pool.slots, pool.n,
                          static_cast<const float*>(pool.in), static_cast<float*>(pool.out), out.p, current_stream(dev)),
          "kda_decode_step");
    return pair(out.object(), Py_NewRef(pool.written));
}

// ------------------------------------------------------------------ short convolution

struct ConvIn {
    const Tensor* x;
    int dev, W;
    int64_t C;
    kda_dtype code;
    const float *weight, *bias;
};
ConvIn conv_in(PyObject* const* o, int dims) {
    ConvIn c;
    c.x = &leading("x", o[0], dims);
    c.dev = (int)c.x->get_device();
    c.code = dtype_code(*c.x);
    c.C = c.x->size(dims - 1);
    const Tensor& w = tensor("weight", o[1]);
    const int64_t W = w.dim() ? w.size(-1) : 0;
    c.W = as_int("W", W);
    c.weight = w.dim() == 3 ? need_f("weight", o[1], {c.C, 1, W}, c.dev) : need_f("weight", o[1], {c.C, W}, c.dev);
    c.bias = need_f("bias", o[2], {c.C}, c.dev);
    return c;
}

// (x, weight, bias, cu_seqlens, host offsets' address, initial_history, out, final_history)
PyObject* short_conv_prompt(PyObject* const* o) {
    const ConvIn c = conv_in(o, 3);
    const int64_t B = c.x->size(0), T = c.x->size(1);
    int64_t rows = B, n = 0;
    const int32_t* cu = nullptr;
    if (o[3] != Py_None) {
        rows = n = documents(o[3]);
        cu = need_i("cu_seqlens", o[3], {rows + 1}, c.dev);
    }
    const ScalarType type = c.x->scalar_type();
    const int64_t hist[3] = {rows, c.W - 1, c.C};
    const void* h0 = need("initial_history", o[5], type, hist, c.dev);
    const Result out("out", o[6], *c.x, c.x->sizes(), type), last("final_history", o[7], *c.x, hist, type);
    check(kda_short_conv_prompt(as_int("B", B), as_int("T", T), as_int("C", c.C), c.W, c.code, c.x->data_ptr(),
                                token_stride("x", *c.x, 2), c.weight, c.bias, cu, host_copy(o[4]), (int)n, h0,
                                out.p, last.p, current_stream(c.dev)), "kda_short_conv_prompt");
    return pair(out.object(), last.object());
}

// (x, weight, bias, history, slots, history_out, out)
PyObject* short_conv_step(PyObject* const* o) {
    const ConvIn c = conv_in(o, 2);
    const int64_t B = c.x->size(0);
    const ScalarType type = c.x->scalar_type();
    const Pool pool("history", o[3], o[4], o[5], B, {c.W - 1, c.C}, type, c.dev);
    const Result out("out", o[6], *c.x, c.x->sizes(), type);
    check(kda_short_conv_step(as_int("B", B), as_int("C", c.C), c.W, c.code, c.x->data_ptr(), token_stride("x", *c.x, 1), c.weight,
                              c.bias, pool.slots, pool.n, pool.in, pool.out, out.p, current_stream(c.dev)), "kda_short_conv_step");
    return pair(out.object(), Py_NewRef(pool.written));
}

// ------------------------------------------------------------------ pages

// A pool [layers, pages, ...].
struct Layers {
    int64_t layers, pages, page, stride;      // page, stride: bytes of a page, and from layer to layer
};
Layers pool_layers(const char* name, const Tensor& t) {
    const IntArrayRef size = t.sizes(), stride = t.strides();
    if (t.dim() < 2 || t.numel() == 0) refuse(std::string(name) + " must be [layers, pages, ...]");
    int64_t want = 1;
    for (int k = (int)t.dim() - 1; k > 0; --k) {
        if (stride[k] != want && size[k] > 1) refuse(std::string(name) + ": the pages of a layer must be contiguous");
        want *= size[k];
    }
    const int64_t es = (int64_t)t.element_size();
    return {size[0], size[1], want / size[1] * es, stride[0] * es};
}

struct Cache {
    const Tensor* table;
    int dev;
    kda_pages_dims d;
    int32_t *t, *l, *r, *t_out, *l_out, *r_out;
    uint8_t* pool;
};
// pool and lengths may be None.
Cache cache_in(PyObject* pool, PyObject* table, PyObject* lengths, PyObject* refs, PyObject* table_out, PyObject* lengths_out,
               PyObject* refs_out, int64_t page_tokens) {
    Cache c;
    c.table = &tensor("table", table);
    if (!c.table->is_cuda() || c.table->dim() != 2) refuse("table must be a CUDA tensor [sequences, pages of a row]");
    c.dev = (int)c.table->get_device();
    const IntArrayRef shape = c.table->sizes();
    const int64_t pages = tensor("refs", refs).numel();
    c.t = need_i("table", table, shape, c.dev);
    c.l = need_i("lengths", lengths, {shape[0]}, c.dev);
    c.r = need_i("refs", refs, {pages}, c.dev);
    c.t_out = table_out == Py_None ? c.t : need_i("table_out", table_out, shape, c.dev);
    c.l_out = lengths_out == Py_None ? c.l : need_i("lengths_out", lengths_out, {shape[0]}, c.dev);
    c.r_out = refs_out == Py_None ? c.r : need_i("refs_out", refs_out, {pages}, c.dev);
    memset(&c.d, 0, sizeof(c.d));
    Layers p = {1, pages, 1, 0};
    c.pool = nullptr;
    if (pool != Py_None) {
        const Tensor& t = tensor("pool", pool);
        p = pool_layers("pool", t);
        on_device("pool", t, c.dev);
        if (p.pages != pages) refuse("refs must hold one count per page (" + std::to_string(p.pages) + "), got " + std::to_string(pages));
        c.pool = static_cast<uint8_t*>(t.data_ptr());
    }
    c.d.layers = as_int("layers", p.layers);
    c.d.num_pages = as_int("pages", pages);
    c.d.num_seqs = as_int("sequences", shape[0]);
    c.d.max_pages = as_int("pages of a row", shape[1]);
    c.d.page_tokens = (int)page_tokens;
    c.d.page_bytes = p.page;
    c.d.layer_stride = p.stride;
    return c;
}

// (pool, src, dst, src_pool)
PyObject* pages_copy(PyObject* const* o) {
    const Tensor &to = tensor("pool", o[0]), &from = o[3] == Py_None ? to : tensor("src_pool", o[3]);
    if (!to.is_cuda() || !from.is_cuda() || to.get_device() != from.get_device()) refuse("both pools must be on one CUDA device");
    const int dev = (int)to.get_device();
    const Layers a = pool_layers("pool", to), b = pool_layers("src_pool", from);
    if (a.layers != b.layers || a.page != b.page) refuse("both pools must have the same layers and page size");
    const int64_t n = tensor("src", o[1]).numel();
    const int32_t *src = need_i("src", o[1], {n}, dev), *dst = need_i("dst", o[2], {n}, dev);
    check(kda_pages_copy(as_int("layers", a.layers), a.page, to.data_ptr(), a.stride, as_int("pages", a.pages), from.data_ptr(),
                         b.stride, as_int("pages", b.pages), src, dst, as_int("requests", n), current_stream(dev)), "kda_pages_copy");
    return Py_NewRef(o[0]);
}

// (pool, table, lengths, refs, parents, children, page_tokens, table_out, lengths_out, refs_out, ok)
PyObject* pages_fork(PyObject* const* o) {
    const int64_t n = tensor("parents", o[4]).numel();
    tensor("pool", o[0]);
    const Cache c = cache_in(o[0], o[1], o[2], o[3], o[7], o[8], o[9], integer("page_tokens", o[6]));
    const int32_t *pa = need_i("parents", o[4], {n}, c.dev), *ch = need_i("children", o[5], {n}, c.dev);
    const cudaStream_t st = current_stream(c.dev);
    const Result ok("ok", o[10], *c.table, {n}, at::kInt);
    const Scratch ws(*c.table, "pages", st, kda_pages_workspace_size(&c.d, as_int("requests", n)));
    check(kda_pages_fork(&c.d, c.pool, c.t, c.l, c.r, pa, ch, (int)n, c.t_out, c.l_out, c.r_out, static_cast<int32_t*>(ok.p), ws.p, ws.size,
                         st), "kda_pages_fork");
    return ok.object();
}

// (table, lengths, refs, seqs, new_lengths, page_tokens, table_out, lengths_out, refs_out, ok)
PyObject* pages_extend(PyObject* const* o) {
    const int64_t n = tensor("seqs", o[3]).numel();
    const Cache c = cache_in(Py_None, o[0], o[1], o[2], o[6], o[7], o[8], integer("page_tokens", o[5]));
    const int32_t *seqs = need_i("seqs", o[3], {n}, c.dev), *lens = need_i("new_lengths", o[4], {n}, c.dev);
    const cudaStream_t st = current_stream(c.dev);
    const Result ok("ok", o[9], *c.table, {n}, at::kInt);
    const Scratch ws(*c.table, "pages", st, kda_pages_workspace_size(&c.d, as_int("requests", n)));
    check(kda_pages_extend(&c.d, c.t, c.l, c.r, seqs, lens, (int)n, c.t_out, c.l_out, c.r_out, static_cast<int32_t*>(ok.p), ws.p, ws.size,
                           st), "kda_pages_extend");
    return ok.object();
}

// (table, lengths, refs, seqs, table_out, lengths_out, refs_out)
PyObject* pages_free(PyObject* const* o) {
    const int64_t n = tensor("seqs", o[3]).numel();
    const Cache c = cache_in(Py_None, o[0], o[1], o[2], o[4], o[5], o[6], 1);
    const int32_t* seqs = need_i("seqs", o[3], {n}, c.dev);
    check(kda_pages_free(&c.d, c.t, c.l, c.r, seqs, as_int("requests", n), c.t_out, c.l_out, c.r_out, current_stream(c.dev)),
          "kda_pages_free");
    return Py_NewRef(Py_None);
}

// (pool, table, refs, table_out, refs_out, page_map)
PyObject* pages_compact(PyObject* const* o) {
    tensor("pool", o[0]);
    const Cache c = cache_in(o[0], o[1], Py_None, o[2], o[3], Py_None, o[4], 1);
    const cudaStream_t st = current_stream(c.dev);
    const Result map("page_map", o[5], *c.table, {(int64_t)c.d.num_pages}, at::kInt);
    const Scratch ws(*c.table, "pages", st, kda_pages_workspace_size(&c.d, 0));
    check(kda_pages_compact(&c.d, c.pool, c.t, c.r, c.t_out, c.r_out, static_cast<int32_t*>(map.p), ws.p, ws.size, st),
          "kda_pages_compact");
    return map.object();
}

// (t, lead)
PyObject* token_stride_of(PyObject* const* o) { return PyLong_FromLongLong(token_stride("x", tensor("x", o[0]), (int)integer("lead", o[1]))); }

// ------------------------------------------------------------------ module

// The device of a call: its first CUDA tensor's (the checks hold the others to it); -1 without one.
int device_of(PyObject* const* args, Py_ssize_t n) {
    for (Py_ssize_t i = 0; i < n; ++i)
        if (THPVariable_Check(args[i]) && THPVariable_Unpack(args[i]).is_cuda()) return (int)THPVariable_Unpack(args[i]).get_device();
    return -1;
}

// Launches, function attributes and the status word's address are the current device's: it is the tensors' for the call.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    c10::cuda::OptionalCUDAGuard guard;
    try {
        const int dev = device_of(args, n);
        if (dev >= 0) guard.set_index((c10::DeviceIndex)dev);
        return F(args);
    } catch (const Refused& e) {
        PyErr_SetString(e.type, e.what.c_str());
        return nullptr;
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// device_of(...): the device that a call with these arguments runs on, -1: none
PyObject* device_of_args(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    return PyLong_FromLong(device_of(args, n));
    END_HANDLE_TH_ERRORS
}

// setup(check, workspaces)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 2 || !PyCallable_Check(args[0]) || !PyDict_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "setup(check, workspaces)");
        return nullptr;
    }
    Py_XSETREF(g_check, Py_NewRef(args[0]));
    Py_XSETREF(g_scratch, Py_NewRef(args[1]));
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<ssm_scan, 13>("ssm_scan"), method<ssm_step, 11>("ssm_step"), method<decode_step, 14>("decode_step"),
    method<short_conv_prompt, 8>("short_conv_prompt"), method<short_conv_step, 7>("short_conv_step"),
    method<pages_copy, 4>("pages_copy"), method<pages_fork, 11>("pages_fork"), method<pages_extend, 10>("pages_extend"),
    method<pages_free, 7>("pages_free"), method<pages_compact, 6>("pages_compact"),
    method<token_stride_of, 2>("token_stride"),
    {"device_of", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&device_of_args)), METH_FASTCALL, nullptr},
    {"setup", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&setup)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module); }
