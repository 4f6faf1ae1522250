// torch_binding.cpp -- native half of the Python binding of the softmax-attention layer.
//
// Argument checks and marshalling only, as the ctypes half does for the other entry points:
// tensors in, one call of the C ABI (resolved from libmuir.so at load), tensors out.  It is
// native because these operators are called once a token and layer: through ctypes a call
// took 12 to 20 us of the host, where the kernels take 2 to 8.
#include <ATen/cuda/CUDAContext.h>
#include <c10/cuda/CUDAGuard.h>
#include <dlfcn.h>
#include <torch/extension.h>

#include <cmath>
#include <optional>
#include <string>
#include <vector>

#include "../../include/muir.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

struct Abi {
    decltype(&muir_rotary) rotary;
    decltype(&muir_attn_fwd) attn_fwd;
    decltype(&muir_attn_fwd_varlen) attn_fwd_varlen;
    decltype(&muir_attn_bwd_workspace) attn_bwd_workspace;
    decltype(&muir_attn_bwd) attn_bwd;
    decltype(&muir_attn_bwd_varlen) attn_bwd_varlen;
    decltype(&muir_kv_append) kv_append;
    decltype(&muir_attn_step_workspace) attn_step_workspace;
    decltype(&muir_attn_step) attn_step;
} abi;
PyObject* error_class = nullptr;  // MuirError(function, code)

template <class F>
void resolve(void* lib, const char* name, F& f) {
    f = reinterpret_cast<F>(dlsym(lib, name));
    if (!f) throw py::import_error(std::string("libmuir.so lacks ") + name);
}

void load(const std::string& path, py::object error) {
    void* lib = dlopen(path.c_str(), RTLD_NOW | RTLD_LOCAL);
    if (!lib) throw py::import_error(dlerror());
    resolve(lib, "muir_rotary", abi.rotary);
    resolve(lib, "muir_attn_fwd", abi.attn_fwd);
    resolve(lib, "muir_attn_fwd_varlen", abi.attn_fwd_varlen);
    resolve(lib, "muir_attn_bwd_workspace", abi.attn_bwd_workspace);
    resolve(lib, "muir_attn_bwd", abi.attn_bwd);
    resolve(lib, "muir_attn_bwd_varlen", abi.attn_bwd_varlen);
    resolve(lib, "muir_kv_append", abi.kv_append);
    resolve(lib, "muir_attn_step_workspace", abi.attn_step_workspace);
    resolve(lib, "muir_attn_step", abi.attn_step);
    error_class = error.release().ptr();
}

void check(const char* fn, muir_status st) {
    if (st == MUIR_OK) return;
    py::object e = py::reinterpret_borrow<py::object>(error_class)(fn, (int)st);
    PyErr_SetObject(error_class, e.ptr());
    throw py::error_already_set();
}

[[noreturn]] void bad(const std::string& what) { throw py::value_error(what); }

muir_dtype dtype_of(const Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return MUIR_BF16;
    if (t.scalar_type() == at::kFloat) return MUIR_FP32;
    throw py::type_error(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) +
                         " (bfloat16 or float32)");
}

void on(const Tensor& t, const char* name, c10::Device dev) {
    if (!t.is_cuda()) bad("libmuir takes CUDA tensors only");
    if (t.device() != dev) bad(std::string(name) + " is on " + t.device().str() + ", not on " + dev.str());
}

// A [B, T, H, d] tensor whose heads are dense within a token and whose tokens are evenly
// spaced (a part of a packed projection qualifies): its address, and the elements between
// tokens (0 = dense).
struct Rows {
    void* p;
    long long ld;
};
Rows rows(const Tensor& t, const char* name, c10::Device dev) {
    if (t.dim() != 4) bad(std::string(name) + " must be [B, T, H, d]");
    on(t, name, dev);
    if (t.is_contiguous()) return {t.data_ptr(), 0};
    const int64_t B = t.size(0), T = t.size(1), H = t.size(2), d = t.size(3);
    int64_t st = t.stride(1);
    if ((t.stride(3) != 1 && d > 1) || (t.stride(2) != d && H > 1))
        bad(std::string(name) + ": channels and heads of a token must be dense");
    if (T == 1) st = B > 1 ? t.stride(0) : H * d;
    else if (B > 1 && t.stride(0) != T * st) bad(std::string(name) + ": tokens must be evenly spaced");
    if (st < H * d) bad(std::string(name) + ": tokens must not overlap (expanded tensors are not taken)");
    return {t.data_ptr(), st};
}

// A contiguous tensor of exactly this shape, type and device.
void* same(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    if (t.sizes() != shape || t.scalar_type() != type || t.device() != dev || !t.is_contiguous()) {
        std::string s = std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape (";
        for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
        bad(s + ") on " + dev.str());
    }
    return t.data_ptr();
}

int as_int(int64_t v, const char* name) {
    if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + " is out of range");
    return (int)v;
}

// The current stream of the tensors' device, that device current while this lives.
struct Call {
    c10::cuda::OptionalCUDAGuard guard;
    void* stream;
    explicit Call(c10::Device dev) {
        if (dev.index() != c10::cuda::current_device()) guard.set_device(dev);
        stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }
};

Tensor workspace(size_t bytes, const OptTensor& ws, c10::Device dev) {
    if (ws && (size_t)ws->numel() * ws->element_size() >= bytes) {
        if (ws->device() != dev || !ws->is_contiguous()) bad("ws must be a contiguous tensor on the call's device");
        return *ws;
    }
    return at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(dev));
}

// ------------------------------------------------------------------ rotary

bool tracked(const Tensor& t) { return t.requires_grad() && at::GradMode::is_enabled(); }
bool tracked(const OptTensor& t) { return t && tracked(*t); }

// A tensor of the caller's was written: autograd's check of what it saved has to see it.
void written(const OptTensor& t) {
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

py::object rotary(const Tensor& q, const OptTensor& k, const OptTensor& positions, const OptTensor& inv_freq,
                  bool interleaved, double mscale, bool inverse, const OptTensor& q_out, const OptTensor& k_out) {
    if (!inv_freq) bad("inv_freq is required (rotary_frequencies makes it)");
    if (tracked(q) || tracked(k) || tracked(q_out) || tracked(k_out))
        bad("rotary records no gradient and would cut or falsify it: call MuirRotaryFunction.apply, or rotary "
            "under torch.no_grad()");
    const muir_dtype dt = dtype_of(q);
    const c10::Device dev = q.device();
    const Rows rq = rows(q, "q", dev);
    const int64_t B = q.size(0), T = q.size(1), Hq = q.size(2), d = q.size(3);
    if (q_out && (q_out->sizes() != q.sizes() || q_out->scalar_type() != q.scalar_type()))
        bad("q_out must have q's shape and dtype");
    if (k_out && !k) bad("k_out without k");
    if (k && (k->dim() != 4 || k->size(0) != B || k->size(1) != T || k->size(3) != d ||
              k->scalar_type() != q.scalar_type()))
        bad("k must have q's batch, tokens, channels and dtype");
    if (k_out && (k_out->sizes() != k->sizes() || k_out->scalar_type() != q.scalar_type()))
        bad("k_out must have k's shape and dtype");
    const Rows rk = k ? rows(*k, "k", dev) : Rows{nullptr, 0};
    const void* pos = positions ? same(*positions, "positions", {B, T}, at::kInt, dev) : nullptr;
    const int64_t half = inv_freq->numel();
    const void* freq = same(*inv_freq, "inv_freq", {half}, at::kDouble, dev);
    Call c(dev);
    const Tensor oq = q_out ? *q_out : at::empty(q.sizes(), q.options());
    const Tensor ok = k ? (k_out ? *k_out : at::empty(k->sizes(), k->options())) : Tensor();
    const Rows wq = rows(oq, "q_out", dev), wk = k ? rows(ok, "k_out", dev) : Rows{nullptr, 0};
    check("muir_rotary",
          abi.rotary(as_int(B, "B"), as_int(T, "T"), as_int(Hq, "Hq"), k ? as_int(k->size(2), "Hk") : 0,
                     as_int(d, "d"), as_int(2 * half, "rot"), dt, rq.p, rq.ld, rk.p, rk.ld,
                     static_cast<const int*>(pos), static_cast<const double*>(freq), (float)mscale, interleaved,
                     inverse, wq.p, wq.ld, wk.p, wk.ld, c.stream));
    written(q_out);
    written(k_out);
    if (!k) return py::cast(oq);
    return py::make_tuple(oq, ok);
}

// ------------------------------------------------------------------ attention

struct Attn {
    muir_attn_shape s;
    Rows q, k, v;
    c10::Device dev;
};
Attn attn_args(const Tensor& q, const Tensor& k, const Tensor& v, bool causal, int64_t window,
               const std::optional<double>& scale) {
    if (q.dim() != 4 || k.dim() != 4) bad("q, k and v must be [B, T, H, d]");
    if (k.size(0) != q.size(0) || k.size(3) != q.size(3) || v.sizes() != k.sizes())
        bad("q, k and v must agree in batch and channels, k and v in shape");
    if (q.scalar_type() != at::kBFloat16 || k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16)
        throw py::type_error("attention takes bfloat16 tensors");
    const c10::Device dev = q.device();
    Attn a{{}, rows(q, "q", dev), rows(k, "k", dev), rows(v, "v", dev), dev};
    const double d = (double)q.size(3);
    a.s = {as_int(q.size(0), "B"), as_int(q.size(1), "Tq"), as_int(k.size(1), "Tk"), as_int(q.size(2), "Hq"),
           as_int(k.size(2), "Hk"), as_int(q.size(3), "d"), causal ? 1 : 0, as_int(window, "window"),
           (float)(scale ? *scale : 1.0 / std::sqrt(d)), a.q.ld, a.k.ld, a.v.ld};
    return a;
}

// Host offsets from a CPU tensor or a sequence of whole numbers.
std::vector<long long> offsets(const py::object& cu) {
    std::vector<long long> v;
    if (THPVariable_Check(cu.ptr())) {
        const Tensor t = THPVariable_Unpack(cu.ptr()).to(at::kCPU, at::kLong).contiguous();
        v.assign(t.data_ptr<int64_t>(), t.data_ptr<int64_t>() + t.numel());
    } else {
        for (const auto& x : py::reinterpret_borrow<py::sequence>(cu)) v.push_back(x.cast<long long>());
    }
    if (v.empty()) bad("cu_seqlens must have an offset more than sequences");
    return v;
}
struct Packed {
    bool on = false;
    std::vector<long long> q, k;
    const long long* kp() const { return k.empty() ? nullptr : k.data(); }
    int n() const { return (int)q.size() - 1; }
};
Packed packed(const py::object& cu, const py::object& cu_k) {
    Packed p;
    if (cu.is_none()) return p;
    p.on = true;
    p.q = offsets(cu);
    if (!cu_k.is_none()) p.k = offsets(cu_k);
    if (!p.k.empty() && p.k.size() != p.q.size()) bad("cu_seqlens_k must have as many offsets as cu_seqlens");
    return p;
}

py::tuple attn_fwd(const Tensor& q, const Tensor& k, const Tensor& v, const py::object& cu, const py::object& cu_k,
                   bool causal, int64_t window, const std::optional<double>& scale) {
    const Packed pk = packed(cu, cu_k);
    const Attn a = attn_args(q, k, v, causal, window, scale);
    Call c(a.dev);
    const Tensor o = at::empty(q.sizes(), q.options());
    const Tensor lse = at::empty({a.s.B, a.s.Hq, a.s.Tq}, q.options().dtype(at::kFloat));
    float* lp = static_cast<float*>(lse.data_ptr());
    if (pk.on)
        check("muir_attn_fwd_varlen", abi.attn_fwd_varlen(&a.s, pk.n(), pk.q.data(), pk.kp(), a.q.p, a.k.p, a.v.p,
                                                          o.data_ptr(), lp, c.stream));
    else
        check("muir_attn_fwd", abi.attn_fwd(&a.s, a.q.p, a.k.p, a.v.p, o.data_ptr(), lp, c.stream));
    return py::make_tuple(o, lse);
}

py::dict attn_bwd(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o, const Tensor& lse,
                  const Tensor& dO, const py::object& cu, const py::object& cu_k, bool causal, int64_t window,
                  const std::optional<double>& scale, const OptTensor& ws) {
    const Packed pk = packed(cu, cu_k);
    const Attn a = attn_args(q, k, v, causal, window, scale);
    const void* op = same(o, "o", q.sizes(), at::kBFloat16, a.dev);
    const void* gp = same(dO, "dO", q.sizes(), at::kBFloat16, a.dev);
    const float* lp = static_cast<const float*>(same(lse, "lse", {a.s.B, a.s.Hq, a.s.Tq}, at::kFloat, a.dev));
    Call c(a.dev);
    const Tensor dq = at::empty(q.sizes(), q.options()), dk = at::empty(k.sizes(), k.options()),
                 dv = at::empty(k.sizes(), k.options());
    const size_t need = abi.attn_bwd_workspace(&a.s);
    const Tensor w = workspace(need, ws, a.dev);
    const size_t bytes = (size_t)w.numel() * w.element_size();
    if (pk.on)
        check("muir_attn_bwd_varlen",
              abi.attn_bwd_varlen(&a.s, pk.n(), pk.q.data(), pk.kp(), a.q.p, a.k.p, a.v.p, op, lp, gp, dq.data_ptr(),
                                  dk.data_ptr(), dv.data_ptr(), w.data_ptr(), bytes, c.stream));
    else
        check("muir_attn_bwd", abi.attn_bwd(&a.s, a.q.p, a.k.p, a.v.p, op, lp, gp, dq.data_ptr(), dk.data_ptr(),
                                            dv.data_ptr(), w.data_ptr(), bytes, c.stream));
    py::dict g;
    g["dq"] = dq;
    g["dk"] = dk;
    g["dv"] = dv;
    return g;
}

// ------------------------------------------------------------------ 8-bit cache

muir_kv_cache cache_args(const Tensor& kp, const Tensor& vp, const Tensor& ks, const Tensor& vs, const Tensor& table,
                         int64_t B, c10::Device dev) {
    if (kp.dim() != 4) bad("k_pages must be [num_pages, Hk, page, d]");
    if (table.dim() != 2 || table.size(0) != B) bad("page_table must be [B, max_pages]");
    const int64_t num = kp.size(0), Hk = kp.size(1);
    muir_kv_cache c;
    c.Hk = as_int(Hk, "Hk");
    c.d = as_int(kp.size(3), "d");
    c.page = as_int(kp.size(2), "page");
    c.num_pages = as_int(num, "num_pages");
    c.max_pages = as_int(table.size(1), "max_pages");
    c.k_pages = same(kp, "k_pages", kp.sizes(), at::kFloat8_e4m3fn, dev);
    c.v_pages = same(vp, "v_pages", kp.sizes(), at::kFloat8_e4m3fn, dev);
    c.k_scale = static_cast<float*>(same(ks, "k_scale", {num, Hk}, at::kFloat, dev));
    c.v_scale = static_cast<float*>(same(vs, "v_scale", {num, Hk}, at::kFloat, dev));
    c.table = static_cast<const int*>(same(table, "page_table", table.sizes(), at::kInt, dev));
    return c;
}

void kv_append(const Tensor& k, const Tensor& v, const Tensor& kp, const Tensor& vp, const Tensor& ks,
               const Tensor& vs, const Tensor& table, const Tensor& start, const OptTensor& count) {
    const muir_dtype dt = dtype_of(k);
    const c10::Device dev = k.device();
    const Rows rk = rows(k, "k", dev);
    if (v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type()) bad("v must have k's shape and dtype");
    const Rows rv = rows(v, "v", dev);
    if (kp.dim() == 4 && (kp.size(1) != k.size(2) || kp.size(3) != k.size(3)))
        bad("the cache's heads and channels must be k's");
    const int64_t B = k.size(0);
    const muir_kv_cache c = cache_args(kp, vp, ks, vs, table, B, dev);
    const void* st = same(start, "start", {B}, at::kInt, dev);
    const void* ct = count ? same(*count, "count", {B}, at::kInt, dev) : nullptr;
    Call call(dev);
    check("muir_kv_append",
          abi.kv_append(as_int(B, "B"), as_int(k.size(1), "T"), dt, rk.p, rk.ld, rv.p, rv.ld, &c,
                        static_cast<const int*>(st), static_cast<const int*>(ct), call.stream));
}

Tensor attn_step(const Tensor& q, const Tensor& kp, const Tensor& vp, const Tensor& ks, const Tensor& vs,
                 const Tensor& table, const Tensor& lens, const std::optional<double>& scale, int64_t window,
                 const OptTensor& out, const OptTensor& ws) {
    if (q.dim() != 3) bad("q must be [B, Hq, d]");
    const c10::Device dev = q.device();
    on(q, "q", dev);
    const int64_t B = q.size(0), Hq = q.size(1), d = q.size(2);
    if (kp.dim() == 4 && kp.size(3) != d) bad("the cache's channels must be q's");
    const void* qp = same(q, "q", q.sizes(), at::kBFloat16, dev);
    const muir_kv_cache c = cache_args(kp, vp, ks, vs, table, B, dev);
    const void* ln = same(lens, "lens", {B}, at::kInt, dev);
    Call call(dev);
    const Tensor o = out ? *out : at::empty(q.sizes(), q.options());
    void* op = same(o, "o", q.sizes(), at::kBFloat16, dev);
    const size_t need = abi.attn_step_workspace(as_int(B, "B"), as_int(Hq, "Hq"), &c);
    Tensor w;
    if (need > 0) w = workspace(need, ws, dev);
    check("muir_attn_step",
          abi.attn_step((int)B, (int)Hq, &c, qp, static_cast<const int*>(ln),
                        (float)(scale ? *scale : 1.0 / std::sqrt((double)d)), as_int(window, "window"), op,
                        need ? w.data_ptr() : nullptr, need ? (size_t)w.numel() * w.element_size() : 0, call.stream));
    return o;
}

}  // namespace

PYBIND11_MODULE(_attn, m) {
    m.def("load", &load);
    m.def("rotary", &rotary);
    m.def("attn_fwd", &attn_fwd);
    m.def("attn_bwd", &attn_bwd);
    m.def("kv_append", &kv_append);
    m.def("attn_step", &attn_step);
}
