// api_attn.cu -- the extern "C" entry points of the softmax-attention layer: host-side
// argument checks, workspace sizing and dispatch to the CUDA kernels.
#include <math.h>

#include "attn.h"
#include "checks.h"
#include "kernels.h"

namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool ok_ints(const int* p) { return p != nullptr && aligned_to(p, 4); }

constexpr float kLog2e = 1.4426950408889634f;
bool ok_scale(float s) { return isfinite(s * kLog2e); }  // as the kernels take it

// Leading dimension of a token-major operand: 0 = dense; else a row's width at least,
// and whole 16-byte vectors.
bool ok_ld(long long ld, long long width, int esize) {
    return ld == 0 || (ld >= width && ld % (16 / esize) == 0 && ld <= (1LL << 40) / 16);
}

muir_status check_attn(const muir_attn_shape* s) {
    if (!s) return MUIR_ERR_INVALID_ARG;
    if (s->B < 0 || s->Tq < 0 || s->Tk < 0 || s->Hq <= 0 || s->Hk <= 0 || s->d <= 0 || s->window < 0)
        return MUIR_ERR_INVALID_ARG;
    if (!(s->scale > 0.f) || !ok_scale(s->scale) || s->Hq % s->Hk) return MUIR_ERR_INVALID_ARG;
    if (s->d != 64 && s->d != 128) return MUIR_ERR_UNSUPPORTED;
    const long long wq = (long long)s->Hq * s->d, wk = (long long)s->Hk * s->d;
    if (!ok_ld(s->q_ld, wq, 2) || !ok_ld(s->k_ld, wk, 2) || !ok_ld(s->v_ld, wk, 2)) return MUIR_ERR_INVALID_ARG;
    // rows are int32 (with room for a tile past the end), blocks of 128 rows and heads a grid
    if ((long long)s->B * s->Tq > 0x7fff0000LL || (long long)s->B * s->Tk > 0x7fff0000LL || s->Hq > 65536)
        return MUIR_ERR_UNSUPPORTED;
    // a query's position less the window, and a key's plus it, stay in int32
    if (s->Tq + 2LL * s->Tk > 0x7fffffffLL) return MUIR_ERR_UNSUPPORTED;
    const long long tq = (s->Tq + 127LL) / 128, tk = (s->Tk + 127LL) / 128;
    if ((s->B * tq + 65536) * s->Hq > 0x7fffffffLL || (s->B * tk + 65536) * s->Hk > 0x7fffffffLL)
        return MUIR_ERR_UNSUPPORTED;
    return MUIR_OK;
}

muir_status check_offsets(const long long* cu, int n, int total) {
    if (cu[0] != 0 || cu[n] != total) return MUIR_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (cu[i + 1] < cu[i]) return MUIR_ERR_INVALID_ARG;
    return MUIR_OK;
}

muir_status check_attn_varlen(const muir_attn_shape* s, int n, const long long* cu_q, const long long* cu_k) {
    muir_status st = check_attn(s);
    if (st != MUIR_OK) return st;
    if (s->B != 1 || n <= 0 || !cu_q) return MUIR_ERR_INVALID_ARG;
    if ((st = check_offsets(cu_q, n, s->Tq)) != MUIR_OK) return st;
    return check_offsets(cu_k ? cu_k : cu_q, n, s->Tk);
}

muir::attn::Problem attn_problem(const muir_attn_shape* s, const void* q, const void* k, const void* v,
                                 int n, const long long* cu_q, const long long* cu_k) {
    muir::attn::Problem p;
    p.Hq = s->Hq; p.Hk = s->Hk; p.d = s->d;
    p.causal = s->causal != 0; p.scale = s->scale;
    p.window = s->window < s->Tk ? s->window : 0;  // one that hides nothing is none
    p.q_ld = s->q_ld ? s->q_ld : (long long)s->Hq * s->d;
    p.k_ld = s->k_ld ? s->k_ld : (long long)s->Hk * s->d;
    p.v_ld = s->v_ld ? s->v_ld : (long long)s->Hk * s->d;
    p.q_rows = (long long)s->B * s->Tq;
    p.k_rows = (long long)s->B * s->Tk;
    // [B][Hq][Tq], or [Hq][Tq] over packed sequences
    p.lse_seq = cu_q ? 1 : s->Hq;
    p.lse_head = s->Tq;
    p.q = q; p.k = k; p.v = v;
    p.n = cu_q ? n : s->B;
    p.Tq = s->Tq; p.Tk = s->Tk;
    p.cu_q = cu_q;
    p.cu_k = cu_k ? cu_k : cu_q;
    return p;
}

// Pointers of tensors without elements may be null.
bool ok_some(const void* p, bool any) { return any ? ok_ptr(p) : true; }

muir_status attn_fwd(const muir_attn_shape* s, int n, const long long* cu_q, const long long* cu_k, const void* q,
                     const void* k, const void* v, void* o, float* lse, void* stream) {
    const bool any_q = s->B > 0 && s->Tq > 0, any_k = s->B > 0 && s->Tk > 0;
    if (!ok_some(q, any_q) || !ok_some(o, any_q) || !ok_some(k, any_k) || !ok_some(v, any_k) ||
        (any_q && (!lse || !aligned_to(lse, 4))))
        return MUIR_ERR_INVALID_ARG;
    const muir_status st = check_device();
    if (st != MUIR_OK) return st;
    return from_cuda(muir::attn::run_fwd(attn_problem(s, q, k, v, n, cu_q, cu_k), o, lse,
                                         static_cast<cudaStream_t>(stream)));
}

muir_status attn_bwd(const muir_attn_shape* s, int n, const long long* cu_q, const long long* cu_k, const void* q,
                     const void* k, const void* v, const void* o, const float* lse, const void* dO, void* dq,
                     void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
    const bool any_q = s->B > 0 && s->Tq > 0, any_k = s->B > 0 && s->Tk > 0;
    if (!ok_some(q, any_q) || !ok_some(o, any_q) || !ok_some(dO, any_q) || !ok_some(dq, any_q) ||
        !ok_some(k, any_k) || !ok_some(v, any_k) || !ok_some(dk, any_k) || !ok_some(dv, any_k) ||
        (any_q && (!lse || !aligned_to(lse, 4))))
        return MUIR_ERR_INVALID_ARG;
    const muir::attn::Problem p = attn_problem(s, q, k, v, n, cu_q, cu_k);
    const size_t need = muir::attn::bwd_ws_bytes(p);
    if (ws_bytes < need || (need > 0 && !ok_ptr(ws))) return MUIR_ERR_WORKSPACE;
    const muir_status st = check_device();
    if (st != MUIR_OK) return st;
    return from_cuda(muir::attn::run_bwd(p, o, lse, dO, dq, dk, dv, ws, static_cast<cudaStream_t>(stream)));
}

muir_status check_cache(const muir_kv_cache* c) {
    if (!c) return MUIR_ERR_INVALID_ARG;
    if (c->Hk <= 0 || c->d <= 0 || c->page <= 0 || c->num_pages <= 0 || c->max_pages <= 0)
        return MUIR_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return MUIR_ERR_UNSUPPORTED;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return MUIR_ERR_UNSUPPORTED;
    // (page, head) blocks are a TMA coordinate; positions are int32
    if ((long long)c->num_pages * c->Hk > 0x7fffffffLL || (long long)c->max_pages * c->page > 0x7fffffffLL ||
        c->Hk > 65535)
        return MUIR_ERR_UNSUPPORTED;
    if (!ok_ptr(c->k_pages) || !ok_ptr(c->v_pages) || !c->k_scale || !c->v_scale ||
        !aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4) || !ok_ints(c->table))
        return MUIR_ERR_INVALID_ARG;
    return MUIR_OK;
}

muir_status check_step(int B, int Hq, const muir_kv_cache* c) {
    const muir_status st = check_cache(c);
    if (st != MUIR_OK) return st;
    if (B <= 0 || Hq <= 0 || Hq % c->Hk) return MUIR_ERR_INVALID_ARG;
    if (B > 65535 || (long long)c->Hk * ((Hq / c->Hk + 15) / 16) > 65535) return MUIR_ERR_UNSUPPORTED;
    return MUIR_OK;
}

}  // namespace

extern "C" {

muir_status muir_rotary(int B, int T, int Hq, int Hk, int d, int rot, muir_dtype dtype,
                        const void* q, long long q_ld, const void* k, long long k_ld,
                        const int* positions, const double* inv_freq, float mscale,
                        int interleaved, int inverse, void* q_out, long long q_out_ld,
                        void* k_out, long long k_out_ld, void* stream) {
    if (B < 0 || T < 0 || Hq <= 0 || Hk < 0 || !ok_dtype(dtype) || !isfinite(mscale)) return MUIR_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return MUIR_ERR_UNSUPPORTED;
    if (rot < 16 || rot > d || rot % 16) return MUIR_ERR_UNSUPPORTED;
    if (Hq > 65536 || Hk > 65536 || (long long)B * T > 0x7fffffffLL) return MUIR_ERR_UNSUPPORTED;
    const int esize = dtype == MUIR_BF16 ? 2 : 4;
    const long long wq = (long long)Hq * d, wk = (long long)Hk * d;
    if (!ok_ld(q_ld, wq, esize) || !ok_ld(q_out_ld, wq, esize) || !ok_ld(k_ld, wk, esize) ||
        !ok_ld(k_out_ld, wk, esize))
        return MUIR_ERR_INVALID_ARG;
    if ((long long)B * T == 0) return MUIR_OK;
    if (!ok_ptr(q) || !ok_ptr(q_out) || !inv_freq || !aligned_to(inv_freq, 8) || !aligned_to(positions, 4))
        return MUIR_ERR_INVALID_ARG;
    if (Hk > 0 ? (!ok_ptr(k) || !ok_ptr(k_out)) : (k || k_out)) return MUIR_ERR_INVALID_ARG;
    muir::RotaryArgs a{};
    a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
    a.q_ld = q_ld ? q_ld : wq;
    a.k_ld = k_ld ? k_ld : wk;
    a.qo_ld = q_out_ld ? q_out_ld : wq;
    a.ko_ld = k_out_ld ? k_out_ld : wk;
    if ((q == q_out && a.q_ld != a.qo_ld) || (Hk > 0 && k == k_out && a.k_ld != a.ko_ld))
        return MUIR_ERR_INVALID_ARG;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.mscale = mscale;
    a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = rot;
    a.inverse = inverse != 0;
    a.tokens = (long long)B * T;
    const muir_status st = check_device();
    if (st != MUIR_OK) return st;
    return from_cuda(muir::launch_rotary(a, dtype == MUIR_BF16, interleaved != 0, static_cast<cudaStream_t>(stream)));
}

muir_status muir_attn_fwd(const muir_attn_shape* s, const void* q, const void* k, const void* v, void* o,
                          float* lse, void* stream) {
    const muir_status st = check_attn(s);
    return st != MUIR_OK ? st : attn_fwd(s, 0, nullptr, nullptr, q, k, v, o, lse, stream);
}

size_t muir_attn_bwd_workspace(const muir_attn_shape* s) {
    if (check_attn(s) != MUIR_OK) return 0;
    return muir::attn::bwd_ws_bytes(attn_problem(s, nullptr, nullptr, nullptr, 0, nullptr, nullptr));
}

muir_status muir_attn_bwd(const muir_attn_shape* s, const void* q, const void* k, const void* v, const void* o,
                          const float* lse, const void* dO, void* dq, void* dk, void* dv, void* ws,
                          size_t ws_bytes, void* stream) {
    const muir_status st = check_attn(s);
    return st != MUIR_OK ? st
                         : attn_bwd(s, 0, nullptr, nullptr, q, k, v, o, lse, dO, dq, dk, dv, ws, ws_bytes, stream);
}

muir_status muir_attn_fwd_varlen(const muir_attn_shape* s, int n, const long long* cu_q, const long long* cu_k,
                                 const void* q, const void* k, const void* v, void* o, float* lse, void* stream) {
    const muir_status st = check_attn_varlen(s, n, cu_q, cu_k);
    return st != MUIR_OK ? st : attn_fwd(s, n, cu_q, cu_k, q, k, v, o, lse, stream);
}

muir_status muir_attn_bwd_varlen(const muir_attn_shape* s, int n, const long long* cu_q, const long long* cu_k,
                                 const void* q, const void* k, const void* v, const void* o, const float* lse,
                                 const void* dO, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                 void* stream) {
    const muir_status st = check_attn_varlen(s, n, cu_q, cu_k);
    return st != MUIR_OK ? st
                         : attn_bwd(s, n, cu_q, cu_k, q, k, v, o, lse, dO, dq, dk, dv, ws, ws_bytes, stream);
}

muir_status muir_kv_append(int B, int T, muir_dtype dtype, const void* k, long long k_ld,
                           const void* v, long long v_ld, const muir_kv_cache* c,
                           const int* start, const int* count, void* stream) {
    muir_status st = check_cache(c);
    if (st != MUIR_OK) return st;
    if (B < 0 || T < 0 || !ok_dtype(dtype)) return MUIR_ERR_INVALID_ARG;
    if (B > 32767) return MUIR_ERR_UNSUPPORTED;
    const int esize = dtype == MUIR_BF16 ? 2 : 4;
    const long long w = (long long)c->Hk * c->d;
    if (!ok_ld(k_ld, w, esize) || !ok_ld(v_ld, w, esize)) return MUIR_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return MUIR_OK;
    if (!ok_ptr(k) || !ok_ptr(v) || !ok_ints(start) || !aligned_to(count, 4)) return MUIR_ERR_INVALID_ARG;
    if ((st = check_device()) != MUIR_OK) return st;
    muir::AppendArgs a{};
    a.k = k; a.v = v;
    a.k_ld = k_ld ? k_ld : w;
    a.v_ld = v_ld ? v_ld : w;
    a.k_pages = c->k_pages; a.v_pages = c->v_pages;
    a.k_scale = c->k_scale; a.v_scale = c->v_scale;
    a.table = c->table; a.start = start; a.count = count;
    a.T = T; a.Hk = c->Hk; a.page = c->page; a.num_pages = c->num_pages; a.max_pages = c->max_pages;
    return from_cuda(muir::launch_kv_append(a, B, c->d, dtype == MUIR_BF16, static_cast<cudaStream_t>(stream)));
}

size_t muir_attn_step_workspace(int B, int Hq, const muir_kv_cache* c) {
    if (check_step(B, Hq, c) != MUIR_OK) return 0;
    return muir::attn_step_ws_bytes(B, Hq, c->Hk, c->d, c->page, c->max_pages);
}

muir_status muir_attn_step(int B, int Hq, const muir_kv_cache* c, const void* q,
                           const int* lens, float scale, int window, void* o, void* ws,
                           size_t ws_bytes, void* stream) {
    muir_status st = check_step(B, Hq, c);
    if (st != MUIR_OK) return st;
    if (!ok_ptr(q) || !ok_ptr(o) || !ok_ints(lens) || !ok_scale(scale) || window < 0) return MUIR_ERR_INVALID_ARG;
    const size_t need = muir::attn_step_ws_bytes(B, Hq, c->Hk, c->d, c->page, c->max_pages);
    if (ws_bytes < need || (need > 0 && !ok_ptr(ws))) return MUIR_ERR_WORKSPACE;
    if ((st = check_device()) != MUIR_OK) return st;
    muir::StepArgs a{};
    a.q = q; a.o = o;
    a.k_pages = c->k_pages; a.v_pages = c->v_pages;
    a.k_scale = c->k_scale; a.v_scale = c->v_scale;
    a.table = c->table; a.lens = lens;
    a.scale_log2 = scale * kLog2e;
    a.window = window;
    a.Hq = Hq; a.Hk = c->Hk; a.page = c->page; a.num_pages = c->num_pages; a.max_pages = c->max_pages;
    return from_cuda(muir::launch_attn_step(a, B, c->d, ws, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
