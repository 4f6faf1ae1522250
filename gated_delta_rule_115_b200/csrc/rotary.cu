// rotary.cu -- rotary positions of q and k (attention layers next to the
// gated-delta-rule mixer; the recurrence itself takes its order from the state
// and needs none).
//
// Per token at position p and channel pair i of the first `rot` channels,
//
//     (a, b) -> m (a cos t - b sin t,  b cos t + a sin t),    t = p f_i
//
// with pairs (2i, 2i+1) (interleaved) or (i, i + rot/2) (half layout); channels
// past `rot` pass through.  The map is linear, so its gradient is its transpose:
// the same with -t ("inverse").
//
// Angles: p f_i reaches 1e6 turns and more in long contexts, where float32 has no
// fraction left, so the angle is formed and reduced to a fraction of a turn in
// float64, and only then rounded to float32 for sincospi.  Near position 2^31 even
// float64 is short: p f, 1 / (2 pi) and their product are each off by 2^-53 of up to
// 2^28 turns, 2^-22.9 half turns together.  The whole turns are therefore taken off the
// unrounded product, and the rests of p f and of 1 / (2 pi) added: the fraction is off by
// 2^-53 half turns and its rounding to float32 by 2^-25, at any int32 position.
//
// Bound by HBM: q and k are read once and written once (32768 tokens of 16 + 4 heads of 128 in
// bfloat16: 54 us, 6.2 TB/s).  A block takes a few
// tokens: it issues its 16-byte loads (two vectors an item: the two halves of the
// same pairs, or two neighbours), computes each (token, pair)'s sine and cosine
// once for all heads into shared memory while they are in flight, and applies
// them.  Every item is read and written by one thread, so the call works in place.
#include "common.cuh"
#include "kernels.h"
#include "profile.h"

namespace muir {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotItems = 2;       // items of two 16-byte vectors in flight per thread
constexpr int kRotTabPairs = 1024; // (token, pair) entries of the table
constexpr double kInv2Pi = 0.15915494309189535, kInv2PiRest = -9.839338337591243e-18;  // 1 / (2 pi), their sum

__device__ __forceinline__ void rot_unpack(const uint4& a, float* v, float) {
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
}
__device__ __forceinline__ void rot_unpack(const uint4& a, float* v, __nv_bfloat16) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 rot_pack(const float* v, float) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 rot_pack(const float* v, __nv_bfloat16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRotThreads, 5) k_rotary(RotaryArgs p) {
    constexpr int V = 16 / (int)sizeof(T);  // channels per vector
    // m cos t, then m sin t, of a token's pairs, four to a vector: [token][2 V / 4][item],
    // where an item's V pairs are the same in every head; lanes of neighbouring items read
    // neighbouring vectors
    constexpr int Q = V / 4;
    __shared__ float4 tab[kRotTabPairs / 2];
    const int half = p.rot / 2;
    const int head_shift = 31 - __clz(p.d / (2 * V));  // log2 of the items of a head
    const int rot_items = p.rot / (2 * V);
    const int heads = p.Hq + p.Hk;
    const int per_tok = heads << head_shift;
    const long long tok0 = (long long)blockIdx.x * p.tokens_per_block;
    const int ntok = (int)min((long long)p.tokens_per_block, p.tokens - tok0);
    const int total = ntok * per_tok;
    const bool copy_rest = p.q_out != p.q || p.k_out != p.k;
    bool have_tab = false;
    for (int base = 0; base < total; base += kRotThreads * kRotItems) {
        uint4 x[kRotItems][2];
        T* dst[kRotItems];
        int ti[kRotItems];   // the item's place in the table, -1: pass through, -2: none
        int gap[kRotItems];  // channels between the item's two vectors
#pragma unroll
        for (int u = 0; u < kRotItems; ++u) {
            const int it = base + u * kRotThreads + (int)threadIdx.x;
            ti[u] = -2;
            if (it >= total) continue;
            const int th = it >> head_shift;
            const int t = (int)((unsigned)th / (unsigned)heads);
            const int h = th - t * heads;
            const int c = it & ((1 << head_shift) - 1);
            const bool is_q = h < p.Hq;
            const int hh = is_q ? h : h - p.Hq;
            int ch;
            if (c < rot_items) {
                ch = INTER ? c * 2 * V : c * V;
                gap[u] = INTER ? V : half;
                ti[u] = t * (2 * Q) * rot_items + c;
            } else {
                ch = c * 2 * V;
                gap[u] = V;
                ti[u] = copy_rest ? -1 : -2;
            }
            const long long row = tok0 + t;
            const T* src = is_q ? static_cast<const T*>(p.q) + row * p.q_ld + (long long)hh * p.d + ch
                                : static_cast<const T*>(p.k) + row * p.k_ld + (long long)hh * p.d + ch;
            dst[u] = is_q ? static_cast<T*>(p.q_out) + row * p.qo_ld + (long long)hh * p.d + ch
                          : static_cast<T*>(p.k_out) + row * p.ko_ld + (long long)hh * p.d + ch;
            if (ti[u] != -2) {
                x[u][0] = *reinterpret_cast<const uint4*>(src);
                x[u][1] = *reinterpret_cast<const uint4*>(src + gap[u]);
            }
        }
        if (!have_tab) {  // block-uniform
            for (int e = threadIdx.x; e < ntok * half; e += kRotThreads) {
                const int t = e / half, i = e - t * half;
                const long long row = tok0 + t;
                const int pos = p.positions ? p.positions[row] : (int)(row % p.T);
                // a + rest is p f exactly, and fma takes a / (2 pi) less its whole turns unrounded
                const double x = pos, f = p.inv_freq[i];
                const double a = __dmul_rn(x, f), rest = fma(x, f, -a);
                const double turn = fma(a, kInv2Pi, -rint(__dmul_rn(a, kInv2Pi)));
                const float w = 2.f * (float)(turn + fma(a, kInv2PiRest, rest * kInv2Pi));  // in [-1, 1]
                float sn, cs;
                sincospif(w, &sn, &cs);
                const int at = (t * (2 * Q) + (i % V) / 4) * rot_items + i / V;
                reinterpret_cast<float*>(tab + at)[i % 4] = cs * p.mscale;
                reinterpret_cast<float*>(tab + at + Q * rot_items)[i % 4] = (p.inverse ? -sn : sn) * p.mscale;
            }
            __syncthreads();
            have_tab = true;
        }
#pragma unroll
        for (int u = 0; u < kRotItems; ++u) {
            if (ti[u] == -2) continue;
            if (ti[u] >= 0) {
                float a[2 * V], y[2 * V];
                rot_unpack(x[u][0], a, T());
                rot_unpack(x[u][1], a + V, T());
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const float4 c4 = tab[ti[u] + q * rot_items], s4 = tab[ti[u] + (Q + q) * rot_items];
                    const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int i = 4 * q + x;
                        const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + V;
                        y[ia] = a[ia] * cs[x] - a[ib] * sn[x];
                        y[ib] = a[ib] * cs[x] + a[ia] * sn[x];
                    }
                }
                x[u][0] = rot_pack(y, T());
                x[u][1] = rot_pack(y + V, T());
            }
            *reinterpret_cast<uint4*>(dst[u]) = x[u][0];
            *reinterpret_cast<uint4*>(dst[u] + gap[u]) = x[u][1];
        }
    }
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, bool bf16, bool interleaved, cudaStream_t st) {
    if (a.tokens == 0) return cudaSuccess;
    const int vec = bf16 ? 8 : 4;
    const int per_tok = (a.Hq + a.Hk) * (a.d / (2 * vec));
    // enough items for every thread's kRotItems, as many tokens as the table holds, and
    // no fewer than two blocks an SM as long as the call has the tokens for it
    long long tpb = (kRotThreads * kRotItems + per_tok - 1) / per_tok;
    tpb = tpb < kRotTabPairs / (a.rot / 2) ? tpb : kRotTabPairs / (a.rot / 2);
    const long long spread = a.tokens / (2 * 148);
    if (tpb > spread) tpb = spread < 1 ? 1 : spread;
    a.tokens_per_block = (int)tpb;
    const unsigned grid = (unsigned)((a.tokens + tpb - 1) / tpb);
    if (bf16) {
        if (interleaved)
            MUIR_TIMED("k_rotary", st, k_rotary<__nv_bfloat16, true><<<grid, kRotThreads, 0, st>>>(a));
        else
            MUIR_TIMED("k_rotary", st, k_rotary<__nv_bfloat16, false><<<grid, kRotThreads, 0, st>>>(a));
    } else {
        if (interleaved)
            MUIR_TIMED("k_rotary", st, k_rotary<float, true><<<grid, kRotThreads, 0, st>>>(a));
        else
            MUIR_TIMED("k_rotary", st, k_rotary<float, false><<<grid, kRotThreads, 0, st>>>(a));
    }
    return cudaGetLastError();
}

}  // namespace muir
