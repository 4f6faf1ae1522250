// kvcache.cu -- the paged 8-bit key/value cache of an attention layer: appending
// tokens, and one query token per sequence attending over it.
//
// A page holds `page` tokens of every key head: codes [Hk][page][d] in e4m3 and one
// float32 scale for each (page, head), value = code * scale.  Scales are powers of
// two: e4m3 carries its own exponent, so a finer scale buys no precision, and a page
// whose scale has to grow when a larger token arrives is encoded again exactly (only
// codes that become subnormal lose bits).
//
//   append:  scale = max(scale held, smallest 2^e >= 2^-100 with amax / 2^e <= 448)
//            code  = e4m3(x / scale), round to nearest even
//   step:    s_j = scale_q k_j.q;  o = sum_j exp(s_j - max) v_j / sum_j exp(s_j - max)
//
// Both are bound by HBM.  The step reads 2 d bytes a key and head and nothing else of
// that size; see k_attn_step for how the codes reach the tensor cores.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"
#include "profile.h"
#include "tc2.cuh"
#include "tmap.h"

namespace muir {

__device__ unsigned int g_kv_timeouts;

namespace {


__device__ __forceinline__ void kv_unpack(const uint4& a, float* v, float) {
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
}
__device__ __forceinline__ void kv_unpack(const uint4& a, float* v, __nv_bfloat16) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Four floats -> four e4m3 codes (round to nearest even, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\ncvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\nmov.b32 %0, {lo, hi};\n}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Running maximum of magnitudes, NaN passed over; infinities count.
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float vec_amax(const uint4& x, float amax, float) {
    amax = fmaxf(fmaxf(amax, fabsf(__uint_as_float(x.x))), fabsf(__uint_as_float(x.y)));
    return fmaxf(fmaxf(amax, fabsf(__uint_as_float(x.z))), fabsf(__uint_as_float(x.w)));
}
__device__ __forceinline__ float vec_amax(const uint4& x, float amax, __nv_bfloat16) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t m = bf16x2_max(bf16x2_max(x.x & kAbs, x.y & kAbs), bf16x2_max(x.z & kAbs, x.w & kAbs));
    return fmaxf(fmaxf(amax, __uint_as_float(m << 16)), __uint_as_float(m & 0xffff0000u));
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Smallest power of two s >= 2^kMinScaleExp with amax <= 448 s (448 = 0.875 2^9).
constexpr int kMinScaleExp = -100;
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    // amax = 1.f 2^x: 2^(x-8) reaches 448 = 1.75 2^8 while 1.f <= 1.75, then the next
    int e = (int)(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7);
    if (e < kMinScaleExp) e = kMinScaleExp;  // zero and subnormal magnitudes too
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Largest of the block's values, which every thread gets.
template <int NT>
__device__ __forceinline__ float block_max(float v, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) v = fmaxf(v, part[w]);
    return v;
}

// One block per (page a sequence's new tokens touch, head, keys or values): the new
// rows' largest finite magnitude, the page's scale, held rows encoded again if the
// scale grew, new rows encoded.  Rows of the page behind the new tokens stay as they are.
// The rows are read once, NV vectors of 16 bytes a thread, all in flight together, and
// wait in registers for the scale.  Bound by issue slots next to HBM: magnitudes are
// compared two bfloat16 at a time (one by one, with addresses formed for every vector, it
// took 18 instructions a value and 16.2 us for 17800 tokens of 4 heads of 128, where this takes
// 10.7: 5.1 TB/s).
template <typename T, int D, int NT, int NV>
__global__ void __launch_bounds__(NT) k_kv_append(AppendArgs p) {
    constexpr int V = 16 / (int)sizeof(T);       // channels per vector
    constexpr int PER_ROW = D / V;
    constexpr int STEP = NT / PER_ROW;  // rows between a thread's vectors
    const int b = blockIdx.z >> 1, which = blockIdx.z & 1, h = blockIdx.y;
    const int start = p.start[b];
    int count = p.count ? p.count[b] : p.T;
    count = count < 0 ? 0 : (count > p.T ? p.T : count);
    if (start < 0 || count == 0) return;
    const long long slot = (long long)start / p.page + blockIdx.x;
    // first and one-past-last new token that fall into this page
    const long long page0 = slot * p.page;
    const int lo = (int)max(0LL, page0 - start);
    const int hi = (int)min((long long)count, page0 + p.page - start);
    if (lo >= hi || slot >= p.max_pages) return;
    const int id = p.table[(long long)b * p.max_pages + slot];

    const int row = threadIdx.x / PER_ROW, col = (threadIdx.x % PER_ROW) * V;  // the thread's first vector
    const long long ld = which ? p.v_ld : p.k_ld;
    const T* src = static_cast<const T*>(which ? p.v : p.k) + ((long long)b * p.T + lo + row) * ld + (long long)h * D + col;
    uint4 x[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        x[n] = make_uint4(0u, 0u, 0u, 0u);
        if (row + n * STEP < hi - lo) x[n] = *reinterpret_cast<const uint4*>(src + n * STEP * ld);
    }
    if (id < 0 || id >= p.num_pages) return;  // the whole block
    unsigned char* page = static_cast<unsigned char*>(which ? p.v_pages : p.k_pages) +
                          ((long long)id * p.Hk + h) * p.page * D;
    float* scale = (which ? p.v_scale : p.k_scale) + (long long)id * p.Hk + h;
    const int held = (int)(start + lo - page0);  // rows of the page before the new ones
    const float old = held > 0 ? *scale : 0.f;

    __shared__ float part[2][NT / 32];
    float amax = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) amax = vec_amax(x[n], amax, T());
    amax = block_max<NT>(amax, part[0]);  // and every thread has read the old scale
    if (amax > 3.402823466e38f) {     // an infinity among them: the largest finite one instead
        amax = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float v[V];
            kv_unpack(x[n], v, T());
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (fabsf(v[j]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(v[j]));
        }
        amax = block_max<NT>(amax, part[1]);
    }
    const float now = fmaxf(old, scale_for(amax));
    if (threadIdx.x == 0) *scale = now;

    const float inv = __frcp_rn(now);  // exact: a power of two in [2^-120, 2^100]
    if (now != old) {
        const float ratio = old / now;
        for (int i = threadIdx.x; i < held * (D / 4); i += NT) {
            uint32_t* w = reinterpret_cast<uint32_t*>(page) + i;
            const uint32_t y = *w;
            const float2 a = from_e4m3x2(y & 0xffffu), c = from_e4m3x2(y >> 16);
            *w = e4m3x4(a.x * ratio, a.y * ratio, c.x * ratio, c.y * ratio);
        }
    }
    unsigned char* dst = page + (held + row) * D + col;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        if (row + n * STEP >= hi - lo) break;
        float v[V];
        kv_unpack(x[n], v, T());
        uint32_t w[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
            w[j] = e4m3x4(v[4 * j] * inv, v[4 * j + 1] * inv, v[4 * j + 2] * inv, v[4 * j + 3] * inv);
        if (V == 8)
            *reinterpret_cast<uint2*>(dst + n * STEP * D) = make_uint2(w[0], w[V / 4 - 1]);
        else
            *reinterpret_cast<uint32_t*>(dst + n * STEP * D) = w[0];
    }
}

// ------------------------------------------------------------------ step

// Keys and values travel in stages of kStepKeys keys, copied by TMA into a swizzled ring by
// one warp that runs ahead; each of four warps takes 32 keys of a stage.
constexpr int kStepKeys = 128;
constexpr int kStepWarps = 4;
constexpr int kWarpKeys = kStepKeys / kStepWarps;
constexpr int kStepThreads = 32 * (kStepWarps + 1);
constexpr int kStepStages = 3;
constexpr int kGroups = kStepKeys / 16;    // groups of 16 keys, within one page each
constexpr int kU = kWarpKeys / 16;         // a warp's
constexpr int kMaxRows = 16;               // query heads of a block
constexpr int kMaxSplits = 128;            // of a sequence; two to a thread of the smallest join
constexpr float kSlack = 8.f;              // log2 of how far a weight may exceed 1
constexpr int kMaxQueryExp = 109;          // log2 of a query row's largest factor
constexpr float kWeightExp = 7.f;          // fp16 weights are 2^(score - reference + 7) <= 2^15

struct StepMeta {        // per group of a stage
    float ks, lv;        // key scale, log2 of the value scale
    int lo, hi;          // visible keys [lo, hi) of the 16
};

template <int D>
struct StepSmem {
    static constexpr int kTile = kStepKeys * D;               // bytes of K (or V) in a stage
    static constexpr int kMeta = kStepStages * 2 * kTile;
    static constexpr int kBars = kMeta + kStepStages * kGroups * (int)sizeof(StepMeta);
    static constexpr int kBytes = kBars + 2 * kStepStages * 8;
    static_assert(kStepWarps * kMaxRows * (D + 2) * 4 <= kMeta, "the warps' parts reuse the ring");
};

__device__ __forceinline__ uint32_t h2_from_e4m3(uint32_t two) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t h2_from_e4m3_hi(uint32_t two) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(r) : "r"(two));
    return r;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held one row to four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(t2::saddr(bar)) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a stage's tile, as the tensor map's swizzle
// places it (128-byte rows: chunk ^ row % 8; 64-byte rows: chunk ^ row / 2 % 4).
template <int D>
__device__ __forceinline__ uint32_t step_off(int r, int c) {
    return D == 128 ? (uint32_t)r * 128u + (uint32_t)((c ^ (r & 7)) << 4)
                    : (uint32_t)r * 64u + (uint32_t)((c ^ ((r >> 1) & 3)) << 4);
}

// One block: up to 8 HT query heads of one key head of one sequence over one range of its
// keys.  Bound by HBM: 64 streams of up to 16384 tokens, 16 query heads over 4 of 128, 100 us,
// 5.6 TB/s.
//
// Both products run transposed on mma.sync m16n8k16, in fp16 with float32 sums: keys (then
// channels) are the 16 rows and query heads the 8 columns, so that the cache's side, which
// is all the work there is, fills the instruction at any group size; with the heads as rows
// instead, four heads left 12 of 16 rows empty and the kernel was bound by issue slots
// (167 us for 64 streams of 16384 tokens, 4 key heads; 46% of the rate of HBM).  e4m3 codes
// are exact in fp16.  A product's contraction may run in any order as long as both operands
// agree: lane (g, c) takes D/4 neighbouring bytes of keys g and g + 8 for the scores, and
// D/8 neighbouring channels of keys 2c, 2c+1, 2c+8, 2c+9 for the output, so both read shared
// memory in 16-byte vectors without a transposition; the weights, which the score product
// leaves by key and the output product takes by head, are transposed in registers.
//
// Query rows are scaled by a power of two to a largest magnitude in [2^13, 2^14): fp16
// then holds bf16 values exactly down to 2^-28 of the row's largest.  The power ends at 2^109,
// under which the smallest bf16 value, 2^-133, is fp16's and all are exact: with more, the
// factor of the scores of queries near 2^-128 would be subnormal, and lose its bits where a
// page's scale near 2^120 makes those scores ordinary ones.  Softmax runs in
// base 2 against references held in float32 that move only when a score outgrows them by
// 2^8: m over the scores for the normaliser, and M over score + log2(value scale) for the
// weights of the value codes, which are kept as fp16(2^(score + log2 scale - M + 7)):
// relative rounding 2^-11 down to 2^-21 of the reference whatever the pages' scales, where
// a weight without its page's scale could vanish next to a page of large values.
template <int D, int HT>
__global__ void __launch_bounds__(kStepThreads, HT == 1 ? 2 : 1) k_attn_step(const __grid_constant__ StepArgs p) {
    using SM = StepSmem<D>;
    constexpr int KSTEPS = D / 16;   // 16-deep steps of the score product
    constexpr int NT = D / 16;       // 16-channel tiles of the output product
    constexpr int ROWS = 8 * HT;
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + SM::kBars);
    uint64_t* empty = full + kStepStages;
    StepMeta* meta = reinterpret_cast<StepMeta*>(sm + SM::kMeta);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.Hq / p.Hk;
    const int gtiles = (G + ROWS - 1) / ROWS;
    const int hk = blockIdx.y / gtiles, g0 = (blockIdx.y % gtiles) * ROWS;
    const int b = blockIdx.z, split = blockIdx.x;

    long long len = p.lens[b];
    const long long cap = (long long)p.max_pages * p.page;
    len = len < 0 ? 0 : (len > cap ? cap : len);
    const long long first = p.window > 0 && len > p.window ? len - p.window : 0;
    // every split takes whole stages from the stage that holds `first`
    const long long base = first / kStepKeys * kStepKeys;
    long long per = (len - base + p.splits - 1) / p.splits;
    per = (per + kStepKeys - 1) / kStepKeys * kStepKeys;
    if (per < p.min_keys) per = p.min_keys;
    const long long lo = base + split * per;
    const long long hi = min(len, lo + per);
    const int nst = hi > lo ? (int)((hi - lo + kStepKeys - 1) / kStepKeys) : 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStepStages; ++i) {
            t2::mbar_init(full + i, 2);  // the copies and the metadata
            t2::mbar_init(empty + i, kStepWarps);
        }
        t2::fence_barrier_init();
    }
    __syncthreads();
    bool bad = false;

    if (warp == kStepWarps) {
        // ---- producer: page ids and scales 32 pages ahead, one copy a page
        const int per_stage = kStepKeys / p.page;
        const int npage = nst * per_stage;
        for (int i0 = 0; i0 < npage && !bad; i0 += 32) {
            int id = -1;
            float ks = 0.f, vs = 0.f;
            const long long key = lo + (long long)(i0 + lane) * p.page;
            if (i0 + lane < npage && key < hi) {
                id = p.table[(long long)b * p.max_pages + key / p.page];
                if (id < 0 || id >= p.num_pages) id = -1;
                if (id >= 0) {
                    ks = p.k_scale[(long long)id * p.Hk + hk];
                    vs = p.v_scale[(long long)id * p.Hk + hk];
                }
            }
            const int n = min(32, npage - i0);
            for (int i = 0; i < n; i += per_stage) {
                const int st = (i0 + i) / per_stage, slot = st % kStepStages;
                if (st >= kStepStages) {
                    const bool ok = t2::mbar_wait(empty + slot, ((st / kStepStages) - 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) {
                        bad = true;
                        break;
                    }
                }
                // the copies first: they need the page ids only, and are on their way while
                // the scales still are
                const bool mine = lane >= i && lane < i + per_stage && id >= 0;  // a page of this stage
                const int copies = __popc(__ballot_sync(0xffffffffu, mine));
                if (lane == 0) t2::mbar_arrive_expect_tx(full + slot, (uint32_t)(copies * 2 * p.page * D));
                __syncwarp();
                if (mine) {
                    unsigned char* kd = sm + (size_t)slot * 2 * SM::kTile + (size_t)(lane - i) * p.page * D;
                    t2::tma_load_3d(kd, &p.tk, 0, 0, id * p.Hk + hk, full + slot);
                    t2::tma_load_3d(kd + SM::kTile, &p.tv, 0, 0, id * p.Hk + hk, full + slot);
                }
                __syncwarp();
                // metadata of the stage's groups
                const int src = i + (lane * 16) / p.page;
                const int gid = __shfl_sync(0xffffffffu, id, src & 31);
                const float gks = __shfl_sync(0xffffffffu, ks, src & 31);
                const float gvs = __shfl_sync(0xffffffffu, vs, src & 31);
                if (lane < kGroups) {
                    const long long k0 = lo + (long long)st * kStepKeys + lane * 16;
                    StepMeta m;
                    m.ks = gks;
                    m.lv = __log2f(gvs);
                    m.lo = (int)max(0LL, min(16LL, first - k0));
                    m.hi = gid < 0 ? 0 : (int)max(0LL, min(16LL, hi - k0));
                    meta[slot * kGroups + lane] = m;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(full + slot);
            }
        }
        if (bad && lane == 0) atomicOr(&g_kv_timeouts, 1u);
        // the copies in flight land in this block's shared memory: consumers wait for
        // each of them below before the block ends
    }

    // ---- consumers: keys g and g + 8 of a group, heads 8 h + 2 c and + 1
    const int g = lane >> 2, c = lane & 3;
    float m[HT][2], M[HT][2], l[HT][2];
    float acc[HT][NT][4];  // channels g * D/8 + 2 t (0, 1) and + 1 (2, 3) of the two heads
#pragma unroll
    for (int h = 0; h < HT; ++h) {
        m[h][0] = m[h][1] = M[h][0] = M[h][1] = -INFINITY;
        l[h][0] = l[h][1] = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[h][t][i] = 0.f;
    }

    if (warp < kStepWarps && nst > 0) {
        // query fragments of head 8 h + g: step s of the contraction takes channels
        // c * D/4 + 4 s .. + 3 of lane c
        uint32_t qb[HT][KSTEPS][2];
        float qscale[HT][2];
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            const int head = g0 + 8 * h + g;
            float x[D / 4];
            float mx = 0.f;
            const bool on = head < G;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                                     ((long long)b * p.Hq + (long long)hk * G + (on ? head : 0)) * D + c * (D / 4);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (on) w = *reinterpret_cast<const uint4*>(q + 8 * i);
                kv_unpack(w, x + 8 * i, __nv_bfloat16());
            }
#pragma unroll
            for (int i = 0; i < D / 4; ++i) mx = fmaxf(mx, fabsf(x[i]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            int e = 0;
            if (mx > 0.f && mx <= 3.4e38f) frexpf(mx, &e);
            const int sh = min(14 - e, kMaxQueryExp);  // from -114: applied in two halves
            const float s1 = ldexpf(1.f, sh / 2), s2 = ldexpf(1.f, sh - sh / 2);
            const float qs = p.scale_log2 / s1 / s2;
#pragma unroll
            for (int i = 0; i < 2; ++i) qscale[h][i] = __shfl_sync(0xffffffffu, qs, 4 * (2 * c + i));
#pragma unroll
            for (int s = 0; s < KSTEPS; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half2 u = __floats2half2_rn(x[4 * s + 2 * i] * s1 * s2, x[4 * s + 2 * i + 1] * s1 * s2);
                    qb[h][s][i] = *reinterpret_cast<const uint32_t*>(&u);
                }
        }

        for (int st = 0; st < nst; ++st) {
            const int slot = st % kStepStages;
            const bool ok = t2::mbar_wait(full + slot, (st / kStepStages) & 1);
            if (!__all_sync(0xffffffffu, ok)) {
                bad = true;
                break;
            }
            const unsigned char* kt = sm + (size_t)slot * 2 * SM::kTile;
            const unsigned char* vt = kt + SM::kTile;
            StepMeta mt[kU];
            bool part = false, any = false;  // uniform in the warp
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                mt[u] = meta[slot * kGroups + kU * warp + u];
                part = part || mt[u].lo > 0 || mt[u].hi < 16;
                any = any || mt[u].hi > mt[u].lo;
            }
            if (any) {
                float s[kU][HT][4];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
#pragma unroll
                    for (int h = 0; h < HT; ++h) s[u][h][0] = s[u][h][1] = s[u][h][2] = s[u][h][3] = 0.f;
                    const int r = kWarpKeys * warp + 16 * u + g;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        const uint4 ka = *reinterpret_cast<const uint4*>(kt + step_off<D>(r, c * (D / 64) + i));
                        const uint4 kb = *reinterpret_cast<const uint4*>(kt + step_off<D>(r + 8, c * (D / 64) + i));
                        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t a0 = h2_from_e4m3(wa[j]), a1 = h2_from_e4m3(wb[j]);
                            const uint32_t a2 = h2_from_e4m3_hi(wa[j]), a3 = h2_from_e4m3_hi(wb[j]);
#pragma unroll
                            for (int h = 0; h < HT; ++h)
                                mma_f16_16816(s[u][h], a0, a1, a2, a3, qb[h][4 * i + j][0], qb[h][4 * i + j][1]);
                        }
                    }
                }
                uint32_t pb[kU][HT][2];  // weights as the output product takes them
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    // scores in base 2; does any outgrow its reference?
                    bool grow = false;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            const float f = qscale[h][i] * mt[u].ks;
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float& x = s[u][h][2 * r + i];
                                x *= f;
                                if (part && (g + 8 * r < mt[u].lo || g + 8 * r >= mt[u].hi)) x = -INFINITY;
                                grow = grow || x > m[h][i] + kSlack || x + mt[u].lv > M[h][i] + kSlack;
                            }
                        }
                    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float top = -INFINITY, tv = -INFINITY;
#pragma unroll
                            for (int u = 0; u < kU; ++u) {
                                const float a = fmaxf(s[u][h][i], s[u][h][2 + i]);
                                top = fmaxf(top, a);
                                tv = fmaxf(tv, a + mt[u].lv);
                            }
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) {
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                                tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, o));
                            }
                            const float mn = fmaxf(m[h][i], top), Mn = fmaxf(M[h][i], tv);
                            l[h][i] *= mn == -INFINITY ? 1.f : ex2(m[h][i] - mn);
                            const float f = Mn == -INFINITY ? 1.f : ex2(M[h][i] - Mn);
                            m[h][i] = mn;
                            M[h][i] = Mn;
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                acc[h][t][i] *= f;
                                acc[h][t][2 + i] *= f;
                            }
                        }
                    }
                    float w[kU][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float ms = m[h][i] == -INFINITY ? 0.f : m[h][i];
                        const float Ms = M[h][i] == -INFINITY ? 0.f : M[h][i];
#pragma unroll
                        for (int u = 0; u < kU; ++u)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float x = s[u][h][2 * r + i];
                                l[h][i] += ex2(x - ms);
                                w[u][2 * r + i] = ex2(x + (mt[u].lv + (kWeightExp - Ms)));
                            }
                    }
#pragma unroll
                    for (int u = 0; u < kU; ++u)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const __half2 two = __floats2half2_rn(w[u][2 * r], w[u][2 * r + 1]);
                            pb[u][h][r] = transpose8(*reinterpret_cast<const uint32_t*>(&two));
                        }
                }
                // value codes of keys 2c, 2c+1, 2c+8, 2c+9, channels g * D/8 .. + D/8
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    uint32_t w[4][D / 32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int kk = 2 * c + (i & 1) + 8 * (i >> 1);
                        const int r = kWarpKeys * warp + 16 * u + kk;
                        if (D == 128) {
                            const uint4 x = *reinterpret_cast<const uint4*>(vt + step_off<D>(r, g));
                            w[i][0] = x.x; w[i][1] = x.y; w[i][D / 32 - 2] = x.z; w[i][D / 32 - 1] = x.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2*>(vt + step_off<D>(r, g >> 1) + 8 * (g & 1));
                            w[i][0] = x.x; w[i][1] = x.y;
                        }
                        // slots behind the sequence may hold anything: no code of theirs is used
                        if (part && (kk < mt[u].lo || kk >= mt[u].hi)) {
#pragma unroll
                            for (int j = 0; j < D / 32; ++j) w[i][j] = 0u;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        const uint32_t a0 = __byte_perm(w[0][j], w[1][j], 0x5140), a1 = __byte_perm(w[0][j], w[1][j], 0x7362);
                        const uint32_t b0 = __byte_perm(w[2][j], w[3][j], 0x5140), b1 = __byte_perm(w[2][j], w[3][j], 0x7362);
                        const uint32_t x[8] = {h2_from_e4m3(a0), h2_from_e4m3_hi(a0), h2_from_e4m3(b0), h2_from_e4m3_hi(b0),
                                               h2_from_e4m3(a1), h2_from_e4m3_hi(a1), h2_from_e4m3(b1), h2_from_e4m3_hi(b1)};
#pragma unroll
                        for (int h = 0; h < HT; ++h) {
                            mma_f16_16816(acc[h][2 * j], x[0], x[1], x[2], x[3], pb[u][h][0], pb[u][h][1]);
                            mma_f16_16816(acc[h][2 * j + 1], x[4], x[5], x[6], x[7], pb[u][h][0], pb[u][h][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + slot);
        }
        if (bad && lane == 0) atomicOr(&g_kv_timeouts, 2u);
    }

    // ---- the four warps' parts together: o = sum_w 2^(m_w - m) ..., through the ring's memory
    __syncthreads();
    float* so = reinterpret_cast<float*>(sm);               // [warp][ROWS][D]
    float* sml = so + kStepWarps * ROWS * D;                // [warp][ROWS][2]: m, l
    if (warp < kStepWarps) {
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float sum = l[h][i];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                // in units of 2^m: the codes' weights carry 2^(7 - M)
                const float u = sum > 0.f ? ex2(M[h][i] - kWeightExp - m[h][i]) : 0.f;
                const int row = warp * ROWS + 8 * h + 2 * c + i;
                float* o = so + row * D + g * (D / 8);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    o[2 * t] = acc[h][t][i] * u;
                    o[2 * t + 1] = acc[h][t][2 + i] * u;
                }
                if (g == 0) {
                    sml[row * 2] = m[h][i];
                    sml[row * 2 + 1] = sum;
                }
            }
    }
    __syncthreads();
    const int rows = min(ROWS, G - g0);
    for (int i = threadIdx.x; i < rows * D; i += kStepThreads) {
        const int r = i / D, ch = i % D;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) mm = fmaxf(mm, sml[(w * ROWS + r) * 2]);
        const float ms = mm == -INFINITY ? 0.f : mm;
        float sum = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) {
            const float f = ex2(sml[(w * ROWS + r) * 2] - ms);
            sum += f * sml[(w * ROWS + r) * 2 + 1];
            o += f * so[(w * ROWS + r) * D + ch];
        }
        o = sum > 0.f || sum != sum ? o / sum : 0.f;
        const long long head = (long long)b * p.Hq + (long long)hk * G + g0 + r;
        if (p.splits == 1) {
            static_cast<__nv_bfloat16*>(p.o)[head * D + ch] = __float2bfloat16_rn(o);
        } else {
            p.part[(head * p.splits + split) * D + ch] = o;
            if (ch == 0) p.part_lse[head * p.splits + split] = sum > 0.f || sum != sum ? ms + __log2f(sum) : -INFINITY;
        }
    }
}

// Splits of a sequence and head together: weights 2^(lse_i - max), in the order of the splits.
// (Joined inside a cluster through shared memory instead, 4097 tokens of one stream took as
// long, and batches waited for whole clusters of free SMs: 106 -> 137 us at 64 streams.)
template <int D>
__global__ void __launch_bounds__(D) k_attn_step_join(const float* part, const float* lse, __nv_bfloat16* o,
                                                      int splits) {
    __shared__ float w[kMaxSplits];
    grid_wait();
    const long long head = blockIdx.x;
    const int ch = threadIdx.x;
    if (ch < splits) w[ch] = lse[head * splits + ch];
    if (ch + D < splits) w[ch + D] = lse[head * splits + ch + D];
    __syncthreads();
    float mx = -INFINITY;
    for (int i = 0; i < splits; ++i) mx = fmaxf(mx, w[i]);
    const float ms = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, a = 0.f;
#pragma unroll 8
    for (int i = 0; i < splits; ++i) {  // a split without visible keys: weight 0, o = 0
        const float f = ex2(w[i] - ms);
        sum += f;
        a += f * part[(head * splits + i) * D + ch];
    }
    o[head * D + ch] = __float2bfloat16_rn(sum > 0.f || sum != sum ? a / sum : 0.f);
}

}  // namespace

template <typename T, int D>
static cudaError_t append(const AppendArgs& a, dim3 grid, cudaStream_t st) {
    // The most rows that one page takes in this call, in vectors a thread.  Fewer threads with
    // more vectors each form fewer addresses and scales: 128 with 8 rather than 256 with 4:
    // 17800 tokens of 4 heads of 128, 12.9 -> 10.7 us.
    const int rows = a.T < a.page ? a.T : a.page;
    const int vecs = rows * D * (int)sizeof(T) / 16;
    if (vecs <= 128) MUIR_TIMED("k_kv_append", st, k_kv_append<T, D, 128, 1><<<grid, 128, 0, st>>>(a));
    else if (vecs <= 128 * 8) MUIR_TIMED("k_kv_append", st, k_kv_append<T, D, 128, 8><<<grid, 128, 0, st>>>(a));
    else MUIR_TIMED("k_kv_append", st, k_kv_append<T, D, 256, 16><<<grid, 256, 0, st>>>(a));
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const AppendArgs& a, int B, int d, bool bf16, cudaStream_t st) {
    const dim3 grid((a.T + a.page - 2) / a.page + 1, a.Hk, 2 * B);
    if (bf16) return d == 128 ? append<__nv_bfloat16, 128>(a, grid, st) : append<__nv_bfloat16, 64>(a, grid, st);
    return d == 128 ? append<float, 128>(a, grid, st) : append<float, 64>(a, grid, st);
}

// Query heads of a block: 8 columns of the products, or 16 where the group has more.
static int step_heads(int Hq, int Hk) { return Hq / Hk <= 8 ? 8 : kMaxRows; }

int attn_step_splits(int B, int Hq, int Hk, int d, int page, int max_pages) {
    const int per = step_heads(Hq, Hk);
    const long long units = (long long)B * Hk * ((Hq / Hk + per - 1) / per);
    const long long cap = (long long)page * max_pages;
    // As many blocks as are resident on 148 SMs, where one more starts a second round: two each (2
    // streams of 8192 tokens and 8 key heads 15.7 us at 19 splits, 12.3 at 16), one with 16 heads
    // of 128 channels, whose 211 registers a thread fill an SM (8 streams of 8192 tokens, 16 heads
    // over 1: 17.9 us at 37 splits, 12.6 at 18; at d = 64, with room for two, 10.0 and 10.4).
    // None longer than 2048 keys, up to kMaxSplits, so that one long sequence of a ragged batch
    // does not run on after the others, nor shorter than 256, where a block is mostly its start
    // (4097 tokens of one stream, 4 key heads: 7.8 us at 256 keys, 8.9 at 512).
    // All this of the page table's width: the lengths are on the device.  A table much wider
    // than the sequences costs blocks of fewer keys and empty ones (64 streams of 8192 tokens, 16
    // heads over 4: 100 us with a table for 16384 tokens, 243 for 131072; of 500: 9.2 for 512, 156).
    const int resident = d == 128 && per == kMaxRows ? 1 : 2;
    long long s = resident * 148 / units;
    const long long by_len = (cap + 2047) / 2048;
    if (s < by_len) s = by_len;
    const long long most = (cap + 255) / 256;
    if (s > most) s = most;
    if (s > kMaxSplits) s = kMaxSplits;
    return s < 1 ? 1 : (int)s;
}

size_t attn_step_ws_bytes(int B, int Hq, int Hk, int d, int page, int max_pages) {
    const size_t s = attn_step_splits(B, Hq, Hk, d, page, max_pages);
    return s == 1 ? 0 : (size_t)B * Hq * s * (d + 1) * 4;
}

template <int D, int HT>
static cudaError_t step(const StepArgs& a, dim3 grid, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t err = allow_smem(k_attn_step<D, HT>, StepSmem<D>::kBytes, done);
    if (err != cudaSuccess) return err;
    MUIR_TIMED("k_attn_step", st, k_attn_step<D, HT><<<grid, kStepThreads, StepSmem<D>::kBytes, st>>>(a));
    return cudaGetLastError();
}

cudaError_t launch_attn_step(StepArgs a, int B, int d, void* ws, cudaStream_t st) {
    a.splits = attn_step_splits(B, a.Hq, a.Hk, d, a.page, a.max_pages);
    a.min_keys = 256;
    a.part = static_cast<float*>(ws);
    a.part_lse = a.part + (size_t)B * a.Hq * a.splits * d;
    cudaError_t err = make_tmap_u8(&a.tk, a.k_pages, d, a.page, (uint64_t)a.num_pages * a.Hk, a.page < kStepKeys ? a.page : kStepKeys);
    if (err != cudaSuccess) return err;
    err = make_tmap_u8(&a.tv, a.v_pages, d, a.page, (uint64_t)a.num_pages * a.Hk, a.page < kStepKeys ? a.page : kStepKeys);
    if (err != cudaSuccess) return err;
    const int per = step_heads(a.Hq, a.Hk);
    const dim3 grid(a.splits, a.Hk * ((a.Hq / a.Hk + per - 1) / per), B);
    if (per == 8) err = d == 128 ? step<128, 1>(a, grid, st) : step<64, 1>(a, grid, st);
    else err = d == 128 ? step<128, 2>(a, grid, st) : step<64, 2>(a, grid, st);
    if (err != cudaSuccess || a.splits == 1) return err;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o);
    const float *part = a.part, *lse = a.part_lse;
    MUIR_TIMED("k_attn_step_join", st,
               err = d == 128 ? launch_early(k_attn_step_join<128>, true, dim3(B * a.Hq), 128, 0, st, part, lse, o, a.splits)
                              : launch_early(k_attn_step_join<64>, true, dim3(B * a.Hq), 64, 0, st, part, lse, o, a.splits));
    return err;
}

unsigned int timeouts_kv() {
    unsigned int n = 0;
    cudaMemcpyFromSymbol(&n, g_kv_timeouts, sizeof(n));
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_kv_timeouts, &z, sizeof(z));
    return n;
}

}  // namespace muir
