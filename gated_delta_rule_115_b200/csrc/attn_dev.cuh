// attn_dev.cuh -- device helpers shared by the softmax-attention kernels.
#pragma once

#include "attn.h"
#include "tc2.cuh"

namespace muir {
namespace attn {

using namespace t2;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}

// kind::f16 with A read from tensor memory: lane m = row m, two 16-bit values a column.
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(id), "r"(acc));
}

__device__ __forceinline__ void tmem_st32u(uint32_t ta, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(ta),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// Two float32 -> bf16 pair in one word (lo in the low half), round to nearest even.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Pairs of float32 in one 64-bit register, rounded as two single operations would be: half
// the instructions of what surrounds the exponentials.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A bit for each of columns 0 .. 31: those in [a, b].
__device__ __forceinline__ uint32_t visible32(int a, int b) {
    const uint32_t upto_b = b < 0 ? 0u : b >= 31 ? ~0u : (2u << b) - 1u;
    const uint32_t below_a = a <= 0 ? 0u : a >= 32 ? ~0u : (1u << a) - 1u;
    return upto_b & ~below_a;
}
// The others' scores become -infinity.
__device__ __forceinline__ void hide(float (&s)[32], uint32_t visible) {
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = visible & (1u << i) ? s[i] : -INFINITY;
}

// One tile of 128 tokens x D channels of one head: D / 64 boxes of 64 channels, 16 KB each.
template <int D>
__device__ __forceinline__ void load_tile(unsigned char* dst, const CUtensorMap* map, int head, int token,
                                          uint64_t* bar) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * kT16Block, map, 64 * c, head, token, bar);
}

// Zeroes rows [first, 128) of a tile (one warp); ordered before the async proxy's reads.
template <int D>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int first) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
        for (int i = first * 8 + lane; i < kTile * 8; i += 32)
            *reinterpret_cast<uint4*>(tile + c * kT16Block + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    __syncwarp();
}

// 128 lanes x W columns of tensor memory, each lane times its f, as bf16 into columns of a
// token-major tensor (`ld` elements between rows, rows < `rows` only), through a tile of
// shared memory that nothing reads any more: a row is a lane in tensor memory, and a lane that
// stored its own row would touch 32 lines with every store.  Four warps; `any` false: zeros.
template <int W>
__device__ __forceinline__ void store_rows(uint32_t tsrc, float f, bool any, unsigned char* tile,
                                           __nv_bfloat16* dst, long long ld, int rows) {
    const int w = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, r = 32 * w + lane;
    const uint32_t lane0 = (uint32_t)w << 21;
    constexpr int N = W >= 64 ? 2 : 1;  // loads of 32 columns in flight
#pragma unroll
    for (int x = 0; x < W; x += 32 * N) {
        float v[N][32];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (any) {
                tmem_ld32(tsrc + lane0 + x + 32 * n, v[n]);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[n][i] = 0.f;
            }
        }
        if (any) tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32 * N; ++i) v[i >> 5][i & 31] *= f;
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) st_chunk16<true>(tile, r, x / 8 + i, v[i >> 2] + 8 * (i & 3));
    }
    __syncwarp();
    constexpr int CH = W / 8, RPI = 32 / CH;  // lanes a row, rows an instruction
    constexpr int U = 32 / RPI < 8 ? 32 / RPI : 8;
    const int rr0 = 32 * w + lane / CH, ch = lane % CH;
    __nv_bfloat16* out = dst + (long long)rr0 * ld + 8 * ch;
#pragma unroll
    for (int i = 0; i < 32 / RPI; i += U) {
        uint4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) v[k] = *reinterpret_cast<const uint4*>(tile + t16_off(rr0 + (i + k) * RPI, ch));
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (rr0 + (i + k) * RPI < rows) *reinterpret_cast<uint4*>(out + (long long)(i + k) * RPI * ld) = v[k];
    }
    __syncwarp();  // the warp's rows of the tile may be written again
}

// Blocks of a launch lie on the grid as (head, block % 65535, block / 65535): no division
// before a block's first load.
constexpr unsigned kGridY = 65535;
inline dim3 block_grid(int heads, long long blocks) {
    return dim3((unsigned)heads, (unsigned)(blocks < kGridY ? blocks : kGridY),
                (unsigned)((blocks + kGridY - 1) / kGridY));
}
__device__ __forceinline__ int block_index() { return (int)(blockIdx.y + kGridY * blockIdx.z); }

// Key head of query head h < 2^16: h / group, by the reciprocal (off by under 2^-22 h / group,
// where half a head's distance to the next integer is 1 / (2 group)).
__device__ __forceinline__ int key_head(int h, float inv_group) { return (int)(((float)h + 0.5f) * inv_group); }

// Block `blk` of a launch: its sequence, and its place in it counted so that a larger `rank`
// has more work under a causal mask.  Blocks come by rank, the largest first, and at one rank
// by sequence (the longest first): whichever order they end in, the last ones are short.  With
// sequence k the k-th longest, ranks from its number of blocks up to the one before's hold k
// blocks each, and the first of them is block seqs[k - 1].block0.
struct Place {
    Seq sq;
    int rank;
};
__device__ __forceinline__ Place place_of(const Seq* seqs, int n, int blk) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seqs[mid].block0 <= blk) lo = mid;
        else hi = mid - 1;
    }
    const unsigned i = (unsigned)(blk - seqs[lo].block0), level = i / (unsigned)(lo + 1);
    return {seqs[i - level * (lo + 1)], seqs[lo].blocks - 1 - (int)level};
}

}  // namespace attn
}  // namespace muir
