// attn_fwd.cu -- softmax attention, forward, on tcgen05.
//
//     s_ij = scale q_i . k_j,   lse_i = log sum_j exp s_ij,   o_i = sum_j exp(s_ij - lse_i) v_j
//
// over the keys j that query i sees: j <= i + lk - lq (causal), j > i + lk - lq - window.
//
// One block takes two tiles of 128 queries of one key head of a sequence and walks the keys in
// tiles of 128 once, with the running maximum and sum of each row (base 2, float32).  The
// score product lands in tensor memory, four warps a tile turn it into weights -- a row to a
// thread, so that no row is reduced across threads -- and write them beside the scores as
// the A operand of the second product, whose sum stays in tensor memory until the end.  A
// step's scores leave their place for registers at once, so the next ones (of the other tile,
// or of the next step) are formed while these are still at their exponentials, and no thread
// waits for a product that it does not need yet.
//
//   warps 0-3, 4-7 : softmax of tile 0, 1     warps 8, 9 : issue the two products
//   warp 10        : loads (TMA, a ring of key and value tiles)
//
// The maximum that the weights are taken against moves only when a row outgrows it by 2^8:
// weights up to 2^8 lose nothing in bf16, and the sum in tensor memory is rescaled a few
// times a row instead of at every step.  Weights are rounded to bf16 (half a step, 2^-8) as
// the product's operands; the sums are of the unrounded ones, in float32.
//
// Bound by the tensor cores (4 d flops a visible pair) and, at d = 64 before anything else,
// by the exponentials (16 a clock and SM).  Causal, 16384 tokens of 16 heads over 4 of 128: 0.80
// ms, 1.37 PFLOP/s, in short runs; 0.93 ms, 1.18, once the power limit sets the clock.  8192 tokens
// of 8 heads of 64: 104 us, 0.66 PFLOP/s.
#include <algorithm>

#include "attn_dev.cuh"
#include "profile.h"
#include "tmap.h"

namespace muir {
namespace attn {

__device__ unsigned int g_fwd_timeouts;

namespace {

constexpr int kThreads = 352;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSMs = 148;
constexpr float kSlack = 8.f;  // log2 of how far a weight may exceed 1

struct FwdParams {
    CUtensorMap tq, tk, tv;
    __nv_bfloat16* o;
    float* lse;
    long long lse_seq, lse_head;
    float scale_log2;
    float inv_group;                       // Hk / Hq
    int Hq, causal, window, blocks, n;
    int tiles, by_heads;                   // query tiles of a block: 1, or 2 of the same head, or
                                           // (by_heads) 2 heads' at the same place
    Seq seq[kMaxSeqs];
};

template <int D>
struct FwdSmem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kBars = kRing + kStages * kTileBytes;
    static constexpr int kBytes = kBars + 256;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_attn_fwd(const __grid_constant__ FwdParams p) {
    using SM = FwdSmem<D>;
    constexpr int NS = SM::kStages;
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + SM::kBars);
    uint64_t* s_full = q_full + 2;     // scores of a tile's step are in tensor memory
    uint64_t* s_free = s_full + 2;     // a place for scores has been read (one place: only the first)
    uint64_t* p_full = s_free + 2;     // a tile's weights are in tensor memory
    uint64_t* pv_done = p_full + 2;    // its second product has finished
    uint64_t* kv_full = pv_done + 2;
    uint64_t* kv_empty = kv_full + NS;
    uint64_t* tail_bar = kv_empty + NS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail_bar + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blk = block_index(), h = p.by_heads ? 2 * blockIdx.x : blockIdx.x;
    const int dh = p.by_heads ? 1 : 0, dt = 1 - dh;  // from one of the block's tiles to the next
    if (blk >= p.blocks) return;
    const Place place = place_of(p.seq, p.n, blk);
    const Seq sq = place.sq;
    const int qt = place.rank << (p.tiles == 2 && !p.by_heads ? 1 : 0);  // its first query tile
    const int hk = key_head(h, p.inv_group);
    const int off = sq.lk - sq.lq;

    // key tiles [lo, hi) of each of the two query tiles
    int lo[2], hi[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int r0 = (qt + t * dt) * kTile, r1 = min(r0 + kTile, sq.lq) - 1;  // its rows [r0, r1]
        int last = sq.lk - 1, first = 0;
        if (p.causal) last = min(last, r1 + off);
        if (p.window) first = max(first, r0 + off - p.window + 1);
        hi[t] = last < 0 ? 0 : last / kTile + 1;
        lo[t] = first / kTile;
        if (t >= p.tiles || r0 >= sq.lq || last < first) hi[t] = lo[t] = 0;
    }
    const bool on0 = hi[0] > lo[0], on1 = hi[1] > lo[1];
    const int jlo = on0 ? (on1 ? min(lo[0], lo[1]) : lo[0]) : lo[1];
    const int jhi = on0 ? (on1 ? max(hi[0], hi[1]) : hi[0]) : hi[1];
    const int loads = 2 * (jhi - jlo);  // K, V of each key tile in turn

    // The loading warp sets the barriers up and sends its first loads off before the block
    // meets: they take longer than everything else that comes before the first product.
    auto load = [&](int i) {
        const int st = i % NS;
        mbar_arrive_expect_tx(kv_full + st, SM::kTileBytes);
        load_tile<D>(sm + SM::kRing + st * SM::kTileBytes, (i & 1) ? &p.tv : &p.tk, hk,
                     sq.k0 + (jlo + i / 2) * kTile, kv_full + st);
    };
    if (threadIdx.x == 32 * 10) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(s_full + i, 1);
            mbar_init(s_free + i, 4);
            mbar_init(p_full + i, 4);
            mbar_init(pv_done + i, 1);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(kv_full + i, 1);
            mbar_init(kv_empty + i, 1);
        }
        mbar_init(tail_bar, 1);
        fence_barrier_init();
        for (int t = 0; t < 2; ++t)
            if (hi[t] > lo[t]) {
                mbar_arrive_expect_tx(q_full + t, SM::kTileBytes);
                load_tile<D>(sm + t * SM::kTileBytes, &p.tq, h + t * dh, sq.q0 + (qt + t * dt) * kTile, q_full + t);
                if (t == 0 || !on0) load(0);
            }
    }
    if (warp == 8) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // columns: scores (one place for both tiles at D = 128, else one each), weights, sums
    constexpr int SLOTS = D == 128 ? 1 : 2;
    const uint32_t tS[2] = {tmem, tmem + (SLOTS - 1) * 128u};
    const uint32_t tP[2] = {tmem + SLOTS * 128u, tmem + SLOTS * 128u + 64u};
    const uint32_t tO[2] = {tmem + SLOTS * 128u + 128u, tmem + SLOTS * 128u + 128u + (uint32_t)D};
    bool bad = false;

    if (warp == 10) {
        // ---------------------------------------------------------------- loads
        for (int i = 1; i < loads; ++i) {  // the first is on its way
            const int st = i % NS, j = jlo + i / 2;
            if (i >= NS) {
                const bool ok = mbar_wait(kv_empty + st, (i / NS - 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    bad = true;
                    break;
                }
            }
            unsigned char* dst = sm + SM::kRing + st * SM::kTileBytes;
            const int rows = sq.lk - j * kTile;
            // The value rows behind the sequence's last key belong to another sequence or to
            // nobody: their weight is zero, which a NaN or an infinity there would survive.
            const bool tail = (i & 1) && rows < kTile;
            if (lane == 0 && !tail) load(i);
            if (tail) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(tail_bar, SM::kTileBytes);
                    load_tile<D>(dst, &p.tv, hk, sq.k0 + j * kTile, tail_bar);
                }
                __syncwarp();
                const bool ok = mbar_wait(tail_bar, 0);
                if (!__all_sync(0xffffffffu, ok)) {
                    bad = true;
                    break;
                }
                zero_rows<D>(dst, rows);
                if (lane == 0) mbar_arrive(kv_full + st);
            }
        }
        if (bad && lane == 0) atomicOr(&g_fwd_timeouts, 1u);
    } else if (warp == 8) {
        // ---------------------------------------------------------------- scores
        // Step j of tile 0, of tile 1, step j + 1 of tile 0, ...: the order in which the
        // tiles, half a step apart, come to need them.
        if (lane == 0) {
            constexpr uint32_t id_s = idesc(kBF16, 128, 128, false, false);
            int n = 0;  // score products issued
            for (int j = jlo; j < jhi && !bad; ++j) {
                const int i = 2 * (j - jlo), st = i % NS;
                const uint32_t b = saddr(sm + SM::kRing + st * SM::kTileBytes);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (j < lo[t] || j >= hi[t]) continue;
                    bool ok = mbar_wait(kv_full + st, (i / NS) & 1);
                    if (j == lo[t]) ok = ok && mbar_wait(q_full + t, 0);
                    // the place is free once the scores before have been read from it
                    if (SLOTS == 1) ok = ok && (n == 0 || mbar_wait(s_free, (n - 1) & 1));
                    else ok = ok && (j == lo[t] || mbar_wait(s_free + t, (j - 1 - lo[t]) & 1));
                    if (!ok) {
                        bad = true;
                        break;
                    }
                    ++n;
                    tc_fence_after();
                    const uint32_t a = saddr(sm + t * SM::kTileBytes);
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        mma_f16(tS[t], kdesc16(a, 0, k), kdesc16(b, 0, k), id_s, k ? 1u : 0u);
                    mma_commit(s_full + t);
                    // the last tile that needs these keys gives their place back
                    if ((t == 1 || j < lo[1] || j >= hi[1]) && i + NS < loads) mma_commit(kv_empty + st);
                }
            }
            if (bad) atomicOr(&g_fwd_timeouts, 2u);
        }
    } else if (warp == 9) {
        // ---------------------------------------------------------------- weights times values
        // A warp of its own: the tensor cores have work while either warp waits for its next.
        if (lane == 0) {
            constexpr uint32_t id_o = idesc(kBF16, 128, D, false, true);
            for (int j = jlo; j < jhi && !bad; ++j) {
                const int i = 2 * (j - jlo) + 1, st = i % NS;
                const uint32_t b = saddr(sm + SM::kRing + st * SM::kTileBytes);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (j < lo[t] || j >= hi[t]) continue;
                    if (!mbar_wait(kv_full + st, (i / NS) & 1) || !mbar_wait(p_full + t, (j - lo[t]) & 1)) {
                        bad = true;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < kTile; k += 16)
                        mma_f16_ta(tO[t], tP[t] + k / 2, mdesc16(b, k, 0), id_o, (j > lo[t] || k) ? 1u : 0u);
                    if ((t == 1 || j < lo[1] || j >= hi[1]) && i + NS < loads) mma_commit(kv_empty + st);
                    mma_commit(pv_done + t);
                }
            }
            if (bad) atomicOr(&g_fwd_timeouts, 8u);
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const int t = warp >> 2;
        const int row = (qt + t * dt) * kTile + (threadIdx.x & 127);  // of the sequence
        const uint32_t lane0 = (uint32_t)(warp & 3) << 21;           // this warp's TMEM lanes
        const int at = row + off;
        const int kmax = p.causal ? min(sq.lk - 1, at) : sq.lk - 1;  // visible keys [kmin, kmax]
        const int kmin = p.window ? at - p.window + 1 : 0;
        // of the tile's first and last row: which key tiles need no mask
        const int r0 = (qt + t * dt) * kTile;
        const int all_max = p.causal ? min(sq.lk - 1, r0 + off) : sq.lk - 1;
        const int all_min = p.window ? r0 + kTile - 1 + off - p.window + 1 : 0;
        float m = -INFINITY, l = 0.f;  // m in units of score * scale * log2 e
        const float c = p.scale_log2;

        for (int j = lo[t]; j < hi[t]; ++j) {
            const bool ok = mbar_wait(s_full + t, (j - lo[t]) & 1);
            if (!__all_sync(0xffffffffu, ok)) {
                bad = true;
                break;
            }
            tc_fence_after();
            float s[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32(tS[t] + lane0 + 32 * i, s[i]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free + (SLOTS == 1 ? 0 : t));
            const int k0 = j * kTile;
            if (k0 + kTile - 1 > all_max || k0 < all_min) {
                const int a = kmin - k0, b = kmax - k0;
#pragma unroll
                for (int i = 0; i < 4; ++i) hide(s[i], visible32(a - 32 * i, b - 32 * i));
            }
            float mx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mx[i] = fmaxf(s[i][0], s[i][1]);
#pragma unroll
                for (int x = 2; x < 32; x += 2) mx[i] = fmaxf(mx[i], fmaxf(s[i][x], s[i][x + 1]));
            }
            // largest s * c: the scale may be negative or zero only with the smallest s, so
            // the callers' scale is required to be positive
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            const bool grow = top > m + kSlack || (m == -INFINITY && top > -INFINITY);
            // the sums and the weights' place are the threads' once the step before is done
            if (j > lo[t]) {
                const bool done = mbar_wait(pv_done + t, (j - 1 - lo[t]) & 1);
                if (!__all_sync(0xffffffffu, done)) {
                    bad = true;
                    break;
                }
                tc_fence_after();
            }
            if (__any_sync(0xffffffffu, grow)) {
                const float mn = fmaxf(m, top);
                const float a = mn == -INFINITY ? 1.f : ex2(m - mn);
                m = mn;
                l *= a;
                if (j > lo[t]) {
#pragma unroll
                    for (int x = 0; x < D; x += 16) {
                        float o[16];
                        tmem_ld16(tO[t] + lane0 + x, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= a;
                        tmem_st16(tO[t] + lane0 + x, o);
                    }
                }
            }
            const float neg = m == -INFINITY ? 0.f : -m;
            const uint64_t c2 = pack2(c, c), neg2 = pack2(neg, neg);
            uint64_t sum[2] = {0, 0};  // of even and odd columns, twice
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t w[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    const float* v = &s[2 * i + (x >> 4)][(2 * x) & 31];
                    float e0, e1;
                    unpack2(fma2(pack2(v[0], v[1]), c2, neg2), e0, e1);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    sum[x & 1] = add2(sum[x & 1], pack2(e0, e1));
                    w[x] = bf16x2(e0, e1);
                }
                tmem_st32u(tP[t] + lane0 + 32 * i, w);
            }
            float even, odd;
            unpack2(add2(sum[0], sum[1]), even, odd);
            l += even + odd;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + t);
        }

        // ---- the row's sum, scaled; through the tile's query rows (no product reads them any more)
        const int steps = hi[t] - lo[t];
        if (steps > 0 && !bad) {
            const bool ok = mbar_wait(pv_done + t, (steps - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) bad = true;
            tc_fence_after();
        }
        if (bad && lane == 0) atomicOr(&g_fwd_timeouts, 4u);
        const float inv = l == 0.f ? 0.f : 1.f / l;  // no key seen: zero; a NaN stays
        if (row < sq.lq && t < p.tiles)
            p.lse[sq.q0 * p.lse_seq + (h + t * dh) * p.lse_head + row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
        store_rows<D>(tO[t], inv, steps > 0, sm + t * SM::kTileBytes,
                      p.o + ((long long)(sq.q0 + (qt + t * dt) * kTile) * p.Hq + h + t * dh) * D, (long long)p.Hq * D,
                      t < p.tiles ? sq.lq - (qt + t * dt) * kTile : 0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch(const FwdParams& a, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t err = allow_smem(k_attn_fwd<D>, FwdSmem<D>::kBytes, done);
    if (err != cudaSuccess) return err;
    MUIR_TIMED("k_attn_fwd", st, k_attn_fwd<D><<<block_grid(a.by_heads ? a.Hq / 2 : a.Hq, a.blocks), kThreads, FwdSmem<D>::kBytes, st>>>(a));
    return cudaGetLastError();
}

}  // namespace

int gather_seqs(const Problem& p, int first, int last, bool by_keys, int rows_per_block, Seq* out,
                long long* blocks) {
    int n = 0;
    for (int i = first; i < last; ++i) {
        const Seq s = p.seq(i);
        if ((by_keys ? s.lk : s.lq) > 0) out[n++] = s;
    }
    std::sort(out, out + n, [by_keys](const Seq& x, const Seq& y) {
        const int lx = by_keys ? x.lk : x.lq, ly = by_keys ? y.lk : y.lq;
        return lx != ly ? lx > ly : x.q0 < y.q0;
    });
    for (int k = 0; k < n; ++k)
        out[k].blocks = ((by_keys ? out[k].lk : out[k].lq) + rows_per_block - 1) / rows_per_block;
    long long total = 0;
    for (int k = 0; k < n; ++k) {
        out[k].block0 = (int)total;
        total += (long long)(k + 1) * (out[k].blocks - (k + 1 < n ? out[k + 1].blocks : 0));
    }
    *blocks = total;
    return n;
}

cudaError_t run_fwd(const Problem& p, void* o, float* lse, cudaStream_t st) {
    FwdParams a;
    if (p.q_rows == 0) return cudaSuccess;
    cudaError_t err = make_tmap_tokens(&a.tq, p.q, p.d, p.Hq, p.q_ld, p.q_rows, kTile);
    if (err == cudaSuccess && p.k_rows > 0) err = make_tmap_tokens(&a.tk, p.k, p.d, p.Hk, p.k_ld, p.k_rows, kTile);
    if (err == cudaSuccess && p.k_rows > 0) err = make_tmap_tokens(&a.tv, p.v, p.d, p.Hk, p.v_ld, p.k_rows, kTile);
    if (err != cudaSuccess) return err;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.lse_seq = p.lse_seq;
    a.lse_head = p.lse_head;
    a.scale_log2 = p.scale * kLog2e;
    a.Hq = p.Hq; a.inv_group = (float)p.Hk / (float)p.Hq; a.causal = p.causal; a.window = p.window;
    for (int i = 0; i < p.n; i += kMaxSeqs) {
        long long blocks;
        const int last = std::min(i + kMaxSeqs, p.n);
        // Two heads of a group where groups are even: they see the same keys, and a sequence's
        // last rows fill half of a tile at worst, not of two (packed documents of 1 to 3331
        // tokens, 16 heads over 4: 97 -> 89 us).
        a.by_heads = (p.Hq / p.Hk) % 2 == 0;
        a.tiles = 2;
        a.n = gather_seqs(p, i, last, false, a.by_heads ? kTile : 2 * kTile, a.seq, &blocks);
        if (a.n == 0) continue;
        // One tile a block where two leave SMs without a block: 256 tokens of 2 heads of 128
        // 11.6 -> 8.3 us, 1024 tokens 21.2 -> 16.8.
        if (blocks * (a.by_heads ? p.Hq / 2 : p.Hq) < kSMs) {
            a.by_heads = 0;
            a.tiles = 1;
            a.n = gather_seqs(p, i, last, false, kTile, a.seq, &blocks);
        }
        a.blocks = (int)blocks;
        err = p.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

unsigned int timeouts_fwd() {
    unsigned int n = 0;
    cudaMemcpyFromSymbol(&n, g_fwd_timeouts, sizeof(n));
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_fwd_timeouts, &z, sizeof(z));
    return n;
}

}  // namespace attn
}  // namespace muir
