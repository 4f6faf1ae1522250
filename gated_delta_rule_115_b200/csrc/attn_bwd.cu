// attn_bwd.cu -- softmax attention, backward, on tcgen05.
//
//     p_ij  = exp(s_ij - lse_i)                       (recomputed; s_ij = scale q_i . k_j)
//     dv_j  = sum_i p_ij dO_i
//     ds_ij = p_ij (dO_i . v_j - D_i),                D_i = dO_i . o_i
//     dq_i  = scale sum_j ds_ij k_j,     dk_j = scale sum_i ds_ij q_i
//
// D first; then two kinds of blocks: for dk and dv, a block owning 128 keys of one key head
// and walking the queries of its group's heads; for dq, one owning 128 queries and walking
// the keys.
// Each sum is therefore formed by one block, in tensor memory, in a fixed order: no atomics,
// no float32 gradient buffers, and shared key heads need no second pass.  The price is that
// the scores and dO . v are formed twice (7 products a pair of tiles, where 5 would do if dq
// were scattered).
//
// In both kinds, tensor memory holds the scores of a step (S, 128 columns), dO . v (P, 128) and the
// sums.  Eight warps take a row and 64 of the 128 columns a thread, turn the scores into p and
// the pair into ds, and write them, rounded to bf16 (half a step, 2^-8), over the columns of S
// that they have read, where they are the A operand of the products that follow.
//
//   warps 0-3, 4-7 : p and ds of columns 0-63, 64-127
//   warps 8, 9, 10 : issue S, P, and the sums' products; a warp each, so that the tensor
//                    cores have work while one waits for its next operands
//   warp 11        : loads (TMA)
//
// Bound by the tensor cores (14 d flops a visible pair here) with the exponentials close
// behind (2 a pair, 16 a clock and SM).  Causal, 2 x 8192 tokens of 8 heads of 128: 0.74 ms, 1.30
// PFLOP/s; 8192 tokens of 8 heads of 64: 0.25 ms, 0.98 PFLOP/s.
#include <algorithm>

#include "attn_dev.cuh"
#include "profile.h"
#include "tmap.h"

namespace muir {
namespace attn {

__device__ unsigned int g_bwd_timeouts;

namespace {

constexpr int kThreads = 384;
constexpr int kSMs = 148;
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
    CUtensorMap tq, tk, tv, tdo;
    const float *lse, *delta, *few;
    __nv_bfloat16 *dq, *dk, *dv;
    long long lse_seq, lse_head;
    float scale, scale_log2;
    int Hq, Hk, group, causal, window;
    int dq_heads;                      // query heads of a block of dq: 1, or (d = 64) 2 of a group
    int kv_blocks, q_blocks, n_kv, n_q;
    Seq kv[kMaxSeqs], q[kMaxSeqs];     // the sequences in blocks of keys, and of queries
};

// ------------------------------------------------------------------ D = dO . o

// D enters every ds of its row, so an error of it does not average out over the keys as the
// roundings of p do.  From the o that the forward pass rounded to bf16 it is off by up to
// 2^-8 sum |dO||o|, which matters where few keys share a row's weight (|o| is then as large
// as |v|): two visible keys leave 0.0038 in dq where everything else leaves 0.0023, sixteen
// 0.0029.  Rows of up to kFewKeys keys take D = sum_j p_j dO . v_j instead, in float32.
constexpr int kFewKeys = 8;
constexpr int kDeltaRows = 4;  // of a lane, all in flight together

struct DeltaParams {
    const __nv_bfloat16 *o, *dO, *q, *k, *v;
    long long q_ld, k_ld, v_ld;
    const float* lse;
    float *delta, *few;  // D = dO . o of every row; D of the rows of few keys, at the same places
    long long lse_seq, lse_head;
    float scale_log2, inv_group;
    int Hq, T, causal, window;
    int release;         // the next kernel's blocks may start beside these
    long long rows;      // (token, head) pairs
    int few_blocks, few_rows;
    int n;               // sequences with rows of few keys
    struct {
        int q0, lq, k0, lk, first, row0;  // their first such row, and how many come before it
    } seq[kMaxSeqs];
};

// How many of a sequence's lk keys the query at key position `at` sees.
__device__ __forceinline__ int keys_seen(int causal, int window, int lk, int at) {
    const int last = causal ? min(lk - 1, at) : lk - 1, first = window ? max(0, at - window + 1) : 0;
    return max(0, last - first + 1);
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
    unpack16<true>(u.x, v[0], v[1]);
    unpack16<true>(u.y, v[2], v[3]);
    unpack16<true>(u.z, v[4], v[5]);
    unpack16<true>(u.w, v[6], v[7]);
}
__device__ __forceinline__ void unpack8(const __nv_bfloat16* p, float (&v)[8]) {
    unpack8(*reinterpret_cast<const uint4*>(p), v);
}

// A row (token, head) of D channels is D / 8 lanes.  The first blocks take the rows of few
// keys, beside the others, which read o and dO once and are bound by HBM (2 x 8192 tokens of 8
// heads of 128, 67 MB: about 15 us).
template <int D>
__global__ void __launch_bounds__(256, 4) k_attn_delta(const __grid_constant__ DeltaParams p) {
    constexpr int G = D / 8, RPW = 32 / G;
    if (p.release) grid_release();
    const int lane = threadIdx.x & 31, sub = (threadIdx.x >> 5) * RPW + lane / G, ch = (lane % G) * 8;
    auto row_sum = [](float s) {
#pragma unroll
        for (int off = G / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        return s;
    };
    if ((int)blockIdx.x < p.few_blocks) {
        const long long r = (long long)blockIdx.x * (8 * RPW) + sub, x = r / p.Hq;
        const bool on = x < p.few_rows;
        const int h = (int)(r - x * p.Hq), hk = key_head(h, p.inv_group);
        int lo = 0, hi = p.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.seq[mid].row0 <= (int)x) lo = mid;
            else hi = mid - 1;
        }
        const int pos = on ? p.seq[lo].first + (int)x - p.seq[lo].row0 : 0;
        const int at = pos + p.seq[lo].lk - p.seq[lo].lq;
        const int seen = on ? keys_seen(p.causal, p.window, p.seq[lo].lk, at) : 0;
        const bool few = seen > 1 && seen <= kFewKeys;
        const long long tok = p.seq[lo].q0 + pos, out = p.seq[lo].q0 * p.lse_seq + h * p.lse_head + pos;
        const long long key = p.seq[lo].k0 + (p.window ? max(0, at - p.window + 1) : 0);
        float q[8] = {}, g[8] = {}, e = 0.f, sum = 0.f;
        if (few) {
            unpack8(p.q + tok * p.q_ld + h * D + ch, q);
            unpack8(p.dO + (tok * p.Hq + h) * D + ch, g);
            e = p.lse[out] * kLog2e;
        }
#pragma unroll 4
        for (int j = 0; j < kFewKeys; ++j) {
            float sc = 0.f, dp = 0.f;
            if (few && j < seen) {
                float k[8], v[8];
                unpack8(p.k + (key + j) * p.k_ld + hk * D + ch, k);
                unpack8(p.v + (key + j) * p.v_ld + hk * D + ch, v);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    sc += q[c] * k[c];
                    dp += g[c] * v[c];
                }
            }
            sc = row_sum(sc);
            dp = row_sum(dp);
            if (few && j < seen) sum += ex2(sc * p.scale_log2 - e) * dp;
        }
        if (few && lane % G == 0) p.few[out] = sum;
        return;
    }
    const long long r0 = (long long)(blockIdx.x - p.few_blocks) * (8 * RPW * kDeltaRows) + sub;
    uint4 x[kDeltaRows], y[kDeltaRows];
#pragma unroll
    for (int n = 0; n < kDeltaRows; ++n) {
        const long long r = r0 + n * 8 * RPW;
        x[n] = y[n] = make_uint4(0u, 0u, 0u, 0u);
        if (r < p.rows) {
            x[n] = *reinterpret_cast<const uint4*>(p.o + r * D + ch);
            y[n] = *reinterpret_cast<const uint4*>(p.dO + r * D + ch);
        }
    }
#pragma unroll
    for (int n = 0; n < kDeltaRows; ++n) {
        const long long r = r0 + n * 8 * RPW;
        float a[8], b[8], s = 0.f;
        unpack8(x[n], a);
        unpack8(y[n], b);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += a[i] * b[i];
        s = row_sum(s);
        if (r < p.rows && lane % G == 0) {
            // token-major rows -> the layout of lse
            const long long tok = r / p.Hq;
            const int h = (int)(r - tok * p.Hq);
            const long long at = p.lse_seq == 1 ? 0 : tok / p.T;
            p.delta[at * p.T * p.lse_seq + h * p.lse_head + (tok - at * p.T)] = s;
        }
    }
}

// ------------------------------------------------------------------ dk, dv

template <int D>
struct DkvSmem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 2 : 4;                   // pairs of query and dO tiles
    static constexpr int kRing = 2 * kTileBytes;                       // after the two resident tiles
    static constexpr int kVec = kRing + kStages * 2 * kTileBytes;      // -lse log2 e and -D of a stage's rows
    static constexpr int kBars = kVec + kStages * 2 * kTile * 4;
    static constexpr int kBytes = kBars + 512;
};

// Whole-warp bounded wait.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}

// Loads one pair of tiles (rows `rows` of 128 belong to the sequence) into a stage: both
// tiles count on `full`, once the rows behind the sequence's end are zero (their weight is
// zero, which a NaN or an infinity of a neighbouring sequence would survive).  The second of
// full's two arrivals is the caller's.  One warp; false if a wait ran out.
template <int D>
__device__ __forceinline__ bool load_pair(unsigned char* dst, const CUtensorMap* ma, const CUtensorMap* mb,
                                          int head, int token, int rows, uint64_t* full, uint64_t* tail_bar,
                                          uint32_t& tail_phase) {
    constexpr int TB = kTile * D * 2;
    const bool tail = rows < kTile;
    uint64_t* bar = tail ? tail_bar : full;
    if ((threadIdx.x & 31) == 0) {
        mbar_arrive_expect_tx(bar, 2 * TB);
        load_tile<D>(dst, ma, head, token, bar);
        load_tile<D>(dst + TB, mb, head, token, bar);
    }
    __syncwarp();
    if (tail) {
        if (!warp_wait(tail_bar, tail_phase & 1)) return false;
        ++tail_phase;
        zero_rows<D>(dst, rows);
        zero_rows<D>(dst + TB, rows);
        if ((threadIdx.x & 31) == 0) mbar_arrive(full);
    }
    return true;
}

template <int NS>
struct DkvBars {
    uint64_t res_full, res_tmem;       // the resident tiles; in tensor memory too
    uint64_t full[NS], empty[NS], tail;
    // of each half of the columns:
    uint64_t s_full[2], dp_full[2];             // its products of a step in tensor memory
    // Four warps: p written (of even, of odd steps: a half may write its next p before the
    // other lets the sums' warp come to this one, and a barrier two phases on looks as if it
    // had not moved), P read, ds written.
    uint64_t p_full[4], dp_read[2], ds_full[2];
    uint64_t acc_done[2];                       // its last product of a step
    uint64_t final_done;
    uint32_t tmem_slot;
};

// dk and dv of 128 keys of one key head: rows of the products are keys, columns queries.
//
// The 128 queries of a step are two halves of 64 that go their own ways, each with its four
// warps, its barriers and 128 columns: its S in 64 of them, its P in the other 64; p and ds
// overwrite S, and the next step's S goes to where P was as soon as P has been read.  The
// halves drift half a step apart, so that one's exponentials run beside the other's products
// (as one whole of 128 columns, each step waited for its own scores and its own exponentials
// in turn: 3400 clocks a step, of which the tensor cores ran 2550).
template <int D>
__device__ __forceinline__ void dkv_block(const BwdParams& p, unsigned char* sm, int blk, int hk) {
    using SM = DkvSmem<D>;
    constexpr int NS = SM::kStages;
    DkvBars<NS>* bar = reinterpret_cast<DkvBars<NS>*>(sm + SM::kBars);
    static_assert(sizeof(DkvBars<NS>) <= SM::kBytes - SM::kBars, "barriers");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Place place = place_of(p.kv, p.n_kv, blk);
    const Seq sq = place.sq;
    const int kb = sq.blocks - 1 - place.rank;  // with a causal mask the first keys are seen most
    const int G = p.group;
    const int off = sq.lk - sq.lq;
    const int k0 = kb * kTile;

    // query tiles [lo, hi) that see any of the block's keys, for each head of the group
    int lo = 0, hi = (sq.lq + kTile - 1) / kTile;
    if (p.causal) lo = max(0, k0 - off) / kTile;
    if (p.window) {
        const int last = min(k0 + kTile, sq.lk) - 1 + p.window - off - 1;
        hi = last < 0 ? 0 : min(hi, last / kTile + 1);
    }
    const int per = max(0, hi - lo), steps = per * G;

    // The loading warp sets the barriers up and sends the resident tiles off before the block
    // meets: they take longer than everything else that comes before the first product.
    if (threadIdx.x == 32 * 11) {
        mbar_init(&bar->res_full, 1);
        mbar_init(&bar->res_tmem, 8);
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar->full + i, 2);
            mbar_init(bar->empty + i, 1);
        }
        mbar_init(&bar->tail, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar->s_full + i, 1);
            mbar_init(bar->dp_full + i, 1);
            mbar_init(bar->p_full + i, 4);
            mbar_init(bar->p_full + 2 + i, 4);
            mbar_init(bar->dp_read + i, 4);
            mbar_init(bar->ds_full + i, 4);
            mbar_init(bar->acc_done + i, 1);
        }
        mbar_init(&bar->final_done, 1);
        fence_barrier_init();
        if (steps > 0) {
            mbar_arrive_expect_tx(&bar->res_full, 2 * SM::kTileBytes);
            load_tile<D>(sm, &p.tk, hk, sq.k0 + k0, &bar->res_full);
            load_tile<D>(sm + SM::kTileBytes, &p.tv, hk, sq.k0 + k0, &bar->res_full);
        }
    }
    if (warp == 8) tmem_alloc(&bar->tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_slot;
    const uint32_t tV = tmem + 256u, tK = tmem + 256u + (uint32_t)D;
    // At D = 64 there is room for the resident tiles beside the sums, K in 32 columns and V in the
    // next: as operands they are then no part of what the products fetch from shared memory,
    // which for 64 columns a product is more than the tensor cores keep up with (8192 tokens, 8
    // heads: 254 -> 250 us; 8 over 2: 312 -> 300).
    constexpr bool RES = D == 64;
    const uint32_t tRes = tmem + 384u;
    float* vec = reinterpret_cast<float*>(sm + SM::kVec);

    if (warp == 11) {
        // ---------------------------------------------------------------- loads
        bool ok = true;
        uint32_t tails = 0;
        int tile = 0, head = 0;  // of step i
        grid_wait();             // for D
        for (int i = 0; i < steps && ok; ++i) {
            const int st = i % NS, i0 = (lo + tile) * kTile;
            const int h = hk * G + head;
            if (++tile == per) {
                tile = 0;
                ++head;
            }
            // -lse log2 e and -D of the tile's queries; -infinity (no weight at all) for rows
            // that do not exist and for queries that see no key; asked for before the stage is free
            const long long at = sq.q0 * p.lse_seq + h * p.lse_head + i0;
            const bool any_few = (p.window && p.window <= kFewKeys) || sq.lk <= kFewKeys ||
                                 (p.causal && i0 + off < kFewKeys);
            float e[kTile / 32], dd[kTile / 32];
#pragma unroll
            for (int n = 0; n < kTile / 32; ++n) {
                const int x = lane + 32 * n;
                const bool on = i0 + x < sq.lq;
                const float* from = p.delta;
                if (any_few && keys_seen(p.causal, p.window, sq.lk, i0 + x + off) <= kFewKeys) from = p.few;
                e[n] = on ? p.lse[at + x] : -INFINITY;
                dd[n] = on ? from[at + x] : 0.f;
            }
            if (i >= NS) ok = warp_wait(bar->empty + st, (i / NS - 1) & 1);
            if (!ok) break;
            ok = load_pair<D>(sm + SM::kRing + st * 2 * SM::kTileBytes, &p.tq, &p.tdo, h, sq.q0 + i0, sq.lq - i0,
                              bar->full + st, &bar->tail, tails);
            float* v = vec + st * 2 * kTile;
#pragma unroll
            for (int n = 0; n < kTile / 32; ++n) {
                const int x = lane + 32 * n;
                // of one key or none: ds is zero, and D has not been formed
                if (any_few && keys_seen(p.causal, p.window, sq.lk, i0 + x + off) <= 1) dd[n] = 0.f;
                v[x] = e[n] == -INFINITY ? -INFINITY : -e[n] * kLog2e;
                v[kTile + x] = -dd[n];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar->full + st);
        }
        if (!ok && lane == 0) atomicOr(&g_bwd_timeouts, 1u);
    } else if (warp >= 8) {
        // ---------------------------------------------------------------- products
        constexpr uint32_t id_s = idesc(kBF16, 128, 64, false, false);
        constexpr uint32_t id_a = idesc(kBF16, 128, D, false, true);
        bool ok = true;
        if (lane != 0 || steps == 0) {
        } else if (warp == 8) {  // S = K Q^T
            ok = mbar_wait(RES ? &bar->res_tmem : &bar->res_full, 0);
            const uint32_t a = saddr(sm);
            for (int j = 0; j < steps && ok; ++j) {
                const uint32_t b = saddr(sm + SM::kRing + (j % NS) * 2 * SM::kTileBytes);
                ok = mbar_wait(bar->full + j % NS, (j / NS) & 1);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    ok = ok && (j == 0 || mbar_wait(bar->dp_read + u, (j - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + 128u * u + (uint32_t)(j & 1) * 64u;
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        if (RES) mma_f16_ta(d, tRes + k / 2, kdesc16(b, 64 * u, k), id_s, k ? 1u : 0u);
                        else mma_f16(d, kdesc16(a, 0, k), kdesc16(b, 64 * u, k), id_s, k ? 1u : 0u);
                    mma_commit(bar->s_full + u);
                }
            }
        } else if (warp == 9) {  // P = V dO^T, where the step before kept p and ds
            ok = mbar_wait(RES ? &bar->res_tmem : &bar->res_full, 0);
            const uint32_t a = saddr(sm + SM::kTileBytes);
            for (int j = 0; j < steps && ok; ++j) {
                const uint32_t b = saddr(sm + SM::kRing + (j % NS) * 2 * SM::kTileBytes + SM::kTileBytes);
                ok = mbar_wait(bar->full + j % NS, (j / NS) & 1);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    ok = ok && (j == 0 || mbar_wait(bar->acc_done + u, (j - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + 128u * u + (uint32_t)(1 - (j & 1)) * 64u;
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        if (RES) mma_f16_ta(d, tRes + 32 + k / 2, kdesc16(b, 64 * u, k), id_s, k ? 1u : 0u);
                        else mma_f16(d, kdesc16(a, 0, k), kdesc16(b, 64 * u, k), id_s, k ? 1u : 0u);
                    mma_commit(bar->dp_full + u);
                }
            }
        } else {  // dv += p^T dO, dk += ds^T Q
            for (int j = 0; j < steps && ok; ++j) {
                const uint32_t q = saddr(sm + SM::kRing + (j % NS) * 2 * SM::kTileBytes), g = q + SM::kTileBytes;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t x = tmem + 128u * u + (uint32_t)(j & 1) * 64u;
                    ok = ok && mbar_wait(bar->p_full + 2 * u + (j & 1), (j >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 64; k += 16)  // p: the first 32 columns of S
                        mma_f16_ta(tV, x + k / 2, mdesc16(g, 64 * u + k, 0), id_a, (j || u || k) ? 1u : 0u);
                    ok = mbar_wait(bar->ds_full + u, j & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 64; k += 16)  // ds: the others
                        mma_f16_ta(tK, x + 32 + k / 2, mdesc16(q, 64 * u + k, 0), id_a, (j || u || k) ? 1u : 0u);
                    // the step's S and P are long done: p and ds were made of them
                    if (u == 1 && j + NS < steps) mma_commit(bar->empty + j % NS);
                    if (j + 1 < steps) mma_commit(bar->acc_done + u);
                }
                if (ok && j + 1 == steps) mma_commit(&bar->final_done);
            }
        }
        if (!ok) atomicOr(&g_bwd_timeouts, 2u);
    } else {
        // ---------------------------------------------------------------- p, ds
        const int wg = warp >> 2;
        const uint32_t lane0 = (uint32_t)(warp & 3) << 21;
        const int key = k0 + (threadIdx.x & 127);  // the thread's row
        const bool all_single = (p.causal && p.window == 1) || sq.lk == 1;  // no query sees two keys
        const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
        bool ok = true;
        if (RES && steps > 0) {
            ok = warp_wait(&bar->res_full, 0);
            const unsigned char* from = sm + wg * SM::kTileBytes;
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(from + t16_off(threadIdx.x & 127, i));
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
            tmem_st32u(tRes + lane0 + 32u * wg, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->res_tmem);
        }
        int tile = 0;  // of step j
        for (int j = 0; j < steps && ok; ++j) {
            const uint32_t x = tmem + lane0 + 128u * wg + (uint32_t)(j & 1) * 64u;
            const uint32_t y = tmem + lane0 + 128u * wg + (uint32_t)(1 - (j & 1)) * 64u;
            const float4* nl = reinterpret_cast<const float4*>(vec + (j % NS) * 2 * kTile + 64 * wg);
            const float4* dl = nl + kTile / 4;
            const int i0 = (lo + tile) * kTile;
            if (++tile == per) tile = 0;
            // the first of the thread's 64 columns that sees its key, and whether some column
            // of the tile does not (causal), or no longer does (window)
            const int sees = key - off - i0 - 64 * wg;
            const bool before = p.causal && i0 + off < k0 + kTile - 1;
            const bool behind = p.window && i0 + kTile - 1 + off - p.window >= k0;
            // the column whose query sees one key only: a causal sequence's first position, or the
            // last one of those that look ahead from their own
            const int single = p.causal ? -off - i0 - 64 * wg : p.window == 1 ? sq.lq - 1 - i0 - 64 * wg : -1;
            ok = warp_wait(bar->s_full + wg, j & 1) && warp_wait(bar->full + j % NS, (j / NS) & 1);
            if (!ok) break;
            tc_fence_after();
            float s[2][32];
            tmem_ld32(x, s[0]);
            tmem_ld32(x + 32, s[1]);
            tmem_wait_ld();
            if (before || behind) {
                const int a = p.causal ? sees : 0, b = p.window ? sees + p.window - 1 : 63;
                hide(s[0], visible32(a, b));
                hide(s[1], visible32(a - 32, b - 32));
            }
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 n = nl[i];
                float* v = &s[i >> 3][(4 * i) & 31];
                unpack2(fma2(pack2(v[0], v[1]), c2, pack2(n.x, n.y)), v[0], v[1]);
                unpack2(fma2(pack2(v[2], v[3]), c2, pack2(n.z, n.w)), v[2], v[3]);
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] = ex2(v[x]);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = bf16x2(s[i >> 4][(2 * i) & 31], s[i >> 4][(2 * i + 1) & 31]);
            tmem_st32u(x, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar->p_full + 2 * wg + (j & 1));

            // A query that sees one key gives it weight 1 whatever their score: ds is zero, where
            // dO . v and D, which are then the same, differ by their roundings.
            if (all_single || (single >= 0 && single < 64)) {
#pragma unroll
                for (int i = 0; i < 64; ++i) s[i >> 5][i & 31] = all_single || i == single ? 0.f : s[i >> 5][i & 31];
            }
            ok = warp_wait(bar->dp_full + wg, j & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int hlf = 0; hlf < 2; ++hlf) {
                float dp[32];
                tmem_ld32(y + 32 * hlf, dp);
                tmem_wait_ld();
                if (hlf) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar->dp_read + wg);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 n = dl[8 * hlf + i];
                    float* v = &s[hlf][4 * i];
                    unpack2(mul2(pack2(v[0], v[1]), add2(pack2(dp[4 * i], dp[4 * i + 1]), pack2(n.x, n.y))), v[0], v[1]);
                    unpack2(mul2(pack2(v[2], v[3]), add2(pack2(dp[4 * i + 2], dp[4 * i + 3]), pack2(n.z, n.w))), v[2],
                            v[3]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) w[16 * hlf + i] = bf16x2(s[hlf][2 * i], s[hlf][2 * i + 1]);
            }
            tmem_st32u(x + 32, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar->ds_full + wg);
        }
        if (steps > 0 && ok) {
            ok = warp_wait(&bar->final_done, 0);
            tc_fence_after();
        }
        if (!ok && lane == 0) atomicOr(&g_bwd_timeouts, 4u);
        const long long ld = (long long)p.Hk * D, at = (long long)(sq.k0 + k0) * ld + hk * D;
        if (wg == 0) store_rows<D>(tK, p.scale, steps > 0, sm, p.dk + at, ld, sq.lk - k0);
        else store_rows<D>(tV, 1.f, steps > 0, sm + SM::kTileBytes, p.dv + at, ld, sq.lk - k0);
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
struct DqSmem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kKeys = D == 128 ? 3 : 4, kVals = D == 128 ? 2 : 4;  // tiles of each ring
    static constexpr int kHeads = D == 128 ? 1 : 2;                    // most heads of a block
    static constexpr int kK = 2 * kHeads * kTileBytes;                 // after the resident tiles
    static constexpr int kV = kK + kKeys * kTileBytes;
    static constexpr int kBars = kV + kVals * kTileBytes;
    static constexpr int kBytes = kBars + 512;
};

template <int NK, int NV>
struct DqBars {
    uint64_t res_full;
    uint64_t k_full[NK], k_empty[NK], v_full[NV], v_empty[NV], tail;
    // of each half of the columns, S, ds and the last product of even and of odd steps:
    uint64_t s_full[4], dp_full[2];    // products of a step in tensor memory
    uint64_t dp_read[2], ds_full[4];   // four warps: P read, ds written
    uint64_t acc_done[4];
    uint64_t final_done;
    uint32_t tmem_slot;
};

// dq of 128 queries of one head: rows of the products are queries, columns keys, in two halves
// that go their own ways as above.  The scores alternate between two places, so that a step's
// are formed while the step before is still at its exponentials.
//
// At D = 64 there is room for the tiles and the sums of two heads: a block of two heads of a
// group takes each key tile for the one and then for the other, and its start and its end,
// which cost as much as four steps, serve both.
template <int D>
__device__ __forceinline__ void dq_block(const BwdParams& p, unsigned char* sm, int blk, int h, int hk) {
    const int sh = DqSmem<D>::kHeads == 1 ? 0 : p.dq_heads - 1;  // heads 1 << sh: h and h + sh
    using SM = DqSmem<D>;
    constexpr int NK = SM::kKeys, NV = SM::kVals;
    DqBars<NK, NV>* bar = reinterpret_cast<DqBars<NK, NV>*>(sm + SM::kBars);
    static_assert(sizeof(DqBars<NK, NV>) <= SM::kBytes - SM::kBars, "barriers");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Place place = place_of(p.q, p.n_q, blk);
    const Seq sq = place.sq;
    const int qb = place.rank;
    const int off = sq.lk - sq.lq;
    const int r0 = qb * kTile, r1 = min(r0 + kTile, sq.lq) - 1;

    int last = sq.lk - 1, first = 0;
    if (p.causal) last = min(last, r1 + off);
    if (p.window) first = max(first, r0 + off - p.window + 1);
    const int lo = first / kTile;
    const int tiles = last < first ? 0 : last / kTile + 1 - lo;
    const int steps = tiles << sh;  // step i: key tile i >> sh, head h + (i & sh)

    if (threadIdx.x == 32 * 11) {  // as above
        mbar_init(&bar->res_full, 1);
        for (int i = 0; i < NK; ++i) {
            mbar_init(bar->k_full + i, 1);
            mbar_init(bar->k_empty + i, 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(bar->v_full + i, 1);
            mbar_init(bar->v_empty + i, 1);
        }
        mbar_init(&bar->tail, 2);
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar->s_full + i, 1);
            mbar_init(bar->ds_full + i, 4);
            mbar_init(bar->acc_done + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar->dp_full + i, 1);
            mbar_init(bar->dp_read + i, 4);
        }
        mbar_init(&bar->final_done, 1);
        fence_barrier_init();
        if (steps > 0) {
            mbar_arrive_expect_tx(&bar->res_full, (2 * SM::kTileBytes) << sh);
            for (int n = 0; n <= sh; ++n) {
                load_tile<D>(sm + 2 * n * SM::kTileBytes, &p.tq, h + n, sq.q0 + r0, &bar->res_full);
                load_tile<D>(sm + (2 * n + 1) * SM::kTileBytes, &p.tdo, h + n, sq.q0 + r0, &bar->res_full);
            }
        }
    }
    if (warp == 8) tmem_alloc(&bar->tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_slot;
    const uint32_t tP = tmem + 256u, tQ = tmem + 384u;

    if (warp == 11) {
        // ---------------------------------------------------------------- loads
        bool ok = true;
        for (int i = 0; i < tiles && ok; ++i) {
            const int j0 = (lo + i) * kTile, rows = sq.lk - j0;
            const int ks = i % NK, vs = i % NV;
            if (i >= NK) ok = warp_wait(bar->k_empty + ks, (i / NK - 1) & 1);
            if (!ok) break;
            // Rows behind the sequence's end: their p and ds are zero, which a NaN or an
            // infinity there would survive.
            unsigned char *kd = sm + SM::kK + ks * SM::kTileBytes, *vd = sm + SM::kV + vs * SM::kTileBytes;
            const bool tail = rows < kTile;
            uint64_t *kb = tail ? &bar->tail : bar->k_full + ks, *vb = tail ? &bar->tail : bar->v_full + vs;
            if (lane == 0) {
                mbar_arrive_expect_tx(kb, SM::kTileBytes);
                load_tile<D>(kd, &p.tk, hk, sq.k0 + j0, kb);
            }
            __syncwarp();
            if (i >= NV) ok = warp_wait(bar->v_empty + vs, (i / NV - 1) & 1);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(vb, SM::kTileBytes);
                load_tile<D>(vd, &p.tv, hk, sq.k0 + j0, vb);
            }
            __syncwarp();
            if (tail) {
                ok = warp_wait(&bar->tail, 0);
                if (!ok) break;
                zero_rows<D>(kd, rows);
                zero_rows<D>(vd, rows);
                if (lane == 0) {
                    mbar_arrive(bar->k_full + ks);
                    mbar_arrive(bar->v_full + vs);
                }
            }
        }
        if (!ok && lane == 0) atomicOr(&g_bwd_timeouts, 8u);
    } else if (warp >= 8) {
        // ---------------------------------------------------------------- products
        constexpr uint32_t id_s = idesc(kBF16, 128, 64, false, false);
        constexpr uint32_t id_a = idesc(kBF16, 128, D, false, true);
        bool ok = true;
        if (lane != 0 || steps == 0) {
        } else if (warp == 8) {  // S = Q K^T, where the ds of two steps before was
            ok = mbar_wait(&bar->res_full, 0);
            for (int i = 0; i < steps && ok; ++i) {
                const int j = i >> sh;
                const uint32_t a = saddr(sm + 2 * (i & sh) * SM::kTileBytes);
                const uint32_t b = saddr(sm + SM::kK + (j % NK) * SM::kTileBytes);
                ok = mbar_wait(bar->k_full + j % NK, (j / NK) & 1);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    ok = ok && (i < 2 || mbar_wait(bar->acc_done + 2 * u + (i & 1), ((i - 2) >> 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(i & 1) * 128u + 64u * u;
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        mma_f16(d, kdesc16(a, 0, k), kdesc16(b, 64 * u, k), id_s, k ? 1u : 0u);
                    mma_commit(bar->s_full + 2 * u + (i & 1));
                }
            }
        } else if (warp == 9) {  // P = dO V^T
            ok = mbar_wait(&bar->res_full, 0);
            for (int i = 0; i < steps && ok; ++i) {
                const int j = i >> sh;
                const uint32_t a = saddr(sm + (2 * (i & sh) + 1) * SM::kTileBytes);
                const uint32_t b = saddr(sm + SM::kV + (j % NV) * SM::kTileBytes);
                ok = mbar_wait(bar->v_full + j % NV, (j / NV) & 1);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    ok = ok && (i == 0 || mbar_wait(bar->dp_read + u, (i - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        mma_f16(tP + 64u * u, kdesc16(a, 0, k), kdesc16(b, 64 * u, k), id_s, k ? 1u : 0u);
                    if (u == 1 && (i & sh) == sh && j + NV < tiles) mma_commit(bar->v_empty + j % NV);
                    mma_commit(bar->dp_full + u);
                }
            }
        } else {  // dq += ds K
            for (int i = 0; i < steps && ok; ++i) {
                const int j = i >> sh;
                const uint32_t b = saddr(sm + SM::kK + (j % NK) * SM::kTileBytes);
                const uint32_t d = tQ + (uint32_t)((i & sh) * D);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    ok = ok && mbar_wait(bar->ds_full + 2 * u + (i & 1), (i >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t x = tmem + (uint32_t)(i & 1) * 128u + 64u * u;
#pragma unroll
                    for (int k = 0; k < 64; k += 16)  // ds: the first 32 columns of S
                        mma_f16_ta(d, x + k / 2, mdesc16(b, 64 * u + k, 0), id_a, (j || u || k) ? 1u : 0u);
                    if (u == 1 && (i & sh) == sh && j + NK < tiles) mma_commit(bar->k_empty + j % NK);
                    if (i + 2 < steps) mma_commit(bar->acc_done + 2 * u + (i & 1));
                }
                if (ok && i + 1 == steps) mma_commit(&bar->final_done);
            }
        }
        if (!ok) atomicOr(&g_bwd_timeouts, 16u);
    } else {
        // ---------------------------------------------------------------- p, ds
        const int wg = warp >> 2;
        const uint32_t lane0 = (uint32_t)(warp & 3) << 21;
        const int row = r0 + (threadIdx.x & 127);
        const int at = row + off;
        const int kmax = p.causal ? min(sq.lk - 1, at) : sq.lk - 1;
        const int kmin = p.window ? at - p.window + 1 : 0;
        const int all_max = p.causal ? min(sq.lk - 1, r0 + off) : sq.lk - 1;
        const int all_min = p.window ? r0 + kTile - 1 + off - p.window + 1 : 0;
        // Rows that do not exist and queries that see no key: no weight.  Nor for queries that
        // see one: their ds is zero.
        grid_wait();  // for D
        const int seen = keys_seen(p.causal, p.window, sq.lk, at);
        const bool some = row < sq.lq && seen > 1;
        float nls[2] = {-INFINITY, -INFINITY}, dls[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < SM::kHeads; ++n)
            if (some && n <= sh) {
                const long long v = sq.q0 * p.lse_seq + (h + n) * p.lse_head + row;
                const float e = p.lse[v];
                if (e != -INFINITY) nls[n] = -e * kLog2e;
                dls[n] = (seen <= kFewKeys ? p.few : p.delta)[v];
            }
        const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
        bool ok = true;
        for (int j = 0; j < steps && ok; ++j) {
            const uint32_t x = tmem + lane0 + (uint32_t)(j & 1) * 128u + 64u * wg;
            const int j0 = (lo + (j >> sh)) * kTile;
            const float nl = j & sh ? nls[1] : nls[0], dl = j & sh ? dls[1] : dls[0];
            const uint64_t nl2 = pack2(nl, nl), dl2 = pack2(-dl, -dl);
            const int a = kmin - j0 - 64 * wg, b = kmax - j0 - 64 * wg;  // visible columns [a, b] of the 64
            ok = warp_wait(bar->s_full + 2 * wg + (j & 1), (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            float s[2][32];
            tmem_ld32(x, s[0]);
            tmem_ld32(x + 32, s[1]);
            tmem_wait_ld();
            if (j0 + kTile - 1 > all_max || j0 < all_min) {
                hide(s[0], visible32(a, b));
                hide(s[1], visible32(a - 32, b - 32));
            }
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
                float* v = &s[i >> 5][i & 31];
                unpack2(fma2(pack2(v[0], v[1]), c2, nl2), v[0], v[1]);
                v[0] = ex2(v[0]);
                v[1] = ex2(v[1]);
            }
            ok = warp_wait(bar->dp_full + wg, j & 1);
            if (!ok) break;
            tc_fence_after();
            uint32_t w[32];
#pragma unroll
            for (int hlf = 0; hlf < 2; ++hlf) {
                float dp[32];
                tmem_ld32(tP + lane0 + 64 * wg + 32 * hlf, dp);
                tmem_wait_ld();
                if (hlf) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar->dp_read + wg);
                }
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float* v = &s[hlf][i];
                    unpack2(mul2(pack2(v[0], v[1]), add2(pack2(dp[i], dp[i + 1]), dl2)), v[0], v[1]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) w[16 * hlf + i] = bf16x2(s[hlf][2 * i], s[hlf][2 * i + 1]);
            }
            tmem_st32u(x, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar->ds_full + 2 * wg + (j & 1));
        }
        if (steps > 0 && ok) {
            ok = warp_wait(&bar->final_done, 0);
            tc_fence_after();
        }
        if (!ok && lane == 0) atomicOr(&g_bwd_timeouts, 32u);
        const long long ld = (long long)p.Hq * D;
        __nv_bfloat16* dq = p.dq + (long long)(sq.q0 + r0) * ld + h * D;
        unsigned char* tile = sm + wg * SM::kTileBytes;
        if (sh)  // a head for each four warps
            store_rows<D>(tQ + wg * D, p.scale, steps > 0, tile, dq + wg * D, ld, sq.lq - r0);
        else     // half of the columns
            store_rows<D / 2>(tQ + wg * (D / 2), p.scale, steps > 0, tile, dq + wg * (D / 2), ld, sq.lq - r0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The blocks of dk and dv, then those of dq, in one launch: the second kind fills the SMs
// that the first leaves idle at its end.  Grid (key head, block): kv_blocks blocks of keys,
// then a block of queries for each dq_heads heads of the group in turn.
template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_attn_bwd(const __grid_constant__ BwdParams p) {
    extern __shared__ __align__(1024) unsigned char sm[];
    const int blk = block_index(), hk = blockIdx.x;
    if (blk < p.kv_blocks) {
        dkv_block<D>(p, sm, blk, hk);
    } else {
        const unsigned i = (unsigned)(blk - p.kv_blocks), per = (unsigned)(p.group / p.dq_heads), qblk = i / per;
        if ((int)qblk < p.q_blocks)
            dq_block<D>(p, sm, (int)qblk, hk * p.group + (int)(i - qblk * per) * p.dq_heads, hk);
    }
    grid_wait();  // blocks that needed no D: what follows in the stream may reuse its memory
}

template <int D>
cudaError_t run(const Problem& p, BwdParams& a, const void* o, const void* dO, float* delta, cudaStream_t st) {
    constexpr int kSmem = DkvSmem<D>::kBytes > DqSmem<D>::kBytes ? DkvSmem<D>::kBytes : DqSmem<D>::kBytes;
    static std::atomic<uint64_t> done{0};
    cudaError_t err = allow_smem(k_attn_bwd<D>, kSmem, done);
    if (err != cudaSuccess) return err;
    DeltaParams d;
    d.o = static_cast<const __nv_bfloat16*>(o);
    d.dO = static_cast<const __nv_bfloat16*>(dO);
    d.q = static_cast<const __nv_bfloat16*>(p.q);
    d.k = static_cast<const __nv_bfloat16*>(p.k);
    d.v = static_cast<const __nv_bfloat16*>(p.v);
    d.q_ld = p.q_ld; d.k_ld = p.k_ld; d.v_ld = p.v_ld;
    d.lse = a.lse;
    d.delta = delta;
    d.few = delta + p.q_rows * p.Hq;
    d.lse_seq = p.lse_seq; d.lse_head = p.lse_head;
    d.scale_log2 = a.scale_log2;
    d.inv_group = (float)p.Hk / (float)p.Hq;
    d.Hq = p.Hq; d.T = p.Tq; d.causal = p.causal; d.window = p.window;
    // The next kernel's blocks set themselves up beside this one's where each has an SM to
    // itself: 128 blocks 25.2 -> 23.6 us a call.  With more, the first ones would crowd onto
    // the SMs that are free early (256 blocks 29.7 -> 32.6, 16 heads over 4 of 4 x 512 tokens
    // 32.3 -> 36.0).
    long long next_blocks = 0;
    for (int x = 0; x < p.n && next_blocks <= kSMs; ++x)
        next_blocks += p.Hk * ((p.seq(x).lk + kTile - 1LL) / kTile) + p.Hq * ((p.seq(x).lq + kTile - 1LL) / kTile);
    d.release = next_blocks <= kSMs;
    constexpr int kRowsPerBlock = 8 * (32 / (D / 8));
    for (int i = 0; i < p.n && p.q_rows > 0; i += kMaxSeqs) {
        // every row with the first launch, and each launch's sequences' rows of few keys
        d.rows = i == 0 ? p.q_rows * p.Hq : 0;
        d.n = 0;
        long long few_rows = 0;
        for (int x = i; x < std::min(i + kMaxSeqs, p.n); ++x) {
            const Seq s = p.seq(x);
            const int off = s.lk - s.lq;
            int first = 0, end = 0;
            if ((p.window && p.window <= kFewKeys) || s.lk <= kFewKeys) {
                end = s.lq;
            } else if (p.causal) {  // positions 1 .. kFewKeys - 1
                first = std::max(0, 1 - off);
                end = std::min(s.lq, kFewKeys - off);
            }
            if (end <= first || s.lk < 2) continue;
            d.seq[d.n++] = {s.q0, s.lq, s.k0, s.lk, first, (int)few_rows};
            few_rows += end - first;
        }
        d.few_rows = (int)few_rows;
        d.few_blocks = (int)((few_rows * p.Hq + kRowsPerBlock - 1) / kRowsPerBlock);
        const unsigned blocks = (unsigned)(d.few_blocks + (d.rows + kRowsPerBlock * kDeltaRows - 1) / (kRowsPerBlock * kDeltaRows));
        if (blocks == 0) continue;
        MUIR_TIMED("k_attn_delta", st, k_attn_delta<D><<<blocks, 256, 0, st>>>(d));
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    }
    for (int i = 0; i < p.n; i += kMaxSeqs) {
        const int last = std::min(i + kMaxSeqs, p.n);
        long long kv_blocks, q_blocks;
        a.n_kv = gather_seqs(p, i, last, true, kTile, a.kv, &kv_blocks);
        a.n_q = gather_seqs(p, i, last, false, kTile, a.q, &q_blocks);
        a.kv_blocks = (int)kv_blocks;
        a.q_blocks = (int)q_blocks;
        // Two heads a block where the group is even, there is room, and the blocks still go
        // round: packed windows of 5245 tokens, 16 heads over 4, 75.7 -> 71.1 us; 8 x 1024
        // tokens 117.8 -> 113.0.
        a.dq_heads = DqSmem<D>::kHeads == 2 && a.group % 2 == 0 && q_blocks * (p.Hq / 2) >= 2 * kSMs ? 2 : 1;
        const long long blocks = kv_blocks + q_blocks * (a.group / a.dq_heads);
        if (blocks == 0) continue;
        MUIR_TIMED("k_attn_bwd", st,
                   err = launch_early(k_attn_bwd<D>, p.q_rows > 0, block_grid(p.Hk, blocks), kThreads, kSmem, st, a));
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace

size_t bwd_ws_bytes(const Problem& p) { return (size_t)p.q_rows * p.Hq * 8; }

cudaError_t run_bwd(const Problem& p, const void* o, const float* lse, const void* dO, void* dq, void* dk,
                    void* dv, void* ws, cudaStream_t st) {
    BwdParams a;
    cudaError_t err = cudaSuccess;
    if (p.q_rows == 0 && p.k_rows == 0) return err;
    if (p.q_rows > 0) {
        err = make_tmap_tokens(&a.tq, p.q, p.d, p.Hq, p.q_ld, p.q_rows, kTile);
        if (err == cudaSuccess)
            err = make_tmap_tokens(&a.tdo, dO, p.d, p.Hq, (long long)p.Hq * p.d, p.q_rows, kTile);
    }
    if (err == cudaSuccess && p.k_rows > 0) {
        err = make_tmap_tokens(&a.tk, p.k, p.d, p.Hk, p.k_ld, p.k_rows, kTile);
        if (err == cudaSuccess) err = make_tmap_tokens(&a.tv, p.v, p.d, p.Hk, p.v_ld, p.k_rows, kTile);
    }
    if (err != cudaSuccess) return err;
    a.lse = lse;
    a.delta = static_cast<float*>(ws);
    a.few = a.delta + p.q_rows * p.Hq;
    a.dq = static_cast<__nv_bfloat16*>(dq);
    a.dk = static_cast<__nv_bfloat16*>(dk);
    a.dv = static_cast<__nv_bfloat16*>(dv);
    a.lse_seq = p.lse_seq;
    a.lse_head = p.lse_head;
    a.scale = p.scale;
    a.scale_log2 = p.scale * kLog2e;
    a.Hq = p.Hq; a.Hk = p.Hk; a.group = p.Hq / p.Hk; a.causal = p.causal; a.window = p.window;
    return p.d == 128 ? run<128>(p, a, o, dO, static_cast<float*>(ws), st)
                      : run<64>(p, a, o, dO, static_cast<float*>(ws), st);
}

unsigned int timeouts_bwd() {
    unsigned int n = 0;
    cudaMemcpyFromSymbol(&n, g_bwd_timeouts, sizeof(n));
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_bwd_timeouts, &z, sizeof(z));
    return n;
}

}  // namespace attn
}  // namespace muir
