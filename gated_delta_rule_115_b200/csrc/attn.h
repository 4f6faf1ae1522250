// attn.h -- internal interface of the softmax-attention kernels; not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>

namespace muir {
namespace attn {

constexpr int kTile = 128;    // query or key rows of a product tile
constexpr int kMaxSeqs = 128; // sequences of one launch (they travel as kernel arguments)

// One sequence: rows [q0, q0 + lq) of the query tensors, [k0, k0 + lk) of the key tensors;
// its blocks for each head, and its entry in the order of the launch's blocks (place_of).
struct Seq {
    int q0, lq, k0, lk, blocks, block0;
};

// What every kernel needs to know of the call.
struct Problem {
    int Hq, Hk, d;
    int causal, window;   // window 0: none
    float scale;
    long long q_ld, k_ld, v_ld;          // elements between tokens
    long long q_rows, k_rows;            // tokens of the query / key tensors
    long long lse_seq, lse_head;         // lse index = q0 * lse_seq + h * lse_head + row
    const void *q, *k, *v;
    // n sequences: packed ones at cu_q / cu_k (host, n + 1 offsets), or, with both null,
    // n times Tq queries and Tk keys
    int n, Tq, Tk;
    const long long *cu_q, *cu_k;
    Seq seq(int i) const {
        if (!cu_q) return Seq{i * Tq, Tq, i * Tk, Tk, 0, 0};
        return Seq{(int)cu_q[i], (int)(cu_q[i + 1] - cu_q[i]), (int)cu_k[i], (int)(cu_k[i + 1] - cu_k[i]), 0, 0};
    }
};

// Sequences [first, last) of the call (at most kMaxSeqs) whose `rows` (queries, or keys with
// by_keys) number at least one, the longest first, with their blocks of rows_per_block rows
// and the order of these.  Returns how many; `blocks`: the total.
int gather_seqs(const Problem& p, int first, int last, bool by_keys, int rows_per_block, Seq* out,
                long long* blocks);

cudaError_t run_fwd(const Problem& p, void* o, float* lse, cudaStream_t st);

cudaError_t run_bwd(const Problem& p, const void* o, const float* lse, const void* dO, void* dq,
                    void* dk, void* dv, void* ws, cudaStream_t st);
size_t bwd_ws_bytes(const Problem& p);

unsigned int timeouts_fwd();
unsigned int timeouts_bwd();

}  // namespace attn
}  // namespace muir
