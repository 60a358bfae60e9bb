// topk.cuh -- exp-free register Top-k ("MiniMax Sparse Attention" explainer, section 05-1).
//
// Softmax preserves order, so block selection ranks the raw pooled scores directly. Each thread
// keeps the best k-1 (score, block) pairs of the blocks it has seen in a register-resident list
// sorted best-first. The list always has L = kMaxK - 1 slots; for a runtime k < kMaxK the first
// L - (k-1) slots hold sentinels (+inf, -1) that nothing can displace, so the admission test is a
// single compare against the last slot (a static register index, no local memory).
//
// Order ("a beats b"): larger score first (-inf last); equal scores, lower block index first.
#pragma once
#include <cstdint>
#include <math_constants.h>

#include "common.cuh"

namespace msa {

struct TopkList {
    static constexpr int L = kMaxK - 1;
    float v[L];
    int b[L];

    // k_keep = k - 1 real slots.
    __device__ __forceinline__ void init(int k_keep)
    {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const bool sentinel = j < L - k_keep;
            v[j] = sentinel ? CUDART_INF_F : CUDART_NAN_F; // NaN: free
            b[j] = sentinel ? -1 : 0x7FFFFFFF;
        }
    }

    // A block whose index exceeds that of every listed block (a row's blocks are offered in ascending order): an equal
    // score never beats a listed one, so the order test is "not at most", which a free slot's NaN passes for every
    // score, -inf too: min(k - 1, blocks offered) slots are filled whatever the scores. The insertion is one
    // independent select per slot (slot j takes its left neighbour if val beats that, else val if val beats slot j,
    // else keeps its entry) instead of a serial shift. Sentinels (+inf) are never displaced. val is no NaN.
    __device__ __forceinline__ void offer_ascending(float val, int blk)
    {
        if (val <= v[L - 1]) return;
        bool c[L];
#pragma unroll
        for (int j = 0; j < L; ++j) c[j] = !(val <= v[j]);
#pragma unroll
        for (int j = L - 1; j >= 1; --j) {
            v[j] = c[j - 1] ? v[j - 1] : (c[j] ? val : v[j]);
            b[j] = c[j - 1] ? b[j - 1] : (c[j] ? blk : b[j]);
        }
        v[0] = c[0] ? val : v[0];
        b[0] = c[0] ? blk : b[0];
    }
};

// Final selection of one (row, group): the admitted blocks plus the local block, ascending,
// padded with -1, written to out[0..k).
__device__ __forceinline__ void emit_selection(const TopkList& t, int local, int k, int32_t* out)
{
    int sel[kMaxK];
#pragma unroll
    for (int j = 0; j < TopkList::L; ++j) sel[j] = (t.b[j] >= 0 && t.b[j] != 0x7FFFFFFF) ? t.b[j] : 0x7FFFFFFF;
    sel[kMaxK - 1] = local;
    // odd-even transposition sort, ascending (invalid = INT_MAX sinks to the end)
#pragma unroll
    for (int pass = 0; pass < kMaxK; ++pass) {
#pragma unroll
        for (int j = pass & 1; j + 1 < kMaxK; j += 2) {
            const int lo = min(sel[j], sel[j + 1]), hi = max(sel[j], sel[j + 1]);
            sel[j] = lo;
            sel[j + 1] = hi;
        }
    }
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
        if (j < k) out[j] = sel[j] == 0x7FFFFFFF ? -1 : sel[j];
}

} // namespace msa
