// kv4_evict.cu -- eviction from the 4-bit key/value cache by accumulated attention weight.
//
// Of the len tokens of a (sequence, KV head) the first `first`, the last `recent` and the heaviest
// others are kept, `keep` in all (equal weights: the lower position), in their order, and their rows
// (codes, scales, index keys, weights) are copied to the front of another cache.
//
//   select : a cluster of CTAs per (sequence, KV head), each with a contiguous part of the tokens,
//            finds the weight of the last token kept by a radix select (three digits of order-preserving
//            integers, most significant first, histograms in shared memory summed over the cluster),
//            then writes the kept positions in order: every warp counts in a contiguous run, the counts
//            are scanned over warps and CTAs, and a second walk writes. No atomics decide an order.
//            Bound by the latency of its rounds: 16 sequences in [20K, 32K] take 21 us, where reading the
//            weights takes 1.
//   move   : CTAs of 64 kept rows; a thread starts all its loads before its stores. Bound by memory: 4096 rows of
//            each, with index keys of 64, take 30 us (5.2 TB/s in the capture, which reads 126 MB for 72 MB
//            of rows: a row's scales are 8 bytes of a 32-byte sector, a weight 4).
#include <cooperative_groups.h>

#include "kv4.cuh"

namespace cg = cooperative_groups;

namespace msa {

namespace {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kDigits = 3;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;           // the portable limit

__device__ __forceinline__ int digit_shift(int d) { return d == 0 ? 21 : (d == 1 ? 10 : 0); }
__device__ __forceinline__ int digit_bits(int d) { return d == 2 ? 10 : 11; }

// Integers that order like the weights (-0 and +0 are one value, and every NaN is one above +inf), without a branch:
// the loads of a thread's weights start together.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) | (w == w ? 0u : 0xFFFFFFFFu);
}

struct SelShared {
    // a histogram for every digit, and its sums of 32 bins, read by the cluster (2, 4 or 8 copies against lanes
    // that meet in a bin gain nothing: 16 prompts of 20K to 32K tokens take 92, 92 and 104 us, 92 without)
    int hist[kDigits][kBins], coarse[kDigits][kBins / 32];
    uint32_t prefix; // of the key looked for, and how many of its equals are still to be taken
    int need, whole;
    int ties[kSelWarps], takes[kSelWarps];
    int cta_ties, cta_sure; // this CTA's equal keys, and tokens kept without a choice
};

// f(r) for every CTA r of the cluster, its loads in flight together.
template <class F>
__device__ __forceinline__ void for_ranks(int size, F f)
{
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
        if (r < size) f(r);
}

// The sum of x over this lane and the lower ones.
__device__ __forceinline__ int warp_sum_upto(int x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Every warp owns a contiguous run of tokens, walked in rounds of 32 * KEYS. RESIDENT: the run is one round,
// whose keys are read from memory once and stay in registers.
template <int KEYS, bool RESIDENT>
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(Kv4EvictArgs a)
{
    __shared__ __align__(16) SelShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), size = cluster.num_blocks();
    const int seg = blockIdx.x / size, b = seg / a.H_kv; // (sequence, KV head)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    const int len = a.lens[b];
    const bool bad = len < 0 || len > a.L_max;
    const int n = bad ? 0 : len, left = min(n, a.keep);
    int32_t* kept = a.kept + (int64_t)seg * a.keep;
    if (tid == 0 && rank == 0 && seg % a.H_kv == 0) {
        if (bad && a.err) report_error(a.err, MSA_ERR_DEVICE_CHECK, 200 + b);
        a.lens_to[b] = left;
    }
    if (n <= a.keep) { // the whole cluster
        for (int j = rank * kSelThreads + tid; j < a.keep; j += size * kSelThreads) kept[j] = j < n ? j : -1;
        return;
    }
    const float* w = a.w + (int64_t)seg * a.L_max;
    const int c0 = a.first, c1 = n - a.recent; // candidates
    constexpr int kRound = 32 * KEYS;
    const int run = RESIDENT ? kRound : (n + size * kSelWarps * kRound - 1) / (size * kSelWarps * kRound) * kRound;
    const int r0 = min(n, (rank * kSelWarps + warp) * run), r1 = min(n, r0 + run);
    uint32_t key[KEYS];
    auto load = [&](int j0) { // keys of tokens j0 + 32 i + lane, 0 for those that are no candidates
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const int j = j0 + 32 * i + lane;
            key[i] = j < r1 && j >= c0 && j < c1 ? weight_key(w[j]) : 0u;
        }
    };
    auto is_mid = [&](int j) { return j < r1 && j >= c0 && j < c1; };
    if (RESIDENT) load(r0);
    uint32_t T = 0xFFFFFFFFu; // no key is above it
    int need = a.keep - a.first - a.recent;
    const bool choose = need > 0;
    if (choose) {
        for (int i = tid; i < kDigits * kBins / 4; i += kSelThreads) reinterpret_cast<int4*>(sh.hist)[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
        T = 0;
        for (int d = 0; d < kDigits; ++d) {
            const int shift = digit_shift(d), bits = digit_bits(d);
            int *hist = sh.hist[d], *coarse = sh.coarse[d];
            const uint32_t above = d == 0 ? 0u : 0xFFFFFFFFu << (shift + bits);
            for (int j0 = r0; j0 < r1; j0 += kRound) {
                if (!RESIDENT) load(j0);
#pragma unroll
                for (int i = 0; i < KEYS; ++i)
                    if (is_mid(j0 + 32 * i + lane) && (key[i] & above) == T)
                        atomicAdd(&hist[(key[i] >> shift) & ((1u << bits) - 1u)], 1);
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kBins / kSelThreads; ++u) { // a warp sums 32 neighbouring bins
                const int i = u * kSelThreads + tid, all = __reduce_add_sync(0xffffffffu, hist[i]);
                if (lane == 0) coarse[i / 32] = all;
            }
            cluster.sync();
            // in descending order, the 32 bins in which the counts reach `need`, and then the bin
            if (warp == 0) {
                static_assert(kBins == 64 * 32, "two groups of bins to a lane");
                int2 c = make_int2(0, 0); // groups 62 - 2 lane and the one above it
                for_ranks(size, [&](int r) {
                    const int2 y = reinterpret_cast<const int2*>(cluster.map_shared_rank(coarse, r))[31 - lane];
                    c.x += y.x, c.y += y.y;
                });
                const int upto = warp_sum_upto(c.x + c.y), above2 = upto - c.x - c.y;
                const int owner = __ffs(__ballot_sync(0xffffffffu, upto >= need)) - 1; // candidates are `need` or more
                const bool second = above2 + c.y < need;
                const int group = __shfl_sync(0xffffffffu, 62 - 2 * lane + !second, owner);
                const int before = __shfl_sync(0xffffffffu, above2 + (second ? c.y : 0), owner);
                const int bin = 32 * group + 31 - lane;
                int x = 0;
                for_ranks(size, [&](int r) { x += cluster.map_shared_rank(hist, r)[bin]; });
                const int reach = before + warp_sum_upto(x);
                if (reach >= need && reach - x < need) { // one lane
                    const uint32_t prefix = T | ((uint32_t)bin << shift);
                    // a bin that is taken whole: its keys are those above prefix - 1, and no further digit is needed
                    sh.whole = reach == need && prefix != 0u;
                    sh.prefix = sh.whole ? prefix - 1u : prefix;
                    sh.need = sh.whole ? 0 : need - (reach - x);
                }
            }
            __syncthreads();
            T = sh.prefix;
            need = sh.need;
            if (sh.whole) break; // the same in the whole cluster
        }
    }
    // ---------------------------------------------------------------- kept positions in order
    // a token stays without a choice (not a candidate, or above T), or as one of the first `need` equal to T
    int n_sure = 0, n_tie = 0;
    for (int j0 = r0; j0 < r1; j0 += kRound) {
        if (!RESIDENT) load(j0);
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const int j = j0 + 32 * i + lane;
            n_sure += j < r1 && (!is_mid(j) || key[i] > T);
            n_tie += is_mid(j) && choose && key[i] == T;
        }
    }
    n_sure = __reduce_add_sync(0xffffffffu, n_sure);
    n_tie = __reduce_add_sync(0xffffffffu, n_tie);
    if (lane == 0) {
        sh.takes[warp] = n_sure;
        sh.ties[warp] = n_tie;
    }
    __syncthreads();
    // of the warps, and of the CTAs, before this one
    int at = __reduce_add_sync(0xffffffffu, lane < warp ? sh.takes[lane] : 0);
    int ties = __reduce_add_sync(0xffffffffu, lane < warp ? sh.ties[lane] : 0);
    if (size > 1) {
        if (warp == kSelWarps - 1 && lane == 0) {
            sh.cta_sure = at + n_sure;
            sh.cta_ties = ties + n_tie;
        }
        cluster.sync();
        at += __reduce_add_sync(0xffffffffu, lane < rank ? *cluster.map_shared_rank(&sh.cta_sure, lane) : 0);
        ties += __reduce_add_sync(0xffffffffu, lane < rank ? *cluster.map_shared_rank(&sh.cta_ties, lane) : 0);
    }
    at += min(ties, need);
    const unsigned below = (1u << lane) - 1u;
    for (int j0 = r0; j0 < r1; j0 += kRound) {
        if (!RESIDENT) load(j0);
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const int j = j0 + 32 * i + lane;
            const bool tie = is_mid(j) && choose && key[i] == T;
            const unsigned tb = __ballot_sync(0xffffffffu, tie);
            const bool take = j < r1 && (!is_mid(j) || key[i] > T || (tie && ties + __popc(tb & below) < need));
            const unsigned kb = __ballot_sync(0xffffffffu, take);
            if (take) kept[at + __popc(kb & below)] = j;
            at += __popc(kb);
            ties += __popc(tb);
        }
    }
    if (size > 1) cluster.sync(); // the cluster has read this CTA's counts
}

constexpr int kMoveRows = 64, kMoveThreads = 256;

template <int DH>
__global__ void __launch_bounds__(kMoveThreads) kv4_move_kernel(Kv4EvictArgs a)
{
    constexpr int CU = DH / 32, SW = DH / 64;                         // 16-byte units of codes, words of scales per row
    constexpr int CN = kMoveRows * CU / kMoveThreads > 0 ? kMoveRows * CU / kMoveThreads : 1;
    constexpr int IN = kMoveRows * 16 / kMoveThreads;                 // index keys: at most 16 units per row
    __shared__ int src[kMoveRows];
    const int b = blockIdx.z, r = blockIdx.y, tid = threadIdx.x, i0 = blockIdx.x * kMoveRows;
    pdl_wait();
    const int rows = min(kMoveRows, a.lens_to[b] - i0);
    if (rows <= 0) return;
    const int64_t seg = (int64_t)b * a.H_kv + r;
    if (tid < rows) src[tid] = a.kept[seg * a.keep + i0 + tid];
    __syncthreads();
    const int64_t from0 = seg * a.L_max, to0 = seg * a.L_to + i0;
    const uint4 *kc = reinterpret_cast<const uint4*>(a.k_codes) + from0 * CU, *vc = reinterpret_cast<const uint4*>(a.v_codes) + from0 * CU;
    const uint4* ki = reinterpret_cast<const uint4*>(a.k_idx);
    const int iu = a.k_idx ? a.d_idx / 8 : 0;
    uint4 xk[CN], xv[CN], xi[IN];
    uint32_t xs = 0;
#pragma unroll
    for (int n = 0; n < CN; ++n) {
        const int u = n * kMoveThreads + tid, i = u / CU;
        if (i < rows) {
            const int64_t p = (int64_t)src[i] * CU + u % CU;
            xk[n] = kc[p];
            xv[n] = vc[p];
        }
    }
#pragma unroll
    for (int n = 0; n < IN; ++n) {
        const int u = n * kMoveThreads + tid;
        if (u < rows * iu) {
            const int i = u / iu;
            xi[n] = ki[(((int64_t)b * a.L_max + src[i]) * a.H_kv + r) * iu + u % iu];
        }
    }
    // scales of K, of V (a word each at d_h = 64, two at 128) and the weight: a quarter of the threads each
    const int part = tid / kMoveRows, i = tid % kMoveRows;
    uint32_t xs2 = 0;
    if (i < rows) {
        const int64_t p = from0 + src[i];
        if (part < 2) {
            const uint32_t* s = reinterpret_cast<const uint32_t*>(part == 0 ? a.k_scales : a.v_scales) + p * SW;
            xs = s[0];
            if (SW == 2) xs2 = s[SW - 1];
        } else if (part == 2 && a.w_to) {
            xs = __float_as_uint(a.w[p]);
        }
    }
#pragma unroll
    for (int n = 0; n < CN; ++n) {
        const int u = n * kMoveThreads + tid;
        if (u / CU < rows) {
            reinterpret_cast<uint4*>(a.k_codes_to)[to0 * CU + u] = xk[n];
            reinterpret_cast<uint4*>(a.v_codes_to)[to0 * CU + u] = xv[n];
        }
    }
#pragma unroll
    for (int n = 0; n < IN; ++n) {
        const int u = n * kMoveThreads + tid;
        if (u < rows * iu)
            reinterpret_cast<uint4*>(a.k_idx_to)[(((int64_t)b * a.L_to + i0 + u / iu) * a.H_kv + r) * iu + u % iu] = xi[n];
    }
    if (i < rows) {
        if (part < 2) {
            uint32_t* s = reinterpret_cast<uint32_t*>(part == 0 ? a.k_scales_to : a.v_scales_to) + (to0 + i) * SW;
            s[0] = xs;
            if (SW == 2) s[SW - 1] = xs2;
        } else if (part == 2 && a.w_to) {
            a.w_to[to0 + i] = __uint_as_float(xs);
        }
    }
}

} // namespace

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t s)
{
    // keys in registers where a cluster of up to 8 CTAs holds a full cache (16 keys to a thread, 32 above 65536
    // tokens): 16 prompts in caches of 32768, cut to 4096 and read back, take 91 us so, 94 with 32 keys to a
    // thread of half the CTAs, 156 with keys read again for every digit, as longer caches need
    constexpr int kCta = kSelThreads * 16;
    int size = 1;
    while (size < kMaxCluster && (int64_t)size * kCta < a.L_max) size *= 2;
    const int which = a.L_max <= (int64_t)size * kCta ? 0 : (a.L_max <= (int64_t)size * kCta * 2 ? 1 : 2);
    const auto kernel = which == 0 ? kv4_select_kernel<16, true> : (which == 1 ? kv4_select_kernel<32, true> : kv4_select_kernel<32, false>);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.B * a.H_kv * size));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)size, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    trace_begin(s);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return e;
    const dim3 grid((a.keep + kMoveRows - 1) / kMoveRows, a.H_kv, a.B);
    e = launch_pdl(a.d_h == 128 ? kv4_move_kernel<128> : kv4_move_kernel<64>, grid, kMoveThreads, 0, s, a);
    trace_end(s, MSA_KERNEL_KV4_EVICT);
    note_launch(2);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

} // namespace msa
