// kv4_evict.cu -- eviction from the 4-bit key/value cache by accumulated attention weight.
//
// Of the len tokens of a (sequence, KV head) the first `first`, the last `recent` and the heaviest
// others are kept, `keep` in all (equal weights: the lower position), in their order, and their rows
// (codes, scales, index keys, weights) are copied to the front of another cache.
//
//   select : one CTA per (sequence, KV head) finds the weight of the last token that is kept, bit by
//            bit on order-preserving integers, and writes the kept positions in order;
//   move   : one warp per kept row copies it.
#include "kv4.cuh"

namespace msa {

namespace {

constexpr int kSelThreads = 1024;

// Integers that order like the weights (-0 and +0 are one value).
__device__ __forceinline__ uint32_t weight_key(float w)
{
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int block_sum(int x, int* tmp)
{
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, tmp[threadIdx.x & 31]);
}

__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(Kv4EvictArgs a)
{
    __shared__ int tmp[32], tmp2[32];
    const int b = blockIdx.y, r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = a.lens[b];
    const bool bad = len < 0 || len > a.L_max;
    const int n = bad ? 0 : len, left = min(n, a.keep);
    int32_t* kept = a.kept + ((int64_t)b * a.H_kv + r) * a.keep;
    if (tid == 0 && r == 0) {
        if (bad) report_error(a.err, MSA_ERR_DEVICE_CHECK, 200 + b);
        a.lens_to[b] = left;
    }
    for (int j = tid; j < a.keep; j += kSelThreads)
        if (n <= a.keep) kept[j] = j < n ? j : -1;
    if (n <= a.keep) return;
    const float* w = a.w + ((int64_t)b * a.H_kv + r) * a.L_max;
    const int c0 = a.first, c1 = n - a.recent, need = a.keep - a.first - a.recent; // candidates [c0, c1)
    uint32_t T = 0; // the need-th largest key
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = T | (1u << bit);
        int cnt = 0;
        for (int j = c0 + tid; j < c1; j += kSelThreads) cnt += weight_key(w[j]) >= cand;
        if (block_sum(cnt, tmp) >= need) T = cand;
    }
    int above = 0;
    for (int j = c0 + tid; j < c1; j += kSelThreads) above += weight_key(w[j]) > T;
    int ties = need - block_sum(above, tmp); // equal weights still to take, in order
    if (need == 0) ties = 0;
    int base = 0;
    for (int j0 = 0; j0 < n; j0 += kSelThreads) {
        const int j = j0 + tid;
        const bool in = j < n, mid = in && j >= c0 && j < c1;
        const uint32_t key = mid ? weight_key(w[j]) : 0u;
        const bool tie = mid && key == T && need > 0;
        const unsigned tb = __ballot_sync(0xffffffffu, tie);
        __syncthreads();
        if (lane == 0) tmp[warp] = __popc(tb);
        __syncthreads();
        int before = 0, all = 0;
        for (int i = 0; i < 32; ++i) {
            before += i < warp ? tmp[i] : 0;
            all += tmp[i];
        }
        const bool take = in && (!mid || (need > 0 && (key > T || (tie && before + __popc(tb & ((1u << lane) - 1u)) < ties))));
        ties -= min(ties, all);
        const unsigned kb = __ballot_sync(0xffffffffu, take);
        if (lane == 0) tmp2[warp] = __popc(kb);
        __syncthreads();
        before = 0;
        all = 0;
        for (int i = 0; i < 32; ++i) {
            before += i < warp ? tmp2[i] : 0;
            all += tmp2[i];
        }
        const int at = base + before + __popc(kb & ((1u << lane) - 1u));
        if (take && at < a.keep) kept[at] = j;
        base += all;
    }
}

__global__ void __launch_bounds__(256) kv4_move_kernel(Kv4EvictArgs a)
{
    const int b = blockIdx.z, r = blockIdx.y, lane = threadIdx.x & 31;
    const int left = a.lens_to[b];
    const int32_t* kept = a.kept + ((int64_t)b * a.H_kv + r) * a.keep;
    const int64_t from0 = ((int64_t)b * a.H_kv + r) * a.L_max, to0 = ((int64_t)b * a.H_kv + r) * a.L_to;
    const int cu = a.d_h / 32, iu = a.k_idx ? a.d_idx / 8 : 0, sb = a.d_h / 16; // 16-byte units; bytes of scales
    for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < left; i += gridDim.x * 8) {
        const int j = kept[i];
        const int64_t from = from0 + j, to = to0 + i;
        int u = lane;
        if (u < cu) {
            reinterpret_cast<uint4*>(a.k_codes_to)[to * cu + u] = reinterpret_cast<const uint4*>(a.k_codes)[from * cu + u];
        } else if ((u -= cu) < cu) {
            reinterpret_cast<uint4*>(a.v_codes_to)[to * cu + u] = reinterpret_cast<const uint4*>(a.v_codes)[from * cu + u];
        } else if ((u -= cu) < sb / 4) {
            reinterpret_cast<uint32_t*>(a.k_scales_to)[to * (sb / 4) + u] = reinterpret_cast<const uint32_t*>(a.k_scales)[from * (sb / 4) + u];
        } else if ((u -= sb / 4) < sb / 4) {
            reinterpret_cast<uint32_t*>(a.v_scales_to)[to * (sb / 4) + u] = reinterpret_cast<const uint32_t*>(a.v_scales)[from * (sb / 4) + u];
        } else if ((u -= sb / 4) == 0 && a.w_to) {
            a.w_to[to] = a.w[from];
        }
        if (lane >= 32 - iu) { // the last lanes: at most 16 units, which the others leave free
            u = lane - (32 - iu);
            reinterpret_cast<uint4*>(a.k_idx_to)[(((int64_t)b * a.L_to + i) * a.H_kv + r) * iu + u] =
                reinterpret_cast<const uint4*>(a.k_idx)[(((int64_t)b * a.L_max + j) * a.H_kv + r) * iu + u];
        }
    }
}

} // namespace

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t s)
{
    trace_begin(s);
    kv4_select_kernel<<<dim3(a.H_kv, a.B), kSelThreads, 0, s>>>(a);
    const int gx = (a.keep + 31) / 32; // 4 rows per warp
    kv4_move_kernel<<<dim3(gx, a.H_kv, a.B), 256, 0, s>>>(a);
    trace_end(s, MSA_KERNEL_KV4_EVICT);
    note_launch(2);
    return cudaGetLastError();
}

} // namespace msa
