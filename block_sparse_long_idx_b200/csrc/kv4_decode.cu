// kv4_decode.cu -- single-token attention over the 4-bit key/value cache (format: kv4.cuh).
//
// For head h of KV head r, over the visible keys j (all j < len, or those of the given blocks):
//   x_j = q[h] . K[j] / sqrt(d_h),  out[h] = sum_j softmax(x)_j V[j],  lse[h] = log sum_j exp(x_j)
//   w_out[r][j] = decay * w_in[r][j] + sum over the heads of r of softmax(x)_j      (optional)
//
// It has to read the cache (d_h + d_h / 8 bytes per token and KV head); with 16 heads of 128 the conversions and
// MMAs of a key, whose issue adds up (6.5 clocks per SM and 8 codes a lane), take longer: 32 sequences in
// [16K, 128K] with 64 heads on 4 take 300 us, 4.5 TB/s of the 6.5 that a copy moves; with up to 8 heads a
// KV head 16 sequences in [8K, 16K] with 8 KV heads take 51 us, of which 35 are the copy's. One CTA per SM walks an
// equal contiguous slice of the flattened list of 128-key blocks of all (sequence, KV head) pairs, so
// ragged batches and single long sequences load every SM alike. Bulk copies bring kBlocks blocks at a
// time into a ring of kStages such chunks; every warp takes 32 keys of a chunk and keeps a running
// maximum, sum and output of its own, joined when the CTA leaves a (sequence, KV head). What several
// CTAs hold of one pair is joined by a second kernel, in a fixed order (results do not depend on timing).
//
// The heads of a KV head are the 16 rows of mma.sync m16n8k16, or with up to 8 heads the 8 columns. (As rows they would
// fill an eighth of a tcgen05 tile; keys as its 128 rows and heads as its columns would fill it, with K converted into
// an operand in shared or tensor memory first, where here codes become fragments in registers: not built.)
// No pipe is saturated: issue 52 %, tensor 40 %, DRAM 48 % in the capture of 8 sequences in [16K, 128K]; the kernels
// of 9 to 16 heads of 128 spill (116 bytes of stores for all keys, 188 for given blocks, 36 in their weights), the
// others do not.
// E2M1 codes become fp16 pairs with the hardware conversion, times the E4M3 scale
// (both exact); no step goes through shared memory, because both products may sum in any order:
//   S = Q K^T: lane (g, t) holds d_h / 4 consecutive codes of key row g, so element t * d_h / 4 + 4 ks
//     + {0, 1, 2, 3} of a row is the contraction index {2t, 2t + 1, 2t + 8, 2t + 9} of step ks, for Q alike;
//   O = P V: lane (g, t) holds d_h / 8 consecutive codes of four keys, so column g of output tile n is
//     element g * d_h / 8 + n, and the nibbles of two keys are joined before the conversion.
// q is held in fp16 as q * 2^-e with e the exponent of the row's largest |q| (elements lose bits only
// below 2^-14 of it, an error of 2^-25 of it at most); P in fp16 relative to a reference that leaves its
// largest value in [2^7, 2^15] (off by 2^-11 of itself at most; weights below 2^-21 of the largest may be
// subnormal and are off by 2^-32 of the largest at most). Sums, maxima and outputs are fp32.
#include <cfloat>
#include <math_constants.h>

#include "kv4.cuh"
#include "mma_sync.cuh"

namespace msa {

namespace {

constexpr int kBlocks = 3;          // blocks of a chunk
constexpr int kStages = 3;          // chunks of the ring
constexpr int kWarps = 4 * kBlocks; // consumer warps: each takes 32 keys of a chunk
constexpr int kThreads = kWarps * 32;
constexpr int kLaunch = kThreads + 128; // and one warpgroup whose first thread starts the copies
constexpr int kRegs = 160, kProducerRegs = 32; // of the 128 a thread is launched with
static_assert(kThreads * kRegs + 128 * kProducerRegs <= kLaunch * 128, "register split");
// What joining a segment costs, in blocks: it counts in the split of the work. Graph replays: 24 ragged
// sequences of 8 heads of 64 take 26.5, 25.5 and 25.4 us with 4, 5 and 6; the block-sparse decode of one
// sequence (16 blocks given) 30.1, 30.2 and 30.8 us with 2, 3 and 4, of 64 sequences 393 to 395 with any.
template <bool GIVEN>
constexpr int kJoin = GIVEN ? 3 : 6;
constexpr int kSlots = kWarps / 2; // join scratch: one output per pair of warps
constexpr int kTile = 32;          // keys of a warp's part
constexpr float kHeadroom = 7.f;   // P's reference: log2 units below the maximum it was set from
constexpr float kRaise = 15.f;     // P stays below 2^15, within fp16

template <int DH>
struct Cfg {
    static constexpr int CODE = DH / 2, NG = DH / 16; // bytes of a row's codes, scales
    static constexpr int KEYS = kBlocks * kBk;        // of a stage
    static constexpr int K_CODES = 0, V_CODES = KEYS * CODE, K_SCALES = 2 * KEYS * CODE, V_SCALES = K_SCALES + KEYS * NG,
                         STAGE = V_SCALES + KEYS * NG;
    // join scratch: [slot][16 rows][4 lanes][DH / 4], padded so that 16-byte accesses do not conflict
    static constexpr int LANE = DH / 4 + 4, ROW = 4 * LANE, WARP = 16 * ROW;
    static constexpr int SMEM = kStages * STAGE + kSlots * WARP * 4;
};

// The flattened list: a segment is a (sequence, KV head); sequence b owns H_kv segments of kJoin units (no
// work, they stand for the join) and blocks(b) blocks. With given blocks every segment has k, padding
// among them.
template <bool GIVEN>
struct Work {
    const Kv4DecodeArgs& a;
    __device__ __forceinline__ bool valid(int len) const { return len >= a.min_len && len <= a.L_max; }
    __device__ __forceinline__ int blocks(int len) const // per KV head
    {
        if (!valid(len) || len == 0) return 0;
        return GIVEN ? a.k : (len + kBk - 1) / kBk;
    }
    __device__ __forceinline__ int units(int len) const // per segment
    {
        const int n = blocks(len);
        return n > 0 ? n + kJoin<GIVEN> : 0;
    }
    // First key of entry `lane % 16` of (b, r), by whole warps (the halves may differ in r): -1 for padding and for
    // entries left out, those outside the sequence and those that do not exceed every block of it before them in the
    // list (an entry left out for that is below one kept, so all entries inside count). bad: left out, not padding.
    __device__ __forceinline__ int given_key0(int b, int r, int len, bool& bad) const
    {
        static_assert(kMaxK <= 16, "a list in 16 lanes");
        const int i = threadIdx.x & 15;
        const int blk = i < a.k ? a.block_idx[((int64_t)b * a.H_kv + r) * a.k + i] : -1;
        const bool inside = blk >= 0 && blk <= (len - 1) / kBk;
        int top = inside ? blk : -1; // the highest block up to this entry
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_up_sync(0xffffffffu, top, o, 16)); // (itself where there is none)
        const int before = __shfl_up_sync(0xffffffffu, top, 1, 16);
        const bool kept = inside && (i == 0 || blk > before);
        bad = !kept && blk != -1;
        return kept ? blk * kBk : -1;
    }
};

// Block-wide: the number of units of all sequences (below 2^31, checked on the host for full caches).
// Sequences [b_lo, b_hi) are the calling thread's, `before` the units of those before them.
template <int THREADS, bool GIVEN>
__device__ __forceinline__ int total_units(const Work<GIVEN>& w, int* warp_units, int& before, int& b_lo, int& b_hi)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (w.a.B + THREADS - 1) / THREADS;
    b_lo = min(w.a.B, tid * per);
    b_hi = min(w.a.B, b_lo + per);
    int n = 0;
    for (int b = b_lo; b < b_hi; ++b) n += w.units(w.a.lens[b]) * w.a.H_kv;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_units[warp] = x;
    __syncthreads();
    int total = 0;
    before = x - n;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        const int y = warp_units[i];
        if (i < warp) before += y;
        total += y;
    }
    return total;
}

// A walk over the slice [lo, hi) of the list, segment by segment.
template <bool GIVEN>
struct Walk {
    int b, r, len, n; // sequence, KV head, length, blocks of a segment of this sequence
    int seg;          // first block of the segment, behind its kJoin units
    int lo, hi;       // the slice
    int pos, end;     // the part of the segment in the slice, from the next block on (pos >= end: none)

    __device__ __forceinline__ void enter()
    {
        pos = max(seg, lo);
        end = min(seg + n, hi);
    }
    __device__ __forceinline__ void begin(const Work<GIVEN>& w, int b0, int seq0, int lo_, int hi_)
    {
        lo = lo_;
        hi = hi_;
        b = b0;
        len = w.a.lens[b];
        n = w.blocks(len);
        r = (lo - seq0) / (n + kJoin<GIVEN>);
        seg = seq0 + r * (n + kJoin<GIVEN>) + kJoin<GIVEN>;
        enter();
    }
    __device__ __forceinline__ bool more() const { return seg < hi; }
    __device__ __forceinline__ void next_segment(const Work<GIVEN>& w)
    {
        seg += n + kJoin<GIVEN>;
        if (++r == w.a.H_kv) {
            r = 0;
            if (seg < hi) { // the list goes on
                int m;
                do {
                    len = w.a.lens[++b];
                    m = w.blocks(len);
                } while (m == 0);
                n = m;
            }
        }
        enter();
    }
};

struct Shared {
    uint64_t full[kStages], empty[kStages];
    float m[kSlots][16], l[kSlots][16];
    uint4 q[8][32]; // Q fragments of the segment
    float2 f[32];   // the lanes' factors on its sums (load_q)
    int key0[16];   // given blocks: the first keys of its list's entries (given_key0)
    int warp_units[kLaunch / 32];
    int b0, seg0; // sequence holding the slice's first unit, first unit of that sequence
    int abort_flag;
};

// Fragments of q's rows g and g + 8 (rows past the G heads are zero) in fp16, and the factors that turn sums of
// the products into logits in log2 units, of the two heads that the lane's scores belong to (rows_of below).
// NARROW: of row g only; qf[i][0], [2] are then the B fragment of step i.
template <int DH, bool NARROW>
__device__ __forceinline__ void load_q(const Kv4DecodeArgs& a, int b, int r, int G, int g, int t, uint32_t (&qf)[DH / 16][4],
                                       float& f0, float& f1)
{
#pragma unroll
    for (int half = 0; half < (NARROW ? 1 : 2); ++half) {
        const int row = g + 8 * half;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + ((int64_t)b * a.H_q + r * G + row) * DH + t * (DH / 4));
        uint32_t x[DH / 8];
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
            const uint4 v = row < G ? src[i] : make_uint4(0u, 0u, 0u, 0u);
            x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(x[i])), fabsf(bf16_hi(x[i]))));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 2^e <= mx; e within [-126, 126] so that 2^-e is a normal number too
        const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -126), 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        // finite and above 0, so that it maps a sum of 0 to 0 and a masked -inf to -inf; a small scale is multiplied by a
        // large 2^e first (exactly), so that no product on the way is subnormal where the factor is not
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        const bool first = a.k_scale < 1.f && e > 0;
        const float f = (first ? a.k_scale * up : a.k_scale) * rsqrtf((float)DH) * 1.4426950408889634f;
        (half ? f1 : f0) = fminf(fmaxf(first ? f : f * up, FLT_MIN), FLT_MAX);
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) // pair i: elements 2 i, 2 i + 1 of the lane's run
            qf[i / 2][2 * (i & 1) + half] = pack_f16x2(bf16_lo(x[i]) * down, bf16_hi(x[i]) * down);
    }
    if (NARROW) {
        const float f = f0;
        f0 = __shfl_sync(0xffffffffu, f, 8 * t);
        f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }
}

// Q fragments of a segment in shared memory: 16 bytes a lane, one step's A fragment, or two steps' B fragments.
template <int DH, bool NARROW>
__device__ __forceinline__ void store_q(uint4 (*q)[32], const uint32_t (&qf)[DH / 16][4], int lane)
{
    if constexpr (NARROW) {
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) q[i][lane] = make_uint4(qf[2 * i][0], qf[2 * i][2], qf[2 * i + 1][0], qf[2 * i + 1][2]);
    } else {
#pragma unroll
        for (int i = 0; i < DH / 16; ++i) q[i][lane] = make_uint4(qf[i][0], qf[i][1], qf[i][2], qf[i][3]);
    }
}

// A lane's part of 32 rows of K whose codes and scales start at kc and ks: of row 8 n + g / 2 + 4 (g % 2)
// (column 2u of step n is key u, column 2u + 1 key u + 4) the codes of its run, and their scales.
template <int DH>
struct KTile {
    uint32_t c[4][DH / 32];
    uint16_t s[4];

    __device__ __forceinline__ void load(const uint8_t* kc, const uint8_t* ks, int g, int t)
    {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int key = 8 * n + (g >> 1) + 4 * (g & 1);
            if constexpr (DH == 128) {
                const uint4 v = *reinterpret_cast<const uint4*>(kc + key * 64 + t * 16);
                c[n][0] = v.x, c[n][1] = v.y, c[n][2] = v.z, c[n][3] = v.w;
                s[n] = *reinterpret_cast<const uint16_t*>(ks + key * 8 + t * 2);
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(kc + key * 32 + t * 8);
                c[n][0] = v.x, c[n][1] = v.y;
                s[n] = ks[key * 4 + t];
            }
        }
    }
};

__device__ __forceinline__ uint4 lds128(const uint4* p)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem_u32(p)));
    return v;
}

// The fp32 sums of q's rows with the 32 keys of the tile, q as store_q left it.
//   x[n][e]         : row g (e < 2) or g + 8, key 8 n + t + 4 (e & 1)
//   NARROW, x[m][e] : row 2 t + (e & 1), key 16 m + 8 (e >> 1) + g / 2 + 4 (g % 2)
template <int DH, bool NARROW>
__device__ __forceinline__ void scores(const KTile<DH>& k, const uint4 (*q)[32], int lane, float (&x)[NARROW ? 2 : 4][4])
{
    uint32_t s[4][DH / 64];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const uint32_t sc = e4m3x2_to_f16x2(k.s[n]);
        s[n][0] = prmt(sc, sc, 0x1010);
        if constexpr (DH == 128) s[n][1] = prmt(sc, sc, 0x3232);
    }
#pragma unroll
    for (int n = 0; n < (NARROW ? 2 : 4); ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
#pragma unroll
    for (int i = 0; i < DH / 32; ++i) {
        uint32_t h[4][4];
        if constexpr (NARROW) {
            const uint4 v = lds128(&q[i][lane]);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                e2m1x8_to_f16x2(k.c[n][i], h[n]);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[n][e] = mul_f16x2(h[n][e], s[n][i / 2]);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t a0[4] = {h[2 * m][0], h[2 * m + 1][0], h[2 * m][1], h[2 * m + 1][1]};
                mma_f16_16816(x[m], a0, v.x, v.y);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t a1[4] = {h[2 * m][2], h[2 * m + 1][2], h[2 * m][3], h[2 * m + 1][3]};
                mma_f16_16816(x[m], a1, v.z, v.w);
            }
        } else {
            const uint4 va = lds128(&q[2 * i][lane]), vb = lds128(&q[2 * i + 1][lane]);
            const uint32_t qa[4] = {va.x, va.y, va.z, va.w}, qb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                e2m1x8_to_f16x2(k.c[n][i], h[n]);
                mma_f16_16816(x[n], qa, mul_f16x2(h[n][0], s[n][i / 2]), mul_f16x2(h[n][1], s[n][i / 2]));
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
                mma_f16_16816(x[n], qb, mul_f16x2(h[n][2], s[n][i / 2]), mul_f16x2(h[n][3], s[n][i / 2]));
        }
    }
}

// ex2(-inf) = 0 keeps empty rows and tiles out of the joins.
__device__ __forceinline__ float join_weight(float m, float M) { return m == -CUDART_INF_F ? 0.f : ex2_approx(m - M); }

// Joins a partial (maximum m, sum l, outputs v) to (M, L, acc).
__device__ __forceinline__ void merge(float& M, float& L, float4& acc, float m, float l, const float4& v)
{
    const float N = fmaxf(M, m), wa = join_weight(M, N), wb = join_weight(m, N);
    M = N;
    L = fmaf(wa, L, wb * l);
    acc.x = fmaf(wa, acc.x, wb * v.x);
    acc.y = fmaf(wa, acc.y, wb * v.y);
    acc.z = fmaf(wa, acc.z, wb * v.z);
    acc.w = fmaf(wa, acc.w, wb * v.w);
}

// Elements d .. d + 3 of one head, and its lse with element 0.
__device__ __forceinline__ void finish(const Kv4DecodeArgs& a, int64_t row, int d, const float4& o, float M, float L)
{
    // L = 0: no key was seen; a NaN among the logits makes L NaN, and out and lse with it
    const float inv = L == 0.f ? 0.f : 1.f / L, t = a.v_scale; // t / L may be no normal number where o / L * t is one
    *reinterpret_cast<uint2*>(a.out + row * a.d_h + d) =
        make_uint2(pack_bf16x2(o.x * inv * t, o.y * inv * t), pack_bf16x2(o.z * inv * t, o.w * inv * t));
    if (a.lse && d == 0) a.lse[row] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * 0.6931471805599453f;
}

// The consumers' barrier (the producer's warpgroup takes no part).
__device__ __forceinline__ void sync_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// A second one, at which half of the warps only arrive: the join scratch is free again.
__device__ __forceinline__ void scratch_release() { asm volatile("bar.arrive 2, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void scratch_acquire() { asm volatile("bar.sync 2, %0;" ::"n"(kThreads) : "memory"); }

template <int DH, bool GIVEN, bool NARROW>
__global__ void __launch_bounds__(kLaunch, 1) kv4_decode_kernel(Kv4DecodeArgs a)
{
    using C = Cfg<DH>;
    constexpr int NT = DH / 8; // elements of V's rows a lane reads
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Shared sh;
    float* join = reinterpret_cast<float*>(ring + kStages * C::STAGE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int G = a.H_q / a.H_kv;
    const Work<GIVEN> w{a};

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        fence_mbar_init();
        sh.abort_flag = 0;
    }
    int before, b_lo, b_hi;
    const int total = total_units<kLaunch>(w, sh.warp_units, before, b_lo, b_hi);
    const int n_cta = min((total + kJoin<GIVEN> + kBlocks - 1) / (kJoin<GIVEN> + kBlocks), (int)gridDim.x); // a chunk or more for each
    const int cta = blockIdx.x;
    // sequences without keys have no units: the last CTA answers for them, and reports what is rejected
    pdl_trigger();
    if (GIVEN) pdl_wait(); // for the blocks
    if (cta == (int)gridDim.x - 1) {
        if (tid == 0 && !a.after_topk) a.err[0] = a.err[1] = 0;
        __syncthreads();
        for (int b = warp; b < a.B; b += kLaunch / 32) {
            const int len = a.lens[b];
            if (!w.valid(len)) {
                if (lane == 0) report_error(a.err, MSA_ERR_DEVICE_CHECK, 200 + b);
            } else if (len == 0) {
                for (int e = lane; e < a.H_q * DH / 2; e += 32)
                    reinterpret_cast<uint32_t*>(a.out + (int64_t)b * a.H_q * DH)[e] = 0u;
                if (a.lse)
                    for (int e = lane; e < a.H_q; e += 32) a.lse[(int64_t)b * a.H_q + e] = -CUDART_INF_F;
            } else if (GIVEN) {
                for (int r0 = 0; r0 < a.H_kv; r0 += 2) { // two lists at a time
                    bool bad;
                    w.given_key0(b, min(r0 + lane / 16, a.H_kv - 1), len, bad);
                    if (bad) report_error(a.err, MSA_ERR_DEVICE_CHECK, 210);
                }
            }
        }
    }
    if (cta >= n_cta) return;
    const int lo = (int)((int64_t)total * cta / n_cta), hi = (int)((int64_t)total * (cta + 1) / n_cta);
    for (int b = b_lo; b < b_hi; ++b) {
        const int n = w.units(a.lens[b]) * a.H_kv;
        if (lo >= before && lo < before + n) {
            sh.b0 = b;
            sh.seg0 = before;
        }
        before += n;
    }
    __syncthreads();

    volatile int* abort_flag = &sh.abort_flag;
    Walk<GIVEN> cons;
    cons.begin(w, sh.b0, sh.seg0, lo, hi);

    if (warp >= kWarps) {
        // ---------------------------------------------------------------- producer
        reg_dealloc<kProducerRegs>();
        if (GIVEN ? warp != kWarps : tid != kThreads) return; // a list of blocks is looked at by a warp
        const bool first_lane = lane == 0;
        uint32_t n = 0; // chunks
        bool ok = true;
        for (; ok && cons.more(); cons.next_segment(w)) {
            const int64_t row0 = ((int64_t)cons.b * a.H_kv + cons.r) * a.L_max;
            bool bad;
            const int listed = GIVEN && cons.pos < cons.end ? w.given_key0(cons.b, cons.r, cons.len, bad) : -1;
            for (; cons.pos < cons.end; cons.pos += kBlocks, ++n) {
                const uint32_t st = n % kStages, round = n / kStages;
                ok = round == 0 || !first_lane || wait_or_abort(&sh.empty[st], (round - 1) & 1, abort_flag, a.err, 62, kWaitLimit);
                if (GIVEN) ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                // up to kBlocks blocks of the segment, the visible rows rounded up to 32 (L_max is whole blocks)
                uint8_t* s = ring + st * C::STAGE;
                const int nb = min(kBlocks, cons.end - cons.pos);
                auto copy = [&](int key, int at, int rows) {
                    bulk_load(s + C::K_CODES + at * C::CODE, a.k_codes + (row0 + key) * C::CODE, rows * C::CODE, &sh.full[st]);
                    bulk_load(s + C::K_SCALES + at * C::NG, a.k_scales + (row0 + key) * C::NG, rows * C::NG, &sh.full[st]);
                    bulk_load(s + C::V_CODES + at * C::CODE, a.v_codes + (row0 + key) * C::CODE, rows * C::CODE, &sh.full[st]);
                    bulk_load(s + C::V_SCALES + at * C::NG, a.v_scales + (row0 + key) * C::NG, rows * C::NG, &sh.full[st]);
                };
                auto rows_of = [&](int key, int most) { return min(most, (cons.len - key + kTile - 1) / kTile * kTile); };
                if (!GIVEN) {
                    const int key = (cons.pos - cons.seg) * kBk, rows = rows_of(key, nb * kBk);
                    mbar_arrive_expect_tx(&sh.full[st], rows * 2 * (C::CODE + C::NG));
                    copy(key, 0, rows);
                } else {
                    int key[kBlocks], all = 0;
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i) {
                        key[i] = __shfl_sync(0xffffffffu, listed, (cons.pos - cons.seg + i) & 15);
                        if (i >= nb) key[i] = -1;
                        if (key[i] >= 0) all += rows_of(key[i], kBk);
                    }
                    if (first_lane) {
                        mbar_arrive_expect_tx(&sh.full[st], all * 2 * (C::CODE + C::NG));
#pragma unroll
                        for (int i = 0; i < kBlocks; ++i)
                            if (key[i] >= 0) copy(key[i], i * kBk, rows_of(key[i], kBk));
                    }
                }
            }
        }
        // after an abort, copies may still be in flight: the shared memory must outlive them
        if (!ok && first_lane)
            for (uint32_t m = n > kStages ? n - kStages : 0; m < n; ++m)
                drain_wait(&sh.full[m % kStages], (m / kStages) & 1, a.err, 61, kWaitLimit);
        return;
    }
    // -------------------------------------------------------------------- consumers
    reg_alloc<kRegs>();
    auto leave = [&](uint32_t st) {
        __syncwarp(); // every lane has read the stage
        if (lane == 0) mbar_arrive(&sh.empty[st]);
    };
    // one warp loads a segment's q, for the second and later ones while the segment before is joined
    auto fetch_q = [&](const Walk<GIVEN>& x) {
        float f0, f1;
        uint32_t qf[DH / 16][4];
        load_q<DH, NARROW>(a, x.b, x.r, G, g, t, qf, f0, f1);
        store_q<DH, NARROW>(sh.q, qf, lane);
        sh.f[lane] = make_float2(f0, f1);
        if (GIVEN) { // and its list of blocks
            bool bad;
            const int key = w.given_key0(x.b, x.r, x.len, bad);
            if (lane < 16) sh.key0[lane] = key;
        }
    };
    auto to_work = [&](Walk<GIVEN>& x) { // on to a segment with blocks in the slice
        while (x.more() && x.pos >= x.end) x.next_segment(w);
    };
    to_work(cons);
    if (warp == kWarps - 1 && cons.more()) fetch_q(cons);
    sync_consumers();
    uint32_t used = 0; // chunks
    bool ok = true, first = true;
    for (; cons.more(); cons.next_segment(w), to_work(cons), first = false) {
        if (!first && warp < kSlots) scratch_release();
        const float f0 = sh.f[lane].x, f1 = sh.f[lane].y;
        // outputs: o[n][2 h + c], of head g + 8 h and element (2 t + c) NT + n; NARROW: o[i][2 u + h], of head 2 t + h
        // and element g NT + 2 i + u
        float o[NARROW ? NT / 2 : NT][4];
#pragma unroll
        for (int n = 0; n < (NARROW ? NT / 2 : NT); ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F; // references of the lane's two heads
        uint64_t l0 = 0, l1 = 0;                      // this lane's sums: of each head over even and odd columns; NARROW: l0, of both heads

        for (; ok && cons.pos < cons.end; cons.pos += kBlocks, ++used) {
            const uint32_t st = used % kStages;
            ok = wait_or_abort(&sh.full[st], (used / kStages) & 1, abort_flag, a.err, 60, kWaitLimit);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            int nk = 0; // visible keys of the warp's 32
            if (cons.pos + warp / 4 < cons.end) {
                const int i = cons.pos + warp / 4 - cons.seg, key = GIVEN ? sh.key0[i] : i * kBk;
                if (key >= 0) nk = min(kTile, cons.len - key - kTile * (warp & 3));
            }
            if (nk <= 0) {
                leave(st);
                continue;
            }
            const uint8_t* s = ring + st * C::STAGE;
            float x[NARROW ? 2 : 4][4];
            {
                KTile<DH> k;
                k.load(s + C::K_CODES + warp * kTile * C::CODE, s + C::K_SCALES + warp * kTile * C::NG, g, t);
                scores<DH, NARROW>(k, sh.q, lane, x);
            }
            const uint8_t* vc = s + C::V_CODES + warp * kTile * C::CODE;
            uint8_t* vs = ring + st * C::STAGE + C::V_SCALES + warp * kTile * C::NG;
            // ------------------------------------------------------------ softmax
            if (nk < kTile) { // the last tile of a segment
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if constexpr (NARROW) {
                        const int m = n >> 1, u = n & 1;
                        if (8 * n + (g >> 1) + 4 * (g & 1) >= nk) x[m][2 * u] = x[m][2 * u + 1] = -CUDART_INF_F;
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (8 * n + t + 4 * e >= nk) x[n][e] = x[n][2 + e] = -CUDART_INF_F;
                    }
                }
                // rows past the length hold anything, NaN scales among it: they weigh 0 and must be finite
                if (lane >= nk)
                    for (int i = 0; i < C::NG; i += 4) *reinterpret_cast<uint32_t*>(vs + lane * C::NG + i) = 0u;
                __syncwarp();
                fence_proxy_async(); // the stage is written by a bulk copy again
            }
            float mx0, mx1;
            if constexpr (NARROW) {
                mx0 = fmaxf(max3f(x[0][0], x[0][2], x[1][0]), x[1][2]);
                mx1 = fmaxf(max3f(x[0][1], x[0][3], x[1][1]), x[1][3]);
            } else {
                mx0 = max3f(x[0][0], x[0][1], x[1][0]), mx1 = max3f(x[0][2], x[0][3], x[1][2]);
                mx0 = max3f(mx0, x[1][1], x[2][0]), mx1 = max3f(mx1, x[1][3], x[2][2]);
                mx0 = max3f(mx0, x[2][1], x[3][0]), mx1 = max3f(mx1, x[2][3], x[3][2]);
                mx0 = fmaxf(mx0, x[3][1]), mx1 = fmaxf(mx1, x[3][3]);
            }
            // the references (equal in the lanes of a head) move up only when P would leave [0, 2^15): exact, and rare
            if (__any_sync(0xffffffffu, mx0 * f0 > m0 + kRaise || mx1 * f1 > m1 + kRaise)) { // f > 0
#pragma unroll
                for (int d = NARROW ? 4 : 1; d < (NARROW ? 32 : 4); d <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
                }
                mx0 *= f0;
                mx1 *= f1;
                const float n0 = mx0 > m0 + kRaise ? mx0 - kHeadroom : m0, n1 = mx1 > m1 + kRaise ? mx1 - kHeadroom : m1;
                const float r0 = join_weight(m0, n0), r1 = join_weight(m1, n1);
                m0 = n0;
                m1 = n1;
                l0 = f2_mul(l0, f2_pack(r0, NARROW ? r1 : r0));
                l1 = f2_mul(l1, f2_pack(r1, r1));
#pragma unroll
                for (int n = 0; n < (NARROW ? NT / 2 : NT); ++n) {
                    o[n][0] *= r0;
                    o[n][1] *= NARROW ? r1 : r0;
                    o[n][2] *= NARROW ? r0 : r1;
                    o[n][3] *= r1;
                }
            }
            // P in fp16: A fragments of 16 keys; NARROW: B fragments (keys by heads), from 8 x 8 transposes
            uint32_t pf[2][4];
            if constexpr (NARROW) {
                const uint64_t ff = f2_pack(f0, f1), mm = f2_pack(-m0, -m1);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint64_t y = f2_fma(f2_pack(x[n >> 1][2 * (n & 1)], x[n >> 1][2 * (n & 1) + 1]), ff, mm);
                    const float p0 = ex2_approx(f2_lo(y)), p1 = ex2_approx(f2_hi(y));
                    l0 = f2_add(l0, f2_pack(p0, p1));
                    pf[n >> 1][n & 1] = transpose_8x8(pack_f16x2(p0, p1));
                }
            } else {
                const uint64_t ff0 = f2_pack(f0, f0), ff1 = f2_pack(f1, f1), mm0 = f2_pack(-m0, -m0), mm1 = f2_pack(-m1, -m1);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint64_t y0 = f2_fma(f2_pack(x[n][0], x[n][1]), ff0, mm0), y1 = f2_fma(f2_pack(x[n][2], x[n][3]), ff1, mm1);
                    const float p0 = ex2_approx(f2_lo(y0)), p1 = ex2_approx(f2_hi(y0));
                    const float p2 = ex2_approx(f2_lo(y1)), p3 = ex2_approx(f2_hi(y1));
                    l0 = f2_add(l0, f2_pack(p0, p1));
                    l1 = f2_add(l1, f2_pack(p2, p3));
                    pf[n >> 1][(n & 1) * 2] = pack_f16x2(p0, p1);
                    pf[n >> 1][(n & 1) * 2 + 1] = pack_f16x2(p2, p3);
                }
            }
            // ------------------------------------------------------------ O += P V, 16 keys a step
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t sc[2], wv[4][DH / 64]; // keys 16 j + t + {0, 4, 8, 12}
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int key = 16 * j + t + 4 * u;
                    if constexpr (DH == 128) {
                        const uint2 c = *reinterpret_cast<const uint2*>(vc + key * 64 + g * 8);
                        wv[u][0] = c.x;
                        wv[u][1] = c.y;
                    } else {
                        wv[u][0] = *reinterpret_cast<const uint32_t*>(vc + key * 32 + g * 4);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int key = 16 * j + t + 8 * u;
                    const int gs = DH == 128 ? g : g >> 1;
                    const uint32_t sa = vs[key * C::NG + gs], sb = vs[(key + 4) * C::NG + gs];
                    sc[u] = e4m3x2_to_f16x2(sa | (sb << 8));
                }
#pragma unroll
                for (int i = 0; i < DH / 64; ++i) {
                    uint32_t b0[2][4], b1[2][4]; // [even, odd elements][4]
                    e2m1x8_to_f16x2((wv[0][i] & 0x0F0F0F0Fu) | ((wv[1][i] << 4) & 0xF0F0F0F0u), b0[0]);
                    e2m1x8_to_f16x2(((wv[0][i] >> 4) & 0x0F0F0F0Fu) | (wv[1][i] & 0xF0F0F0F0u), b0[1]);
                    e2m1x8_to_f16x2((wv[2][i] & 0x0F0F0F0Fu) | ((wv[3][i] << 4) & 0xF0F0F0F0u), b1[0]);
                    e2m1x8_to_f16x2(((wv[2][i] >> 4) & 0x0F0F0F0Fu) | (wv[3][i] & 0xF0F0F0F0u), b1[1]);
                    if constexpr (NARROW) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t va[4] = {mul_f16x2(b0[0][e], sc[0]), mul_f16x2(b0[1][e], sc[0]), mul_f16x2(b1[0][e], sc[1]),
                                                    mul_f16x2(b1[1][e], sc[1])};
                            mma_f16_16816(o[4 * i + e], va, pf[j][0], pf[j][1]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            mma_f16_16816(o[8 * i + e], pf[j], mul_f16x2(b0[e & 1][e >> 1], sc[0]),
                                          mul_f16x2(b1[e & 1][e >> 1], sc[1]));
                    }
                }
            }
            leave(st);
        }
        // ------------------------------------------------------------ join the warps
        float s0 = NARROW ? f2_lo(l0) : f2_lo(l0) + f2_hi(l0), s1 = NARROW ? f2_hi(l0) : f2_lo(l1) + f2_hi(l1);
#pragma unroll
        for (int d = NARROW ? 4 : 1; d < (NARROW ? 32 : 4); d <<= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, d);
            s1 += __shfl_xor_sync(0xffffffffu, s1, d);
        }
        // the lane's two heads, and its run of their elements in the scratch
        constexpr int RUN = NARROW ? NT : 2 * NT;
        const int h0 = NARROW ? 2 * t : g, h1 = NARROW ? 2 * t + 1 : g + 8;
        float* mine = join + (warp % kSlots) * C::WARP + (NARROW ? (g >> 1) * C::LANE + (g & 1) * NT : t * C::LANE);
        auto at = [&](int h, int e) -> float& { // element e of the run of head h0 (h = 0) or h1
            if constexpr (NARROW)
                return o[e >> 1][2 * (e & 1) + h];
            else
                return o[e % NT][2 * h + e / NT];
        };
        // two steps: the upper half of the warps hand theirs to the lower half
        auto put = [&] {
            if (NARROW ? g == 0 : t == 0) {
                sh.m[warp % kSlots][h0] = m0;
                sh.m[warp % kSlots][h1] = m1;
                sh.l[warp % kSlots][h0] = s0;
                sh.l[warp % kSlots][h1] = s1;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < RUN; e += 4)
                    *reinterpret_cast<float4*>(mine + (h ? h1 : h0) * C::ROW + e) = make_float4(at(h, e), at(h, e + 1), at(h, e + 2), at(h, e + 3));
        };
        if (warp >= kSlots) {
            if (!first) scratch_acquire();
            put();
        }
        sync_consumers();
        if (warp == kWarps - 1) {
            Walk<GIVEN> next = cons;
            next.next_segment(w);
            to_work(next);
            if (next.more()) fetch_q(next);
        }
        if (warp < kSlots) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float &m = h ? m1 : m0, &l = h ? s1 : s0;
                const int row = h ? h1 : h0;
                const float om = sh.m[warp][row], M = fmaxf(m, om);
                const float wa = join_weight(m, M), wb = join_weight(om, M);
                l = fmaf(wa, l, wb * sh.l[warp][row]);
                m = M;
#pragma unroll
                for (int e = 0; e < RUN; e += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(mine + row * C::ROW + e);
                    at(h, e) = fmaf(wa, at(h, e), wb * v.x);
                    at(h, e + 1) = fmaf(wa, at(h, e + 1), wb * v.y);
                    at(h, e + 2) = fmaf(wa, at(h, e + 2), wb * v.z);
                    at(h, e + 3) = fmaf(wa, at(h, e + 3), wb * v.w);
                }
            }
            __syncwarp(); // every lane has read the rows' maxima and sums
            put();
        }
        sync_consumers();
        const bool whole = cons.seg >= lo && cons.seg + cons.n <= hi; // no other CTA has tiles of it
        float* part = a.parts + (int64_t)(2 * cta + (cons.seg > lo ? 1 : 0)) * kKv4PartFloats;
        for (int e = tid; e < G * (DH / 4); e += kThreads) {
            const int row = e / (DH / 4), q4 = e % (DH / 4); // 4 elements at 4 * q4
            float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) M = fmaxf(M, sh.m[i][row]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            const float* src = join + row * C::ROW + (q4 / (DH / 16)) * C::LANE + (q4 % (DH / 16)) * 4;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const float c = join_weight(sh.m[i][row], M);
                const float4 v = *reinterpret_cast<const float4*>(src + i * C::WARP);
                L = fmaf(c, sh.l[i][row], L);
                acc.x = fmaf(c, v.x, acc.x);
                acc.y = fmaf(c, v.y, acc.y);
                acc.z = fmaf(c, v.z, acc.z);
                acc.w = fmaf(c, v.w, acc.w);
            }
            if (whole) {
                finish(a, (int64_t)cons.b * a.H_q + cons.r * G + row, q4 * 4, acc, M, L);
            } else {
                *reinterpret_cast<float4*>(part + row * DH + q4 * 4) = acc;
                if (q4 == 0) {
                    part[16 * 128 + row] = M;
                    part[16 * 128 + 16 + row] = L;
                }
            }
        }
    }
}

// Joins the partials of the segments that several CTAs share. CTA (c, y): the segment whose first block is in
// CTA c's slice and whose last is not (there is at most one), heads kJoinRows y and on; kJoinGroups warps a
// head, each with every kJoinGroups-th partial, in a fixed order. Bound by latency (37 partials of 16 heads for each
// KV head of one long sequence). It is launched early, but an SM has registers for it only once its attention CTA, which
// holds all of them, has left: its start overlaps the attention's last CTAs.
constexpr int kJoinRows = 4, kJoinGroups = 4, kJoinThreads = kJoinRows * kJoinGroups * 32;

template <int DH, bool GIVEN>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(Kv4DecodeArgs a)
{
    constexpr int L4 = DH / 4; // lanes with 4 elements each
    __shared__ int warp_units[kJoinThreads / 32], found[4];
    __shared__ float4 sv[kJoinRows][kJoinGroups][L4];
    __shared__ float2 sml[kJoinRows][kJoinGroups];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (a.w_out) pdl_trigger(); // for the weights; else the call ends here
    const Work<GIVEN> w{a};
    int before, b_lo, b_hi;
    const int total = total_units<kJoinThreads>(w, warp_units, before, b_lo, b_hi);
    const int n_cta = min((total + kJoin<GIVEN> + kBlocks - 1) / (kJoin<GIVEN> + kBlocks), kKv4Ctas);
    const int c0 = blockIdx.x;
    if (tid == 0) found[0] = -1;
    __syncthreads();
    const int lo = c0 < n_cta ? (int)((int64_t)total * c0 / n_cta) : 0, hi = c0 < n_cta ? (int)((int64_t)total * (c0 + 1) / n_cta) : 0;
    for (int b = b_lo; b < b_hi; ++b) { // the segment of the slice's last unit
        const int u = w.units(a.lens[b]), n = u * a.H_kv;
        if (hi > before && hi <= before + n) {
            const int r = (hi - 1 - before) / u, seg = before + r * u + kJoin<GIVEN>;
            if (seg >= lo && seg < hi && seg + u - kJoin<GIVEN> > hi) {
                found[0] = b;
                found[1] = r;
                found[2] = seg;
                found[3] = u - kJoin<GIVEN>;
            }
        }
        before += n;
    }
    __syncthreads();
    pdl_wait();
    const int b = found[0], row = blockIdx.y * kJoinRows + warp / kJoinGroups, grp = warp % kJoinGroups, G = a.H_q / a.H_kv;
    if (b < 0) return;
    const int c1 = (int)(((int64_t)(found[2] + found[3]) * n_cta - 1) / total), np = c1 - c0 + 1;
    // slot of CTA c: the segment is its slice's first unless the slice starts before it (only c0's can)
    const float* parts = a.parts + (int64_t)2 * c0 * kKv4PartFloats;
    const int first = found[2] > lo ? 1 : 0;
    float M = -CUDART_INF_F, L = 0.f;
    float4 acc = {};
    if (row < G) {
#pragma unroll 8
        for (int c = grp; c < np; c += kJoinGroups) {
            const float* p = parts + (int64_t)(c == 0 ? first : 2 * c) * kKv4PartFloats;
            const float4 v = lane < L4 ? reinterpret_cast<const float4*>(p + row * DH)[lane] : float4{};
            merge(M, L, acc, p[16 * 128 + row], p[16 * 128 + 16 + row], v);
        }
        if (lane < L4) sv[warp / kJoinGroups][grp][lane] = acc;
        if (lane == 0) sml[warp / kJoinGroups][grp] = make_float2(M, L);
    }
    __syncthreads();
    if (row < G && grp == 0 && lane < L4) {
#pragma unroll
        for (int i = 1; i < kJoinGroups; ++i) {
            const float2 ml = sml[warp / kJoinGroups][i];
            merge(M, L, acc, ml.x, ml.y, sv[warp / kJoinGroups][i][lane]);
        }
        finish(a, (int64_t)b * a.H_q + found[1] * G + row, lane * 4, acc, M, L);
    }
}

// Accumulated weights, after the attention (they need the final lse): K is read once more. A warp takes 32
// visible keys at a time and writes decay * w_in plus the group's sum of softmax weights; with given blocks
// the keys of the others get decay * w_in alone. 16 sequences in [1K, 16K] with 64 heads on 4: 21 us, of which
// reading K, w_in and writing w_out are 7; conversions, MMAs and the latency of short slices are the rest.
constexpr int kWThreads = 256;

template <int DH, bool GIVEN, bool NARROW>
__global__ void __launch_bounds__(kWThreads, 2) kv4_weights_kernel(Kv4DecodeArgs a)
{
    using C = Cfg<DH>;
    __shared__ int warp_units[kWThreads / 32], b0, seg0;
    __shared__ uint4 q[DH / 16][32]; // Q fragments of the segment
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int G = a.H_q / a.H_kv;
    const Work<false> w{a}; // all visible blocks
    int before, b_lo, b_hi;
    const int total = total_units<kWThreads>(w, warp_units, before, b_lo, b_hi);
    const int lo = (int)((int64_t)total * blockIdx.x / gridDim.x), hi = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
    if (lo >= hi) {
        pdl_wait();
        return;
    }
    for (int b = b_lo; b < b_hi; ++b) {
        const int n = w.units(a.lens[b]) * a.H_kv;
        if (lo >= before && lo < before + n) {
            b0 = b;
            seg0 = before;
        }
        before += n;
    }
    __syncthreads();
    bool waited = GIVEN; // for the lse; for the blocks too, at once
    if (GIVEN) pdl_wait();
    const bool rest = !(a.w_in == a.w_out && a.decay == 1.f); // keys of other blocks change too
    Walk<false> cons;
    for (cons.begin(w, b0, seg0, lo, hi); cons.more(); cons.next_segment(w)) {
        if (cons.pos >= cons.end) continue;
        float f0, f1;
        __syncthreads(); // the segment before is done with q
        {
            uint32_t qf[DH / 16][4];
            load_q<DH, NARROW>(a, cons.b, cons.r, G, g, t, qf, f0, f1);
            if (warp == 0) store_q<DH, NARROW>(q, qf, lane);
        }
        __syncthreads();
        float z0, z1;
        int mine = -1; // given blocks: the first key of this lane's
        if (GIVEN) {
            bool bad;
            mine = Work<true>{a}.given_key0(cons.b, cons.r, cons.len, bad);
        }
        const int64_t row0 = ((int64_t)cons.b * a.H_kv + cons.r) * a.L_max;
        // the key whose weight ends in this lane (of the sums below)
        const int my_key = NARROW ? 8 * t + (g >> 1) + 4 * (g & 1) : 8 * (g >> 1) + t + 4 * (g & 1), last = min(cons.len, (cons.end - cons.seg) * kBk);
        int next = (cons.pos - cons.seg) * kBk + warp * kTile; // first key of the warp's next tile
        // a tile's rows and the lane's old weight are loaded one tile ahead
        struct Tile {
            KTile<DH> k;
            int key0; // first key; last or more: no tile
            bool chosen;
            float old;
        };
        auto fetch = [&](Tile& x) {
            for (;; next += kWThreads) {
                x.key0 = next;
                if (next >= last) return;
                x.chosen = !GIVEN || __any_sync(0xffffffffu, mine == next / kBk * kBk);
                if (x.chosen || rest) break;
            }
            const int64_t row = row0 + next;
            if (x.chosen) x.k.load(a.k_codes + row * C::CODE, a.k_scales + row * C::NG, g, t);
            x.old = a.w_in && next + my_key < last ? a.decay * a.w_in[row + my_key] : 0.f;
            next += kWThreads;
        };
        auto finish_tile = [&](const Tile& now) {
            float add = 0.f;
            if (now.chosen) {
                float x[NARROW ? 2 : 4][4];
                scores<DH, NARROW>(now.k, q, lane, x);
                // the heads' weights of the lane's keys (v = 2 n + e, or 2 m + u), summed over the lanes that hold the key's
                // other heads: these are as many as the keys, and each ends with one
                constexpr int KEYS = NARROW ? 4 : 8;
                float p[KEYS];
#pragma unroll
                for (int v = 0; v < KEYS; ++v)
                    p[v] = NARROW ? ex2_approx(fmaf(x[v >> 1][2 * (v & 1)], f0, -z0)) + ex2_approx(fmaf(x[v >> 1][2 * (v & 1) + 1], f1, -z1))
                                  : ex2_approx(fmaf(x[v >> 1][v & 1], f0, -z0)) + ex2_approx(fmaf(x[v >> 1][2 + (v & 1)], f1, -z1));
#pragma unroll
                for (int half = KEYS / 2; half > 0; half >>= 1) {
                    const bool up = (NARROW ? t : g) & half;
#pragma unroll
                    for (int v = 0; v < half; ++v) {
                        const float give = up ? p[v] : p[v + half], keep = up ? p[v + half] : p[v];
                        p[v] = keep + __shfl_xor_sync(0xffffffffu, give, NARROW ? half : 4 * half);
                    }
                }
                add = p[0];
            }
            if (now.key0 + my_key < last) a.w_out[row0 + now.key0 + my_key] = now.old + add;
        };
        Tile even, odd;
        fetch(even);
        if (!waited) { // q and the first keys are on their way
            pdl_wait();
            waited = true;
        }
        const float* lse = a.lse + (int64_t)cons.b * a.H_q + cons.r * G;
        const int h0 = NARROW ? 2 * t : g, h1 = NARROW ? 2 * t + 1 : g + 8;
        z0 = h0 < G ? lse[h0] * 1.4426950408889634f : CUDART_INF_F; // rows past the heads weigh nothing
        z1 = h1 < G ? lse[h1] * 1.4426950408889634f : CUDART_INF_F;
        while (even.key0 < last) {
            fetch(odd);
            finish_tile(even);
            if (odd.key0 >= last) break;
            fetch(even);
            finish_tile(odd);
        }
    }
    if (!waited) pdl_wait(); // a slice without blocks
}

template <int DH, bool GIVEN, bool NARROW>
cudaError_t launch(const Kv4DecodeArgs& a, cudaStream_t s)
{
    static SmemOptIn opt_in;
    if (cudaError_t e = opt_in.set(kv4_decode_kernel<DH, GIVEN, NARROW>, Cfg<DH>::SMEM)) return e;
    trace_begin(s);
    const int smem = Cfg<DH>::SMEM;
    // only kernels of one call overlap (a kernel before it may write the lengths, which are read at once)
    cudaError_t e = cudaSuccess;
    if (GIVEN && a.after_topk)
        e = launch_pdl(kv4_decode_kernel<DH, GIVEN, NARROW>, dim3(kKv4Ctas), kLaunch, smem, s, a);
    else
        kv4_decode_kernel<DH, GIVEN, NARROW><<<kKv4Ctas, kLaunch, smem, s>>>(a);
    if (e == cudaSuccess)
        e = launch_pdl(kv4_join_kernel<DH, GIVEN>, dim3(kKv4Ctas, (a.H_q / a.H_kv + kJoinRows - 1) / kJoinRows), kJoinThreads, 0, s, a);
    trace_end(s, MSA_KERNEL_KV4_ATTN);
    note_launch(2);
    if (a.w_out && e == cudaSuccess) {
        trace_begin(s);
        e = launch_pdl(kv4_weights_kernel<DH, GIVEN, NARROW>, dim3(2 * kKv4Ctas), kWThreads, 0, s, a);
        trace_end(s, MSA_KERNEL_KV4_WEIGHTS);
        note_launch(1);
    }
    return e == cudaSuccess ? cudaGetLastError() : e;
}

} // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t s)
{
    // up to 8 heads a KV head: keys are the rows of the products and heads the 8 columns, half the tensor-core
    // work of 16 rows that are mostly padding. 16 sequences in [8K, 16K] of 8 KV heads of 128 take 51 us with 1
    // head each, 51 with 8 and 67 with 16; with 16 rows for all 61, 63 and 68.
    const bool narrow = a.H_q / a.H_kv <= 8, given = a.block_idx != nullptr;
    if (a.d_h == 128) {
        if (given) return narrow ? launch<128, true, true>(a, s) : launch<128, true, false>(a, s);
        return narrow ? launch<128, false, true>(a, s) : launch<128, false, false>(a, s);
    }
    if (given) return narrow ? launch<64, true, true>(a, s) : launch<64, true, false>(a, s);
    return narrow ? launch<64, false, true>(a, s) : launch<64, false, false>(a, s);
}

} // namespace msa
