// kv4_decode.cu -- single-token attention over the 4-bit key/value cache (format: kv4.cuh).
//
// For head h of KV head r, over the visible keys j (all j < len, or those of the given blocks):
//   x_j = q[h] . K[j] / sqrt(d_h),  out[h] = sum_j softmax(x)_j V[j],  lse[h] = log sum_j exp(x_j)
//   w_out[r][j] = decay * w_in[r][j] + sum over the heads of r of softmax(x)_j      (optional)
//
// Bound by reading the cache (d_h + d_h / 8 bytes per token and KV head). One CTA per SM walks an
// equal contiguous slice of the flattened list of 32-key tiles of all (sequence, KV head) pairs, so
// ragged batches and single long sequences load every SM alike. Inside a CTA every warp takes every
// kWarps-th tile, streams it by bulk copies into a ring of its own (no CTA-wide synchronisation in
// the loop) and keeps a running maximum, sum and output of its tiles; the warps' results are joined
// at the end of each (sequence, KV head), and those of a pair that several CTAs share by the CTA
// that finishes it last, in a fixed order (results do not depend on timing).
//
// The heads of a KV head are the 16 rows of mma.sync m16n8k16 (a 16-row problem is below the 128-row
// tcgen05 tile). E2M1 codes become fp16 pairs with the hardware conversion, times the E4M3 scale
// (both exact); no step goes through shared memory, because both products may sum in any order:
//   S = Q K^T: lane (g, t) holds d_h / 4 consecutive codes of key row g, so element t * d_h / 4 + 4 ks
//     + {0, 1, 2, 3} of a row is the contraction index {2t, 2t + 1, 2t + 8, 2t + 9} of step ks, for Q alike;
//   O = P V: lane (g, t) holds d_h / 8 consecutive codes of four keys, so column g of output tile n is
//     element g * d_h / 8 + n, and the nibbles of two keys are joined before the conversion.
// q is held in fp16 as q * 2^-e with e the exponent of the row's largest |q| (elements lose bits only
// below 2^-14 of it, an error of 2^-25 of it at most); P in fp16 relative to a reference at most 2^15
// below its largest value (relative error 2^-12; weights below 2^-24 of fp16's unit, 2^-31 of the
// largest, are the first to lose bits). Sums, maxima and outputs are fp32.
#include <math_constants.h>

#include "kv4.cuh"
#include "mma_sync.cuh"

namespace msa {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;  // keys of a tile
constexpr int kStages = 4; // tiles in flight per warp
constexpr int kTilesPerBlock = kBk / kTile;
constexpr float kHeadroom = 7.f; // P's reference: log2 units below the maximum it was set from
constexpr float kRaise = 15.f;   // P stays below 2^15, within fp16

template <int DH>
struct Cfg {
    static constexpr int CODE = DH / 2, NG = DH / 16; // bytes of a row's codes, scales
    static constexpr int K_CODES = 0, V_CODES = kTile * CODE, K_SCALES = 2 * kTile * CODE,
                         V_SCALES = K_SCALES + kTile * NG, STAGE = V_SCALES + kTile * NG;
    // join scratch: [warp][16 rows][4 lanes][DH / 4], padded so that 16-byte accesses do not conflict
    static constexpr int LANE = DH / 4 + 4, ROW = 4 * LANE, WARP = 16 * ROW;
    static constexpr int SMEM = kWarps * kStages * STAGE + kWarps * WARP * 4;
};

struct Shared {
    uint64_t full[kWarps][kStages];
    float m[kWarps][16], l[kWarps][16];
    int warp_tiles[kWarps];
    int b0, seg0;  // sequence holding the slice's first tile, first tile of that sequence
    int last;      // this CTA joins the partials of the segment
    int abort_flag;
};

// The flattened list: sequence b owns H_kv * tiles(b) tiles, KV head by KV head.
struct Work {
    const Kv4DecodeArgs& a;
    __device__ __forceinline__ bool valid(int len) const { return len >= a.min_len && len <= a.L_max; }
    __device__ __forceinline__ int tiles(int b) const // per KV head
    {
        const int len = a.lens[b];
        if (!valid(len) || len == 0) return 0;
        return a.block_idx ? a.k * kTilesPerBlock : (len + kTile - 1) / kTile;
    }
    // Tile `tile` of (b, r): its first key and how many of its keys are visible (0: nothing to read).
    __device__ __forceinline__ int keys(int b, int r, int tile, int len, int& key0) const
    {
        if (!a.block_idx) {
            key0 = tile * kTile;
            return min(kTile, len - key0);
        }
        const int slot = tile / kTilesPerBlock;
        const int32_t* sel = a.block_idx + ((int64_t)b * a.H_kv + r) * a.k;
        const int blk = sel[slot];
        if (blk < 0 || blk > (len - 1) / kBk || (slot > 0 && blk <= sel[slot - 1])) return 0; // padding, or reported by the check
        key0 = blk * kBk + (tile % kTilesPerBlock) * kTile;
        return max(0, min(kTile, len - key0));
    }
};

// Block-wide: number of tiles of all sequences, and for the caller's slice its first sequence.
// Sequences are split among the threads in contiguous runs.
__device__ __forceinline__ int64_t total_tiles(const Work& w, Shared& sh, int64_t& before, int& b_lo, int& b_hi)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (w.a.B + kThreads - 1) / kThreads;
    b_lo = min(w.a.B, tid * per);
    b_hi = min(w.a.B, b_lo + per);
    int n = 0;
    for (int b = b_lo; b < b_hi; ++b) n += w.tiles(b) * w.a.H_kv;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sh.warp_tiles[warp] = x;
    __syncthreads();
    int64_t total = 0;
    before = x - n;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const int y = sh.warp_tiles[i];
        if (i < warp) before += y;
        total += y;
    }
    return total;
}

// A warp's walk over its tiles of the CTA's slice [lo, hi): segment by segment (a segment is a
// (sequence, KV head)), every kWarps-th tile of the part of it that lies in the slice.
struct Walk {
    int b, r, n;       // sequence, KV head, tiles of a segment of this sequence
    int64_t seg;       // first tile of the segment
    int64_t lo, hi;    // the slice
    int64_t tile, end; // next tile of this warp, end of the segment's part
    int len;

    __device__ __forceinline__ void enter(int warp)
    {
        tile = (seg > lo ? seg : lo) + warp;
        end = seg + n < hi ? seg + n : hi;
    }
    __device__ __forceinline__ void begin(const Work& w, int b0, int64_t seq0, int64_t lo_, int64_t hi_, int warp)
    {
        lo = lo_;
        hi = hi_;
        b = b0;
        n = w.tiles(b);
        len = w.a.lens[b];
        r = (int)((lo - seq0) / n);
        seg = seq0 + (int64_t)r * n;
        enter(warp);
    }
    __device__ __forceinline__ bool more() const { return seg < hi; }
    __device__ __forceinline__ void next_segment(const Work& w, int warp)
    {
        seg += n;
        if (++r == w.a.H_kv) {
            r = 0;
            if (seg < hi) {
                do { ++b; } while ((n = w.tiles(b)) == 0);
                len = w.a.lens[b];
            }
        }
        enter(warp);
    }
};

// A fragments of q's rows g and g + 8 (rows past the G heads are zero) in fp16, and the factors that
// turn sums of the products into logits in log2 units.
template <int DH>
__device__ __forceinline__ void load_q(const Kv4DecodeArgs& a, int b, int r, int G, int g, int t, uint32_t (&qf)[DH / 16][4],
                                       float& f0, float& f1)
{
    const float base = a.k_scale * rsqrtf((float)DH) * 1.4426950408889634f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
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
        (half ? f1 : f0) = base * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) // pair i: elements 2 i, 2 i + 1 of the lane's run
            qf[i / 2][2 * (i & 1) + half] = pack_f16x2(bf16_lo(x[i]) * down, bf16_hi(x[i]) * down);
    }
}

// x[n][e] = the fp32 sums of q's rows (e < 2: g, else g + 8) with key 8 n + t + 4 (e & 1) of a tile
// whose codes and scales start at kc and ks (column 2u of step n is key 8 n + u, column 2u + 1 key
// 8 n + u + 4, which spreads O's reads of V over the shared-memory banks).
template <int DH>
__device__ __forceinline__ void scores(const uint8_t* kc, const uint8_t* ks, const uint32_t (&qf)[DH / 16][4], int g, int t,
                                       float (&x)[4][4])
{
#pragma unroll
    for (int n = 0; n < 4; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
        const int key = 8 * n + (g >> 1) + 4 * (g & 1);
        uint32_t c[DH / 32], s[2];
        if constexpr (DH == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(kc + key * 64 + t * 16);
            c[0] = v.x, c[1] = v.y, c[2] = v.z, c[3] = v.w;
            const uint32_t sc = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks + key * 8 + t * 2));
            s[0] = prmt(sc, sc, 0x1010);
            s[1] = prmt(sc, sc, 0x3232);
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(kc + key * 32 + t * 8);
            c[0] = v.x, c[1] = v.y;
            const uint32_t sc = e4m3x2_to_f16x2(ks[key * 4 + t]);
            s[0] = prmt(sc, sc, 0x1010);
        }
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
            uint32_t h[4];
            e2m1x8_to_f16x2(c[i], h);
            mma_f16_16816(x[n], qf[2 * i], mul_f16x2(h[0], s[i / 2]), mul_f16x2(h[1], s[i / 2]));
            mma_f16_16816(x[n], qf[2 * i + 1], mul_f16x2(h[2], s[i / 2]), mul_f16x2(h[3], s[i / 2]));
        }
    }
}

// ex2(-inf) = 0 keeps empty rows and tiles out of the joins.
__device__ __forceinline__ float join_weight(float m, float M) { return m == -CUDART_INF_F ? 0.f : ex2_approx(m - M); }

// One output element run: 4 consecutive elements of one head.
__device__ __forceinline__ void store_out(const Kv4DecodeArgs& a, int64_t row, int d, const float4& o, float inv)
{
    *reinterpret_cast<uint2*>(a.out + row * a.d_h + d) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1) kv4_decode_kernel(Kv4DecodeArgs a)
{
    using C = Cfg<DH>;
    constexpr int KS = DH / 16; // contraction steps of S
    constexpr int NT = DH / 8;  // output tiles of O
    extern __shared__ __align__(128) uint8_t ring_smem[];
    __shared__ Shared sh;
    float* join = reinterpret_cast<float*>(ring_smem + kWarps * kStages * C::STAGE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int G = a.H_q / a.H_kv;
    const Work w{a};

    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[warp][i], 1);
        fence_mbar_init();
    }
    if (tid == 0) sh.abort_flag = 0;
    int64_t before;
    int b_lo, b_hi;
    const int64_t total = total_tiles(w, sh, before, b_lo, b_hi);
    // every CTA gets at least one tile per warp where there are that many
    int64_t n_cta = (total + kWarps - 1) / kWarps;
    n_cta = n_cta < gridDim.x ? n_cta : gridDim.x;
    const int cta = blockIdx.x;
    // sequences without keys (and rejected ones) have no tiles: CTA 0 answers for them
    if (cta == 0) {
        for (int b = warp; b < a.B; b += kWarps) {
            const int len = a.lens[b];
            if (!w.valid(len)) {
                if (lane == 0) report_error(a.err, MSA_ERR_DEVICE_CHECK, 200 + b);
            } else if (len == 0) {
                for (int e = lane; e < a.H_q * DH / 2; e += 32)
                    reinterpret_cast<uint32_t*>(a.out + (int64_t)b * a.H_q * DH)[e] = 0u;
                if (a.lse)
                    for (int e = lane; e < a.H_q; e += 32) a.lse[(int64_t)b * a.H_q + e] = -CUDART_INF_F;
            } else if (a.block_idx) {
                for (int e = lane; e < a.H_kv * a.k; e += 32) {
                    const int32_t* sel = a.block_idx + (int64_t)b * a.H_kv * a.k + e;
                    const bool ok = *sel >= -1 && *sel <= (len - 1) / kBk && (e % a.k == 0 || *sel < 0 || sel[-1] < *sel);
                    if (!ok) report_error(a.err, MSA_ERR_DEVICE_CHECK, 210);
                }
            }
        }
    }
    if (cta >= n_cta) return;
    const int64_t lo = total * cta / n_cta, hi = total * (cta + 1) / n_cta;
    for (int b = b_lo; b < b_hi; ++b) {
        const int64_t n = (int64_t)w.tiles(b) * a.H_kv;
        if (lo >= before && lo < before + n) {
            sh.b0 = b;
            sh.seg0 = (int)before;
        }
        before += n;
    }
    __syncthreads();

    uint8_t* ring = ring_smem + warp * kStages * C::STAGE;
    uint64_t* full = sh.full[warp];
    volatile int* abort_flag = &sh.abort_flag;
    Walk prod, cons;
    cons.begin(w, sh.b0, sh.seg0, lo, hi, warp);
    prod = cons;
    int64_t issued = 0, used = 0;
    // Starts the copies of the warp's next tile that has visible keys; false when there is none.
    auto issue = [&]() {
        while (prod.more()) {
            while (prod.tile < prod.end) {
                int key0;
                const int nk = w.keys(prod.b, prod.r, (int)(prod.tile - prod.seg), prod.len, key0);
                prod.tile += kWarps;
                if (nk == 0) continue;
                if (lane == 0) {
                    uint8_t* st = ring + (issued % kStages) * C::STAGE;
                    uint64_t* bar = &full[issued % kStages];
                    const int64_t row = ((int64_t)prod.b * a.H_kv + prod.r) * a.L_max + key0; // L_max is whole blocks
                    mbar_arrive_expect_tx(bar, C::STAGE);
                    bulk_load(st + C::K_CODES, a.k_codes + row * C::CODE, kTile * C::CODE, bar);
                    bulk_load(st + C::K_SCALES, a.k_scales + row * C::NG, kTile * C::NG, bar);
                    bulk_load(st + C::V_CODES, a.v_codes + row * C::CODE, kTile * C::CODE, bar);
                    bulk_load(st + C::V_SCALES, a.v_scales + row * C::NG, kTile * C::NG, bar);
                }
                ++issued;
                return;
            }
            prod.next_segment(w, warp);
        }
    };
    for (int i = 0; i < kStages; ++i) issue();

    bool ok = true;
    for (; cons.more(); cons.next_segment(w, warp)) {
        uint32_t qf[KS][4];
        float f0, f1;
        load_q<DH>(a, cons.b, cons.r, G, g, t, qf, f0, f1);
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f; // references, this lane's sums

        for (; ok && cons.tile < cons.end; cons.tile += kWarps) {
            int key0;
            const int nk = w.keys(cons.b, cons.r, (int)(cons.tile - cons.seg), cons.len, key0);
            if (nk == 0) continue;
            const int st = (int)(used % kStages);
            ok = wait_or_abort(&full[st], (uint32_t)((used / kStages) & 1), abort_flag, a.err, 60, kWaitLimit);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++used;
            const uint8_t* s = ring + st * C::STAGE;
            // ------------------------------------------------------------ S = Q K^T
            float x[4][4];
            scores<DH>(s + C::K_CODES, s + C::K_SCALES, qf, g, t, x);
            // ------------------------------------------------------------ softmax
            float mx0 = -CUDART_INF_F, mx1 = -CUDART_INF_F;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool seen = 8 * n + t + 4 * e < nk;
                    x[n][e] = seen ? x[n][e] * f0 : -CUDART_INF_F;
                    x[n][2 + e] = seen ? x[n][2 + e] * f1 : -CUDART_INF_F;
                    mx0 = fmaxf(mx0, x[n][e]);
                    mx1 = fmaxf(mx1, x[n][2 + e]);
                }
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
            }
            // the references move up only when P would leave [0, 2^15): exact, and rare
            if (__any_sync(0xffffffffu, mx0 > m0 + kRaise || mx1 > m1 + kRaise)) {
                const float n0 = mx0 > m0 + kRaise ? mx0 - kHeadroom : m0, n1 = mx1 > m1 + kRaise ? mx1 - kHeadroom : m1;
                const float r0 = join_weight(m0, n0), r1 = join_weight(m1, n1);
                m0 = n0;
                m1 = n1;
                l0 *= r0;
                l1 *= r1;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][0] *= r0;
                    o[n][1] *= r0;
                    o[n][2] *= r1;
                    o[n][3] *= r1;
                }
            }
            uint32_t pf[2][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float p0 = ex2_approx(x[n][0] - m0), p1 = ex2_approx(x[n][1] - m0);
                const float p2 = ex2_approx(x[n][2] - m1), p3 = ex2_approx(x[n][3] - m1);
                l0 += p0 + p1;
                l1 += p2 + p3;
                pf[n >> 1][(n & 1) * 2] = pack_f16x2(p0, p1);
                pf[n >> 1][(n & 1) * 2 + 1] = pack_f16x2(p2, p3);
            }
            // ------------------------------------------------------------ O += P V, 16 keys a step
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t sc[2], wv[4][DH / 64]; // keys 16 j + t + {0, 4, 8, 12}
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int key = 16 * j + t + 4 * u;
                    if constexpr (DH == 128) {
                        const uint2 c = *reinterpret_cast<const uint2*>(s + C::V_CODES + key * 64 + g * 8);
                        wv[u][0] = c.x;
                        wv[u][1] = c.y;
                    } else {
                        wv[u][0] = *reinterpret_cast<const uint32_t*>(s + C::V_CODES + key * 32 + g * 4);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int key = 16 * j + t + 8 * u;
                    const int gs = DH == 128 ? g : g >> 1;
                    uint32_t sa = s[C::V_SCALES + key * C::NG + gs], sb = s[C::V_SCALES + (key + 4) * C::NG + gs];
                    // rows past the length hold anything, NaN scales among it: they weigh 0 and must be finite
                    if (key >= nk) sa = 0u;
                    if (key + 4 >= nk) sb = 0u;
                    sc[u] = e4m3x2_to_f16x2(sa | (sb << 8));
                }
#pragma unroll
                for (int i = 0; i < DH / 64; ++i) {
                    uint32_t b0[2][4], b1[2][4]; // [even, odd elements][4]
                    e2m1x8_to_f16x2((wv[0][i] & 0x0F0F0F0Fu) | ((wv[1][i] << 4) & 0xF0F0F0F0u), b0[0]);
                    e2m1x8_to_f16x2(((wv[0][i] >> 4) & 0x0F0F0F0Fu) | (wv[1][i] & 0xF0F0F0F0u), b0[1]);
                    e2m1x8_to_f16x2((wv[2][i] & 0x0F0F0F0Fu) | ((wv[3][i] << 4) & 0xF0F0F0F0u), b1[0]);
                    e2m1x8_to_f16x2(((wv[2][i] >> 4) & 0x0F0F0F0Fu) | (wv[3][i] & 0xF0F0F0F0u), b1[1]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        mma_f16_16816(o[8 * i + e], pf[j], mul_f16x2(b0[e & 1][e >> 1], sc[0]),
                                      mul_f16x2(b1[e & 1][e >> 1], sc[1]));
                }
            }
            __syncwarp(); // every lane has read the stage
            issue();
        }
        // ------------------------------------------------------------ join the warps
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, d);
            l1 += __shfl_xor_sync(0xffffffffu, l1, d);
        }
        if (t == 0) {
            sh.m[warp][g] = m0;
            sh.m[warp][g + 8] = m1;
            sh.l[warp][g] = l0;
            sh.l[warp][g + 8] = l1;
        }
        float* mine = join + warp * C::WARP + t * C::LANE;
#pragma unroll
        for (int half = 0; half < 2; ++half) // row g + 8 half: elements t * DH / 4 + (0 .. DH / 4)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int n = 0; n < NT; n += 4)
                    *reinterpret_cast<float4*>(mine + (g + 8 * half) * C::ROW + c * NT + n) =
                        make_float4(o[n][2 * half + c], o[n + 1][2 * half + c], o[n + 2][2 * half + c], o[n + 3][2 * half + c]);
        __syncthreads();
        const bool whole = cons.seg >= lo && cons.seg + cons.n <= hi; // no other CTA has tiles of it
        float* part = a.parts + (int64_t)(2 * cta + (cons.seg > lo ? 1 : 0)) * kKv4PartFloats;
        for (int e = tid; e < G * (DH / 4); e += kThreads) {
            const int row = e / (DH / 4), q4 = e % (DH / 4); // 4 elements at 4 * q4
            float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sh.m[i][row]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            const float* src = join + row * C::ROW + (q4 / (DH / 16)) * C::LANE + (q4 % (DH / 16)) * 4;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float c = join_weight(sh.m[i][row], M);
                const float4 v = *reinterpret_cast<const float4*>(src + i * C::WARP);
                L = fmaf(c, sh.l[i][row], L);
                acc.x = fmaf(c, v.x, acc.x);
                acc.y = fmaf(c, v.y, acc.y);
                acc.z = fmaf(c, v.z, acc.z);
                acc.w = fmaf(c, v.w, acc.w);
            }
            if (whole) {
                const int64_t orow = (int64_t)cons.b * a.H_q + cons.r * G + row;
                store_out(a, orow, q4 * 4, acc, L > 0.f ? a.v_scale / L : 0.f);
                if (a.lse && q4 == 0) a.lse[orow] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -CUDART_INF_F;
            } else {
                *reinterpret_cast<float4*>(part + row * DH + q4 * 4) = acc;
                if (q4 == 0) {
                    part[16 * 128 + row] = M;
                    part[16 * 128 + 16 + row] = L;
                }
            }
        }
        if (!whole) {
            // the CTAs with tiles of this segment: that of its first tile .. that of its last
            const int c0 = (int)(((cons.seg + 1) * n_cta - 1) / total), c1 = (int)(((cons.seg + cons.n) * n_cta - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) sh.last = atomicAdd(&a.arrived[c0], 1) == c1 - c0;
            __syncthreads();
            if (sh.last) {
                __threadfence();
                const int np = c1 - c0 + 1;
                const int64_t lo0 = total * c0 / n_cta;
                // slot of CTA c: the segment is its slice's first unless the slice starts before it (only c0's can)
                auto slot = [&](int c) { return a.parts + (int64_t)(2 * c + (c == c0 && cons.seg > lo0 ? 1 : 0)) * kKv4PartFloats; };
                for (int e = tid; e < G * (DH / 4); e += kThreads) {
                    const int row = e / (DH / 4), q4 = e % (DH / 4);
                    float M = -CUDART_INF_F, L = 0.f;
                    for (int c = 0; c < np; ++c) M = fmaxf(M, __ldcg(slot(c0 + c) + 16 * 128 + row));
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int c = 0; c < np; ++c) {
                        const float* p = slot(c0 + c);
                        const float cw = join_weight(__ldcg(p + 16 * 128 + row), M);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(p + row * DH + q4 * 4));
                        L = fmaf(cw, __ldcg(p + 16 * 128 + 16 + row), L);
                        acc.x = fmaf(cw, v.x, acc.x);
                        acc.y = fmaf(cw, v.y, acc.y);
                        acc.z = fmaf(cw, v.z, acc.z);
                        acc.w = fmaf(cw, v.w, acc.w);
                    }
                    const int64_t orow = (int64_t)cons.b * a.H_q + cons.r * G + row;
                    store_out(a, orow, q4 * 4, acc, L > 0.f ? a.v_scale / L : 0.f);
                    if (a.lse && q4 == 0) a.lse[orow] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -CUDART_INF_F;
                }
            }
        }
        __syncthreads(); // the join scratch is free again
    }
    // after an abort, copies may still be in flight: the shared memory must outlive them
    if (!ok && lane == 0)
        for (; used < issued; ++used) drain_wait(&full[used % kStages], (uint32_t)((used / kStages) & 1), a.err, 61, kWaitLimit);
}

// Accumulated weights, after the attention (they need the final lse): K is read once more, and every
// visible key of the list gets its group's sum of softmax weights.
template <int DH>
__global__ void __launch_bounds__(kThreads) kv4_weights_kernel(Kv4DecodeArgs a)
{
    using C = Cfg<DH>;
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int G = a.H_q / a.H_kv;
    const Work w{a};
    int64_t before;
    int b_lo, b_hi;
    const int64_t total = total_tiles(w, sh, before, b_lo, b_hi);
    const int64_t lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
    if (lo >= hi) return;
    for (int b = b_lo; b < b_hi; ++b) {
        const int64_t n = (int64_t)w.tiles(b) * a.H_kv;
        if (lo >= before && lo < before + n) {
            sh.b0 = b;
            sh.seg0 = (int)before;
        }
        before += n;
    }
    __syncthreads();
    Walk cons;
    for (cons.begin(w, sh.b0, sh.seg0, lo, hi, warp); cons.more(); cons.next_segment(w, warp)) {
        if (cons.tile >= cons.end) continue;
        uint32_t qf[DH / 16][4];
        float f0, f1;
        load_q<DH>(a, cons.b, cons.r, G, g, t, qf, f0, f1);
        const float* lse = a.lse + (int64_t)cons.b * a.H_q + cons.r * G;
        const float z0 = g < G ? lse[g] * 1.4426950408889634f : CUDART_INF_F; // rows past the heads weigh nothing
        const float z1 = g + 8 < G ? lse[g + 8] * 1.4426950408889634f : CUDART_INF_F;
        for (; cons.tile < cons.end; cons.tile += kWarps) {
            int key0;
            const int nk = w.keys(cons.b, cons.r, (int)(cons.tile - cons.seg), cons.len, key0);
            if (nk == 0) continue;
            const int64_t row = ((int64_t)cons.b * a.H_kv + cons.r) * a.L_max + key0;
            float x[4][4];
            scores<DH>(a.k_codes + row * C::CODE, a.k_scales + row * C::NG, qf, g, t, x);
            float mine = 0.f; // lane (g, t): key 8 (g / 2) + t + 4 (g % 2)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float p = ex2_approx(fmaf(x[n][e], f0, -z0)) + ex2_approx(fmaf(x[n][2 + e], f1, -z1));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) p += __shfl_xor_sync(0xffffffffu, p, d);
                    if (g == 2 * n + e) mine = p;
                }
            const int key = 8 * (g >> 1) + t + 4 * (g & 1);
            if (key < nk) {
                // given blocks: kv4_decay_kernel has written decay * w_in to every visible key
                const float old = a.block_idx ? a.w_out[row + key] : (a.w_in ? a.decay * a.w_in[row + key] : 0.f);
                a.w_out[row + key] = old + mine;
            }
        }
    }
}

// w_out = decay * w_in (0 without w_in) on the visible keys of every valid sequence.
__global__ void __launch_bounds__(256) kv4_decay_kernel(Kv4DecodeArgs a)
{
    const int b = blockIdx.y / a.H_kv;
    const int len = a.lens[b];
    if (len < a.min_len || len > a.L_max) return;
    const int64_t base = (int64_t)blockIdx.y * a.L_max;
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < len; j += (int64_t)gridDim.x * 256)
        a.w_out[base + j] = a.w_in ? a.decay * a.w_in[base + j] : 0.f;
}

template <int DH>
cudaError_t launch(const Kv4DecodeArgs& a, cudaStream_t s)
{
    cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<DH>::SMEM);
    if (e != cudaSuccess) return e;
    trace_begin(s);
    kv4_decode_kernel<DH><<<kKv4Ctas, kThreads, Cfg<DH>::SMEM, s>>>(a);
    trace_end(s, MSA_KERNEL_KV4_ATTN);
    note_launch(1);
    if (!a.w_out) return cudaGetLastError();
    trace_begin(s);
    if (a.block_idx && !(a.w_in == a.w_out && a.decay == 1.f)) {
        kv4_decay_kernel<<<dim3(8, a.B * a.H_kv), 256, 0, s>>>(a);
        note_launch(1);
    }
    kv4_weights_kernel<DH><<<2 * kKv4Ctas, kThreads, 0, s>>>(a);
    note_launch(1);
    trace_end(s, MSA_KERNEL_KV4_WEIGHTS);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t s)
{
    return a.d_h == 128 ? launch<128>(a, s) : launch<64>(a, s);
}

} // namespace msa
