// kv4.cu -- rows into and out of the 4-bit key/value cache (format: kv4.cuh).
//
// append: for every 16 elements x of a new row
//   y = fl32(x / t), a = max |y|, s = E4M3(min(fl32(a / 6), 448)), code = E2M1(fl32(y / s))
// with all roundings to nearest even and codes saturating at 6; s = 0 gives zero codes. read: the
// values code * s * t rounded to bf16. CTAs take one head's consecutive rows of K and of V, so that the
// head-major cache side is written (read) in whole contiguous runs and the token-major side in whole
// rows of d_h elements; the rows' places are looked up once per CTA.
#include "kv4.cuh"

namespace msa {

namespace {

constexpr int kRowThreads = 256;
// Row steps of a reading CTA (its loads in flight) where there are rows enough for every SM: 30200 rows of 4
// heads of 128 are read in 19.2 us with 1, 15.4 with 2 and 15.2 with 4. Appending them takes 23.4 us with 1
// and 23.9 with 2. In its capture warps wait first at the barrier behind the look-up of the CTA's places (5.0 warps an issue,
// 1.7 for math pipes; ALU 52 %, DRAM 38 %).
constexpr int kReadSteps = 4;

// Cache row (counting rows of all sequences and heads, for head 0) of packed row i; -1 (reported) when the
// batch tables do not place it.
__device__ __forceinline__ int64_t locate_row(const Kv4RowsArgs& a, int64_t i)
{
    int b = (int)i; // without tables T = B
    int64_t off = 0;
    if (a.cu) {
        int lo = 0, hi = a.B - 1; // the last b with cu[b] <= i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu[mid] <= i) lo = mid; else hi = mid - 1;
        }
        b = lo;
        off = i - a.cu[b];
        if (off < 0 || i >= a.cu[b + 1]) {
            if (a.err) report_error(a.err, MSA_ERR_DEVICE_CHECK, 300);
            return -1;
        }
    }
    const int start = a.starts[b];
    if (start < 0 || start + off >= a.L_max) {
        if (a.err) report_error(a.err, MSA_ERR_DEVICE_CHECK, 301);
        return -1;
    }
    return (int64_t)b * a.H_kv * a.L_max + start + off;
}

// The CTA's rows [i0, i0 + n): their cache rows in `place` (-1: none), by the first threads.
__device__ __forceinline__ void locate_rows(const Kv4RowsArgs& a, int64_t i0, int n, int64_t* place)
{
    if (threadIdx.x < n) place[threadIdx.x] = i0 + threadIdx.x < a.T ? locate_row(a, i0 + threadIdx.x) : -1;
    __syncthreads();
}

// Correctly rounded -x / d, two at a time, from nr = -1 / d correctly rounded (Markstein's correction of the
// product by its exact residual), for d > 0 and where nothing over- or underflows: see quantise16. The
// residual is taken as q d + x, so that a zero keeps its sign.
__device__ __forceinline__ uint64_t minus_quotient2(uint64_t x, uint64_t d, uint64_t nr)
{
    const uint64_t q = f2_mul(x, nr);
    return f2_fma(f2_fma(q, d, x), nr, q);
}

// The 16 elements of w as codes c and their scale's byte. rt = 1 / t, or 0 where t is outside [2^-20,
// 2^20]: then, and where an element is 2^100 or more, all quotients are plain divisions. Elements small
// enough for the correction's residual to underflow (below 2^-100) are far below the smallest scale's
// smallest code, and end as 0 either way.
__device__ __forceinline__ uint32_t quantise16(const uint32_t (&w)[8], float t, float rt, uint32_t (&c)[2])
{
    uint32_t m = 0u; // largest |x|: bf16 magnitudes order like integers
#pragma unroll
    for (int e = 0; e < 8; ++e) m = __vmaxu2(m, w[e] & 0x7FFF7FFFu);
    m = max(m >> 16, m & 0xFFFFu);
    float amax = __uint_as_float(m << 16);
    c[0] = c[1] = 0u;
    const bool plain = rt == 0.f || !(amax < 0x1p100f);
    if (t != 1.f) amax = __fdiv_rn(amax, t); // rounding keeps the order
    const uint32_t s8 = e4m3x2_pack(__fdiv_rn(amax, 6.f), 0.f) & 0xFFu;
    if (s8 == 0) return 0u;
    const float s = e4m3x2_unpack(s8).x;
    float q[16];
    if (plain) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            q[2 * e] = __fdiv_rn(__fdiv_rn(bf16_lo(w[e]), t), s);
            q[2 * e + 1] = __fdiv_rn(__fdiv_rn(bf16_hi(w[e]), t), s);
        }
    } else {
        const float rs = __frcp_rn(s);
        const uint64_t ss = f2_pack(s, s), nrs = f2_pack(-rs, -rs), tt = f2_pack(t, t), nrt = f2_pack(-rt, -rt);
        const uint32_t flip = t != 1.f ? 0u : 0x80008000u; // either way y below is -x / t
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t v = w[e] ^ flip;
            uint64_t y = f2_pack(bf16_lo(v), bf16_hi(v));
            if (t != 1.f) y = minus_quotient2(y, tt, nrt);
            y = minus_quotient2(y, ss, nrs);
            q[2 * e] = f2_lo(y);
            q[2 * e + 1] = f2_hi(y);
        }
    }
    c[0] = e2m1x8_pack(q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]);
    c[1] = e2m1x8_pack(q[8], q[9], q[10], q[11], q[12], q[13], q[14], q[15]);
    return s8;
}

// A thread takes 16 elements of K and of V of one row.
template <int DH>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(Kv4RowsArgs a)
{
    constexpr int NG = DH / 16, ROWS = kRowThreads / NG;
    __shared__ int64_t place[ROWS];
    const int g = threadIdx.x % NG, i = threadIdx.x / NG, r = blockIdx.x % a.H_kv;
    const int64_t i0 = (int64_t)(blockIdx.x / a.H_kv) * ROWS;
    uint32_t w[2][8];
    if (i0 + i < a.T) { // in flight while the places are looked up
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint4* src = reinterpret_cast<const uint4*>(a.x[which] + (i0 + i) * a.x_stride[which] + (int64_t)r * DH + g * 16);
            const uint4 v0 = src[0], v1 = src[1];
            uint32_t* x = w[which];
            x[0] = v0.x, x[1] = v0.y, x[2] = v0.z, x[3] = v0.w, x[4] = v1.x, x[5] = v1.y, x[6] = v1.z, x[7] = v1.w;
        }
    }
    locate_rows(a, i0, ROWS, place);
    if (place[i] < 0) return;
    const int64_t row = place[i] + r * a.L_max;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        uint32_t c[2];
        const uint32_t s8 = quantise16(w[which], a.t[which], a.rt[which], c);
        *reinterpret_cast<uint2*>(a.codes[which] + row * (DH / 2) + g * 8) = make_uint2(c[0], c[1]);
        a.scales[which][row * NG + g] = (uint8_t)s8;
    }
}

// A thread takes 8 elements of K and of V of one row per step: 16-byte stores, whole rows to a warp's.
template <int DH, int STEPS>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(Kv4RowsArgs a)
{
    constexpr int NU = DH / 8, ROWS = kRowThreads / NU, N = ROWS * STEPS;
    __shared__ int64_t place[N];
    const int e8 = threadIdx.x % NU, i = threadIdx.x / NU, r = blockIdx.x % a.H_kv; // the heads of a row run together
    const int64_t i0 = (int64_t)(blockIdx.x / a.H_kv) * N;
    locate_rows(a, i0, N, place);
    uint32_t c[STEPS][2], s8[STEPS][2];
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
        const int64_t row = place[u * ROWS + i] + r * a.L_max;
        if (place[u * ROWS + i] < 0) continue;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            c[u][which] = *reinterpret_cast<const uint32_t*>(a.codes[which] + row * (DH / 2) + e8 * 4);
            s8[u][which] = a.scales[which][row * (DH / 16) + e8 / 2];
        }
    }
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
        if (place[u * ROWS + i] < 0) continue;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const float s = e4m3x2_unpack(s8[u][which]).x, t = a.t[which];
            uint32_t h[4], o[4];
            e2m1x8_to_f16x2(c[u][which], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpack_f16x2(h[e]);
                o[e] = pack_bf16x2(f.x * s * t, f.y * s * t); // code * s is exact
            }
            *reinterpret_cast<uint4*>(a.y[which] + ((i0 + u * ROWS + i) * a.H_kv + r) * (int64_t)DH + e8 * 8) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// CTAs for all rows of all heads, `rows` to a CTA.
int64_t row_ctas(const Kv4RowsArgs& a, int rows) { return (a.T + rows - 1) / rows * a.H_kv; }

template <int DH>
void append(const Kv4RowsArgs& a, cudaStream_t s)
{
    kv4_append_kernel<DH><<<(unsigned)row_ctas(a, kRowThreads / (DH / 16)), kRowThreads, 0, s>>>(a);
}

// kReadSteps row steps to a CTA once that leaves two CTAs for every SM, else one.
template <int DH>
void read(const Kv4RowsArgs& a, cudaStream_t s)
{
    constexpr int ROWS = kRowThreads / (DH / 8);
    if (row_ctas(a, ROWS * kReadSteps) >= 2 * kKv4Ctas)
        kv4_read_kernel<DH, kReadSteps><<<(unsigned)row_ctas(a, ROWS * kReadSteps), kRowThreads, 0, s>>>(a);
    else
        kv4_read_kernel<DH, 1><<<(unsigned)row_ctas(a, ROWS), kRowThreads, 0, s>>>(a);
}

} // namespace

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t s)
{
    a.d_h == 128 ? append<128>(a, s) : append<64>(a, s);
    note_launch(1);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsArgs& a, cudaStream_t s)
{
    a.d_h == 128 ? read<128>(a, s) : read<64>(a, s);
    note_launch(1);
    return cudaGetLastError();
}

} // namespace msa
