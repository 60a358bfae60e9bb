// kv4.cu -- rows into and out of the 4-bit key/value cache (format: kv4.cuh).
//
// append: for every 16 elements x of a new row
//   y = fl32(x / t), a = max |y|, s = E4M3(min(fl32(a / 6), 448)), code = E2M1(fl32(y / s))
// with all roundings to nearest even and codes saturating at 6; s = 0 gives zero codes. read: the
// values code * s * t rounded to bf16. One thread per 16 elements of K and of V, CTAs of one head's consecutive
// rows, so that the head-major cache side is written (read) in whole contiguous runs and the
// token-major side in whole rows of d_h elements.
#include "kv4.cuh"

namespace msa {

namespace {

constexpr int kRowThreads = 256;

// Sequence and cache position of packed row i; false (reported) when the batch tables do not place it.
__device__ __forceinline__ bool locate_row(const Kv4RowsArgs& a, int64_t i, int& b, int64_t& pos)
{
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
            report_error(a.err, MSA_ERR_DEVICE_CHECK, 300);
            return false;
        }
    } else {
        b = (int)i; // T = B
    }
    pos = (int64_t)a.starts[b] + off;
    if (a.starts[b] < 0 || pos >= a.L_max) {
        report_error(a.err, MSA_ERR_DEVICE_CHECK, 301);
        return false;
    }
    return true;
}

// Correctly rounded x / d from r = 1 / d correctly rounded (Markstein's correction of x * r by its exact
// residual), for d > 0 and where nothing over- or underflows: see quantise16.
__device__ __forceinline__ float quotient(float x, float d, float r)
{
    const float q = x * r;
    return copysignf(fmaf(fmaf(-q, d, x), r, q), x); // the correction loses the sign of a zero
}

// The 16 elements of w as codes c and their scale's byte. rt = 1 / t, or 0 where t is outside [2^-20,
// 2^20]: then, and where an element is 2^100 or more, all quotients are plain divisions. Elements small
// enough for the correction's residual to underflow (below 2^-100) are far below the smallest scale's
// smallest code, and end as 0 either way.
__device__ __forceinline__ uint32_t quantise16(const uint32_t (&w)[8], float t, float rt, uint32_t (&c)[2])
{
    float y[16], amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        y[2 * e] = bf16_lo(w[e]);
        y[2 * e + 1] = bf16_hi(w[e]);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(y[e]));
    const bool plain = rt == 0.f || !(amax < 0x1p100f);
    c[0] = c[1] = 0u;
    if (plain) {
        amax = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            y[e] = __fdiv_rn(y[e], t);
            amax = fmaxf(amax, fabsf(y[e]));
        }
    } else if (t != 1.f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = quotient(y[e], t, rt);
        amax = quotient(amax, t, rt); // rounding keeps the order
    }
    const uint32_t s8 = e4m3x2_pack(__fdiv_rn(amax, 6.f), 0.f) & 0xFFu;
    if (s8 == 0) return 0u;
    const float s = e4m3x2_unpack(s8).x;
    if (plain) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c[e >> 2] |= e2m1x2_pack(__fdiv_rn(y[2 * e], s), __fdiv_rn(y[2 * e + 1], s)) << (8 * (e & 3));
    } else {
        const float rs = __frcp_rn(s);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c[e >> 2] |= e2m1x2_pack(quotient(y[2 * e], s, rs), quotient(y[2 * e + 1], s, rs)) << (8 * (e & 3));
    }
    return s8;
}

template <int DH>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(Kv4RowsArgs a)
{
    constexpr int NG = DH / 16, ROWS = kRowThreads / NG;
    const int g = threadIdx.x % NG, r = blockIdx.y;
    const int64_t i = (int64_t)blockIdx.x * ROWS + threadIdx.x / NG;
    if (i >= a.T) return;
    uint32_t w[2][8];
#pragma unroll
    for (int which = 0; which < 2; ++which) { // the loads of both tensors, and of the tables, in flight together
        const uint4* src = reinterpret_cast<const uint4*>(a.x[which] + i * a.x_stride[which] + (int64_t)r * DH + g * 16);
        const uint4 v0 = src[0], v1 = src[1];
        w[which][0] = v0.x, w[which][1] = v0.y, w[which][2] = v0.z, w[which][3] = v0.w;
        w[which][4] = v1.x, w[which][5] = v1.y, w[which][6] = v1.z, w[which][7] = v1.w;
    }
    int b;
    int64_t pos;
    if (!locate_row(a, i, b, pos)) return;
    const int64_t row = ((int64_t)b * a.H_kv + r) * a.L_max + pos;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        uint32_t c[2];
        const uint32_t s8 = quantise16(w[which], a.t[which], a.rt[which], c);
        *reinterpret_cast<uint2*>(a.codes[which] + row * (DH / 2) + g * 8) = make_uint2(c[0], c[1]);
        a.scales[which][row * NG + g] = (uint8_t)s8;
    }
}

template <int DH>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(Kv4RowsArgs a)
{
    constexpr int NG = DH / 16, ROWS = kRowThreads / NG;
    const int g = threadIdx.x % NG, r = blockIdx.y;
    const int64_t i = (int64_t)blockIdx.x * ROWS + threadIdx.x / NG;
    int b;
    int64_t pos;
    if (i >= a.T || !locate_row(a, i, b, pos)) return;
    const int64_t row = ((int64_t)b * a.H_kv + r) * a.L_max + pos;
    uint2 c[2];
    uint32_t s8[2];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        c[which] = *reinterpret_cast<const uint2*>(a.codes[which] + row * (DH / 2) + g * 8);
        s8[which] = a.scales[which][row * NG + g];
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float s = e4m3x2_unpack(s8[which]).x, t = a.t[which];
        uint32_t h[2][4], o[8];
        e2m1x8_to_f16x2(c[which].x, h[0]);
        e2m1x8_to_f16x2(c[which].y, h[1]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 f = unpack_f16x2(h[e >> 2][e & 3]);
            o[e] = pack_bf16x2(f.x * s * t, f.y * s * t); // code * s is exact
        }
        uint4* dst = reinterpret_cast<uint4*>(a.y[which] + (i * a.H_kv + r) * (int64_t)DH + g * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

dim3 rows_grid(const Kv4RowsArgs& a)
{
    const int rows = kRowThreads / (a.d_h / 16);
    return dim3((unsigned)((a.T + rows - 1) / rows), a.H_kv);
}

} // namespace

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t s)
{
    if (a.d_h == 128)
        kv4_append_kernel<128><<<rows_grid(a), kRowThreads, 0, s>>>(a);
    else
        kv4_append_kernel<64><<<rows_grid(a), kRowThreads, 0, s>>>(a);
    note_launch(1);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsArgs& a, cudaStream_t s)
{
    if (a.d_h == 128)
        kv4_read_kernel<128><<<rows_grid(a), kRowThreads, 0, s>>>(a);
    else
        kv4_read_kernel<64><<<rows_grid(a), kRowThreads, 0, s>>>(a);
    note_launch(1);
    return cudaGetLastError();
}

} // namespace msa
