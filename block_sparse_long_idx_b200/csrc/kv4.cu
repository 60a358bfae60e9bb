// kv4.cu -- rows into and out of the 4-bit key/value cache (format: kv4.cuh).
//
// append: for every 16 elements x of a new row
//   y = fl32(x / t), a = max |y|, s = E4M3(min(fl32(a / 6), 448)), code = E2M1(fl32(y / s))
// with all roundings to nearest even and codes saturating at 6; s = 0 gives zero codes. read: the
// values code * s * t rounded to bf16. One thread per 16 elements, CTAs of one head's consecutive
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

template <int DH>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(Kv4RowsArgs a)
{
    constexpr int NG = DH / 16, ROWS = kRowThreads / NG;
    const int g = threadIdx.x % NG, which = blockIdx.z, r = blockIdx.y;
    const int64_t i = (int64_t)blockIdx.x * ROWS + threadIdx.x / NG;
    int b;
    int64_t pos;
    if (i >= a.T || !locate_row(a, i, b, pos)) return;
    const uint4* src = reinterpret_cast<const uint4*>(a.x[which] + i * a.x_stride[which] + (int64_t)r * DH + g * 16);
    const uint4 v0 = src[0], v1 = src[1];
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    const float t = a.t[which];
    float y[16], amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        y[2 * e] = __fdiv_rn(bf16_lo(w[e]), t);
        y[2 * e + 1] = __fdiv_rn(bf16_hi(w[e]), t);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(y[e]));
    const uint32_t s8 = e4m3x2_pack(__fdiv_rn(amax, 6.f), 0.f) & 0xFFu;
    uint32_t c[2] = {0u, 0u};
    if (s8 != 0) {
        const float s = e4m3x2_unpack(s8).x;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c[e >> 2] |= e2m1x2_pack(__fdiv_rn(y[2 * e], s), __fdiv_rn(y[2 * e + 1], s)) << (8 * (e & 3));
    }
    const int64_t row = ((int64_t)b * a.H_kv + r) * a.L_max + pos;
    *reinterpret_cast<uint2*>(a.codes[which] + row * (DH / 2) + g * 8) = make_uint2(c[0], c[1]);
    a.scales[which][row * NG + g] = (uint8_t)s8;
}

template <int DH>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(Kv4RowsArgs a)
{
    constexpr int NG = DH / 16, ROWS = kRowThreads / NG;
    const int g = threadIdx.x % NG, which = blockIdx.z, r = blockIdx.y;
    const int64_t i = (int64_t)blockIdx.x * ROWS + threadIdx.x / NG;
    int b;
    int64_t pos;
    if (i >= a.T || !locate_row(a, i, b, pos)) return;
    const int64_t row = ((int64_t)b * a.H_kv + r) * a.L_max + pos;
    const uint2 c = *reinterpret_cast<const uint2*>(a.codes[which] + row * (DH / 2) + g * 8);
    const float s = e4m3x2_unpack(a.scales[which][row * NG + g]).x, t = a.t[which];
    uint32_t h[2][4], o[8];
    e2m1x8_to_f16x2(c.x, h[0]);
    e2m1x8_to_f16x2(c.y, h[1]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 f = unpack_f16x2(h[e >> 2][e & 3]);
        o[e] = pack_bf16x2(f.x * s * t, f.y * s * t); // code * s is exact
    }
    uint4* dst = reinterpret_cast<uint4*>(a.y[which] + (i * a.H_kv + r) * (int64_t)DH + g * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

dim3 rows_grid(const Kv4RowsArgs& a)
{
    const int rows = kRowThreads / (a.d_h / 16);
    return dim3((unsigned)((a.T + rows - 1) / rows), a.H_kv, 2);
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
