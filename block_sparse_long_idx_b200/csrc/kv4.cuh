// kv4.cuh -- the 4-bit key/value cache: device helpers of its format and the launchers of kv4.cu,
// kv4_decode.cu and kv4_evict.cu.
//
// Format (per K and V): E2M1 codes (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; bit 3 the sign), element
// 2i of a row in the low nibble of byte i and 2i + 1 in the high one; one E4M3 scale per 16 elements;
// one fp32 scale t per tensor. value = code * scale * t. code * scale has at most 6 significant bits
// and lies in [2^-10, 2688], so it is exact in fp16, the type the tensor cores read it in.
// Head-major: codes [B][H_kv][L_max][d_h / 2], scales [B][H_kv][L_max][d_h / 16], so that the tokens
// of a (sequence, head) are one contiguous run a bulk copy can stream.
#pragma once
#include <atomic>

#include "common.cuh"
#include "sm100.cuh"

namespace msa {

// Eight E2M1 codes (byte i = codes 2i, 2i + 1) -> four fp16 pairs, h[i] = (code 2i, code 2i + 1).
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Eight fp32 values -> eight E2M1 codes, the first in the lowest nibble: nearest, ties to the even code,
// saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8_pack(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3), "f"(x4), "f"(x5), "f"(x6), "f"(x7));
    return r;
}

// Two E4M3 bytes (bits 0-7 and 8-15 of v) -> an fp16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v)
{
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(v));
    return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float2 unpack_f16x2(uint32_t h)
{
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return make_float2(lo, hi);
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// Raises a kernel's dynamic shared memory limit, once per device (the call costs as much as a launch).
class SmemOptIn {
    std::atomic<uint64_t> done_{0}; // one bit per device; devices from 64 on are set every time

public:
    template <class F>
    cudaError_t set(F* kernel, int bytes)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
        if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// Rows of a packed batch: row i of T belongs to the sequence b with cu[b] <= i < cu[b + 1] (cu =
// nullptr: one row per sequence) and to position starts[b] + i - cu[b] of its cache.
struct Kv4RowsArgs {
    uint8_t* codes[2]; // K, V
    uint8_t* scales[2];
    float t[2];
    float rt[2];       // 1 / t, or 0 (see quantise16)
    const uint16_t* x[2]; // append: [T][H_kv][d_h] bf16, rows x_stride[i] elements apart
    int64_t x_stride[2];
    uint16_t* y[2]; // read: [T][H_kv][d_h] bf16
    const int32_t* starts;
    const int32_t* cu;
    int64_t T, L_max;
    int B, H_kv, d_h;
    int* err; // nullptr: nothing is reported
};
cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4RowsArgs& a, cudaStream_t s);

// CTAs of the decode grid (one per SM of a B200) and its scratch: every CTA walks a contiguous slice
// of the work, so at most its first and its last (sequence, head) are shared with other CTAs.
constexpr int kKv4Ctas = 148;
constexpr int kKv4PartFloats = 16 * 128 + 32; // partial output, maximum and sum of 16 rows

struct Kv4DecodeArgs {
    const uint16_t* q; // [B][H_q][d_h]
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    float k_scale, v_scale;
    const int32_t* lens;
    const int32_t* block_idx; // [B][H_kv][k], or nullptr: every visible key
    int B, H_q, H_kv, d_h, k;
    int64_t L_max;
    int min_len;          // smallest valid length: 0, or 1 for the block-sparse decode
    bool after_topk;      // the blocks are those of the Top-k kernel just launched, which has cleared the error word
    uint16_t* out;        // [B][H_q][d_h]
    float* lse;           // [B][H_q], or nullptr
    float* parts;         // [2 * kKv4Ctas][kKv4PartFloats]
    const float* w_in;    // [B][H_kv][L_max], or nullptr
    float* w_out;         // [B][H_kv][L_max], or nullptr: no weights (lse is set when it is not)
    float decay;
    int* err;
};
cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t s);

struct Kv4EvictArgs {
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    uint8_t *k_codes_to, *k_scales_to, *v_codes_to, *v_scales_to;
    const uint16_t* k_idx; // [B][L_max][H_kv][d_idx], or nullptr
    uint16_t* k_idx_to;    // [B][L_to][H_kv][d_idx]
    const float* w;        // [B][H_kv][L_max]
    float* w_to;           // [B][H_kv][L_to], or nullptr
    const int32_t* lens;
    int32_t* lens_to;
    int32_t* kept; // [B][H_kv][keep]
    int B, H_kv, d_h, d_idx, keep, recent, first;
    int64_t L_max, L_to;
    int* err; // nullptr: nothing is reported
};
cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t s);

} // namespace msa
