// mxfp4.cuh -- the MXFP4 storage format: quantizer and stand-alone decoder.
//
// OCP Microscaling Formats v1.0: blocks of 32 consecutive elements of a row share one E8M0 scale
// 2^(e - 127), elements are E2M1 (sign, 2 exponent bits with bias 1, 1 mantissa bit: magnitudes
// 0, 0.5, 1, 1.5, 2, 3, 4, 6).  Conversion of a block, as the specification gives it:
//   e    = max(0, floor(log2 max|x|) - 2 + 127)           (2: the exponent of E2M1's largest value)
//   code = E2M1(x 2^(127 - e))                            round to nearest even, saturating at 6
// A power-of-two scale makes the product x 2^(127 - e) and every decoded value exact in fp32, so the
// format is defined bit for bit.  A block that holds a NaN or an infinity gets e = 255 (E8M0's NaN)
// and codes 0: it decodes to NaN, and so does every product that reads it.
//
// Layout: codes [rows, cols / 2], element 2j in the low nibble of byte j.  Scales in 512-byte tiles
// of 128 rows x 4 blocks, tile (row / 128, block / 4) at index (row / 128) ceil(blocks / 4) + block / 4:
//   byte (row % 32) 16 + (row / 32 % 4) 4 + block % 4
// -- 32 lines of 16 bytes, the shape tcgen05.cp.32x128b copies into tensor memory, so the
// block-scaled MMAs read a stored scale tile without any rearrangement.  Bytes of a tile outside
// the matrix are 0.
#pragma once

#include "common.cuh"

namespace qlora {

constexpr int kMxBlock = 32;          // elements per scale
constexpr int kMxTileBytes = 512;     // scales of 128 rows x 4 blocks

__host__ __device__ __forceinline__ int64_t mx_col_tiles(int64_t cols) { return (cols + 127) / 128; }

__device__ __forceinline__ int64_t mx_scale_offset(int64_t row, int64_t blk, int64_t col_tiles) {
    return ((row >> 7) * col_tiles + (blk >> 2)) * kMxTileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
           (blk & 3);
}

// 2^(e - 127) as fp32: exact for every E8M0 byte (e = 0 is subnormal), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t e) {
    return __uint_as_float(e == 255u ? 0x7FFFFFFFu : (e == 0u ? 0x00400000u : e << 23));
}

// Eight elements as fp32, and the largest |x| among them as fp32 bits (an integer maximum: NaN and
// infinity bits order above every finite value).
__device__ __forceinline__ uint32_t load8(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return m;
}
__device__ __forceinline__ uint32_t load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        m = max(m, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
    }
    return m;
}

// Maximum over the four lanes that share a block of 32.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Eight fp32 values to packed E2M1 codes, round to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
    uint32_t q;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(q)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return q;
}

// One 128 x 128 scale tile of a matrix: 256 threads, sixteen lanes per row (8 elements each, four
// lanes per block), 8 passes of 16 rows.  The tile's scales are gathered in shared memory
// and written once, 512 contiguous bytes.
template <typename T>
__device__ __forceinline__ void mxfp4_quantize_tile(const T* __restrict__ X, int64_t rows, int64_t cols,
                                                    int64_t rt, int64_t kt, uint8_t* __restrict__ codes,
                                                    uint8_t* __restrict__ scales, uint8_t* s_sc) {
    const int seg = threadIdx.x & 15;
    const int64_t col = kt * 128 + seg * 8;
    float x[8][8];
    uint32_t m[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t row = rt * 128 + p * 16 + (threadIdx.x >> 4);
        m[p] = 0;
        if (row < rows && col < cols) m[p] = load8(X + row * cols + col, x[p]);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) x[p][i] = 0.f;
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int lr = p * 16 + (threadIdx.x >> 4);
        const int64_t row = rt * 128 + lr;
        const uint32_t ef = quad_max(m[p]) >> 23;                // biased exponent of max|x|
        const uint32_t e = ef == 255u ? 255u : (ef > 2u ? ef - 2u : 0u);
        // 2^(127 - e); 0 for a NaN block, whose codes are 0
        const float inv = __uint_as_float(e == 255u ? 0u : (254u - e) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[p][i] = __fmul_rn(x[p][i], inv);
        const uint32_t q = e == 255u ? 0u : e2m1x8(x[p]);
        if (row < rows && col < cols) *reinterpret_cast<uint32_t*>(codes + (row * cols + col) / 2) = q;
        if ((seg & 3) == 0)
            s_sc[(lr & 31) * 16 + (lr >> 5) * 4 + (seg >> 2)] =
                (row < rows && col < cols) ? static_cast<uint8_t>(e) : 0;
    }
    __syncthreads();
    if (threadIdx.x < kMxTileBytes / 16)
        reinterpret_cast<uint4*>(scales + (rt * mx_col_tiles(cols) + kt) * kMxTileBytes)[threadIdx.x] =
            reinterpret_cast<const uint4*>(s_sc)[threadIdx.x];
}

// grid: one CTA per scale tile, column tiles fastest.
// zero[0, n_zero): ticket counters of a later kernel of the call, cleared on the way.
template <typename T>
__global__ void __launch_bounds__(256) k_mxfp4_quantize(const T* __restrict__ X, int64_t rows, int64_t cols,
                                                        uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales, int* __restrict__ zero,
                                                        int n_zero) {
    __shared__ __align__(16) uint8_t s_sc[kMxTileBytes];
    griddep_enter();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < n_zero; i += 256) zero[i] = 0;
    const int64_t kts = mx_col_tiles(cols);
    mxfp4_quantize_tile(X, rows, cols, blockIdx.x / kts, blockIdx.x % kts, codes, scales, s_sc);
}

// Eight packed codes as four bf16x2 words (element order), unscaled: every E2M1 magnitude is a bf16
// value whose high byte is one of {00, 3F, 40} and low byte one of {00, 40, 80, C0}, so two
// byte-permute tables indexed by the magnitude hold all eight.
__device__ __forceinline__ uint4 e2m1_decode8_bf16(uint32_t q) {
    // magnitudes 0..7 = 0, 0.5, 1, 1.5, 2, 3, 4, 6 = 0000 3F00 3F80 3FC0 4000 4040 4080 40C0
    constexpr uint32_t hi0 = 0x3F3F3F00u, hi1 = 0x40404040u;
    constexpr uint32_t lo0 = 0xC0800000u, lo1 = 0xC0804000u;
    const uint32_t m = q & 0x77777777u;
    const uint32_t lo_a = prmt(lo0, lo1, m), lo_b = prmt(lo0, lo1, m >> 16);
    uint32_t hi_a = prmt(hi0, hi1, m), hi_b = prmt(hi0, hi1, m >> 16);
    // sign bytes: element 2j's bit 3 is the msb of byte j of (q << 4), element 2j+1's that of byte j of q
    const uint32_t q4 = q << 4;
    hi_a |= prmt(q4, q, 0xD9C8) & 0x80808080u;
    hi_b |= prmt(q4, q, 0xFBEA) & 0x80808080u;
    return make_uint4(prmt(lo_a, hi_a, 0x5140), prmt(lo_a, hi_a, 0x7362), prmt(lo_b, hi_b, 0x5140),
                      prmt(lo_b, hi_b, 0x7362));
}

// One thread per 8 elements: 4 code bytes in, 16 (bf16) or 32 (fp32) bytes out.
template <typename T>
__global__ void __launch_bounds__(256) k_mxfp4_dequant(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, int64_t rows,
                                                       int64_t cols, T* __restrict__ out, int* __restrict__ zero,
                                                       int n_zero) {
    griddep_enter();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < n_zero; i += 256) zero[i] = 0;
    const int64_t n8 = rows * cols / 8, per_row = cols / 8, kts = mx_col_tiles(cols);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n8;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = i / per_row, blk = (i - row * per_row) >> 2;
        const uint32_t e = __ldg(scales + mx_scale_offset(row, blk, kts));
        const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
        const uint4 v = e2m1_decode8_bf16(q);
        // in fp32, so that the one rounding to bf16 is that of the exact value
        const float s = e8m0_value(e);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = __fmul_rn(__uint_as_float(w[k] << 16), s);
            f[2 * k + 1] = __fmul_rn(__uint_as_float(w[k] & 0xFFFF0000u), s);
        }
        if constexpr (sizeof(T) == 4) {
            float4* o = reinterpret_cast<float4*>(out) + 2 * i;
            o[0] = make_float4(f[0], f[1], f[2], f[3]);
            o[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            reinterpret_cast<uint4*>(out)[i] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        }
    }
}

}  // namespace qlora
