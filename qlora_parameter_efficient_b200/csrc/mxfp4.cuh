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

// Eight consecutive elements as loaded, their values in fp32, and the largest |x| among them as fp32
// bits (an integer maximum: NaN and infinity bits order above every finite value).
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ uint32_t values(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
        return m;
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ uint32_t values(float (&x)[8]) const {
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
};
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    Raw8<__nv_bfloat16> r;
    r.load(p);
    r.values(x);
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

// MXFP4 of one whole block of 32 in one thread.
__device__ __forceinline__ void mxfp4_block32(const Raw8<__nv_bfloat16> (&raw)[4], uint32_t& e, uint32_t (&q)[4]) {
    float x[4][8];
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) m = max(m, raw[c].values(x[c]));
    const uint32_t ef = m >> 23;
    e = ef == 255u ? 255u : (ef > 2u ? ef - 2u : 0u);
    const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = __fmul_rn(x[c][i], inv);
        q[c] = e == 255u ? 0u : e2m1x8(x[c]);
    }
}

// One 128 x 128 scale tile of a matrix: 256 threads (any more of the block stand by), sixteen lanes per
// row (8 elements each, four lanes per block), 8 passes of 16 rows whose loads are all issued first
// (4 passes at a time for fp32).  The tile's scales are gathered in shared memory and written once, 512
// contiguous bytes.
template <typename T>
__device__ __forceinline__ void mxfp4_quantize_tile(const T* __restrict__ X, int64_t rows, int64_t cols,
                                                    int64_t rt, int64_t kt, uint8_t* __restrict__ codes,
                                                    uint8_t* __restrict__ scales, uint8_t* s_sc) {
    constexpr int kBatch = sizeof(T) == 4 ? 4 : 8;
    const int seg = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const int64_t col = kt * 128 + seg * 8;
    const int64_t left = col < cols ? rows - rt * 128 : 0;       // rows of this tile that exist
    const bool mine = threadIdx.x < 256;
    const T* src = X + (rt * 128 + r0) * cols + col;
    uint8_t* dst = codes + ((rt * 128 + r0) * cols + col) / 2;
#pragma unroll
    for (int p0 = 0; p0 < 8; p0 += kBatch) {
        Raw8<T> raw[kBatch];
#pragma unroll
        for (int p = 0; p < kBatch; ++p) {
            if (mine && (p0 + p) * 16 + r0 < left) raw[p].load(src + (p0 + p) * 16 * cols);
            else raw[p].zero();
        }
#pragma unroll
        for (int p = 0; p < kBatch; ++p) {
            const int lr = (p0 + p) * 16 + r0;
            float x[8];
            const uint32_t ef = quad_max(raw[p].values(x)) >> 23;     // biased exponent of max|x|
            const uint32_t e = ef == 255u ? 255u : (ef > 2u ? ef - 2u : 0u);
            const float inv = __uint_as_float((254u - e) << 23);      // 2^(127 - e)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], inv);
            const uint32_t q = e == 255u ? 0u : e2m1x8(x);
            if (mine && lr < left) *reinterpret_cast<uint32_t*>(dst + (p0 + p) * 8 * cols) = q;
            if (mine && (seg & 3) == 0) s_sc[(lr & 31) * 16 + (lr >> 5) * 4 + (seg >> 2)] = lr < left ? static_cast<uint8_t>(e) : 0;
        }
    }
    __syncthreads();
    if (threadIdx.x < kMxTileBytes / 16)
        reinterpret_cast<uint4*>(scales + (rt * mx_col_tiles(cols) + kt) * kMxTileBytes)[threadIdx.x] =
            reinterpret_cast<const uint4*>(s_sc)[threadIdx.x];
}

// grid: one CTA per scale tile, column tiles fastest.  Bound by HBM: 4096 x 11008 fp32 in 31.8 us (204 MB,
// 6.4 TB/s); 203 x 448 bf16 in 4.3 us, launch and one round of loads.
template <typename T>
__global__ void __launch_bounds__(256) k_mxfp4_quantize(const T* __restrict__ X, int64_t rows, int64_t cols,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    __shared__ __align__(16) uint8_t s_sc[kMxTileBytes];
    griddep_enter();
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

// Eight packed codes times the block's scale.  The products are formed in fp32, so that the one rounding
// to bf16 is that of the exact value.
__device__ __forceinline__ void e2m1_scale8(uint32_t q, float s, float (&f)[8]) {
    const uint4 v = e2m1_decode8_bf16(q);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __fmul_rn(__uint_as_float(w[k] << 16), s);
        f[2 * k + 1] = __fmul_rn(__uint_as_float(w[k] & 0xFFFF0000u), s);
    }
}
__device__ __forceinline__ uint4 e2m1_scale8_bf16(uint32_t q, float s) {
    float f[8];
    e2m1_scale8(q, s, f);
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// One 128 x 128 tile of a matrix, as mxfp4_quantize_tile lays it out: the tile's 512 bytes of scales in
// shared memory, sixteen lanes per row, eight rows' codes (4 bytes a lane) in flight, 16 (bf16) or 32 (fp32)
// bytes out.
template <typename T>
__device__ __forceinline__ void mxfp4_dequantize_tile(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, int64_t rows, int64_t cols,
                                                      int64_t rt, int64_t kt, T* __restrict__ out, uint8_t* s_sc) {
    const int seg = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const int64_t col = kt * 128 + seg * 8;
    const int64_t left = col < cols ? rows - rt * 128 : 0;
    const int64_t at = (rt * 128 + r0) * cols + col;
    uint32_t q[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        q[p] = 0;
        if (p * 16 + r0 < left) q[p] = __ldg(reinterpret_cast<const uint32_t*>(codes + (at + p * 16 * cols) / 2));
    }
    if (threadIdx.x < kMxTileBytes / 16)
        reinterpret_cast<uint4*>(s_sc)[threadIdx.x] =
            __ldg(reinterpret_cast<const uint4*>(scales + (rt * mx_col_tiles(cols) + kt) * kMxTileBytes) + threadIdx.x);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int lr = p * 16 + r0;
        if (lr >= left) continue;
        const float s = e8m0_value(s_sc[(lr & 31) * 16 + (lr >> 5) * 4 + (seg >> 2)]);
        T* o = out + at + p * 16 * cols;
        if constexpr (sizeof(T) == 4) {
            float f[8];
            e2m1_scale8(q[p], s, f);
            reinterpret_cast<float4*>(o)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4*>(o)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4*>(o) = e2m1_scale8_bf16(q[p], s);
        }
    }
}

// grid: one CTA per scale tile, column tiles fastest.  Bound by HBM: 4096 x 11008 to bf16 in 21.7 us (114 MB,
// 5.3 TB/s, four fifths of it writes).
template <typename T>
__global__ void __launch_bounds__(256) k_mxfp4_dequant(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, int64_t rows,
                                                       int64_t cols, T* __restrict__ out) {
    __shared__ __align__(16) uint8_t s_sc[kMxTileBytes];
    griddep_enter();
    const int64_t kts = mx_col_tiles(cols);
    mxfp4_dequantize_tile(codes, scales, rows, cols, blockIdx.x / kts, blockIdx.x % kts, out, s_sc);
}

}  // namespace qlora
