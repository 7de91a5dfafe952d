// act8.cuh -- 8-bit activation checkpoints: quantizer, stand-alone decoder, and the adapter-gradient
// product that reads them.
//
// "LoRA and QLoRA Fine-Tuning Under the Hood", section "1.3 Activation Memory Savings via
// FlashAttention-2 & Activation Checkpointing": the activation a layer keeps for its backward is what
// fills memory in training.  Here it is kept as OCP MXINT8: blocks of 32 consecutive elements of a
// row share an E8M0 scale, elements are 8-bit integers with 6 fractional bits:
//   e = floor(log2 max|x|) + 127,   q = RNE(x 2^(133 - e)) in [-127, 127],   x~ = q 2^(e - 133)
// (1.03 bytes per element).  A 7-bit magnitude times a power of two is a bf16 value -- down to
// e = 0, where 2^-133 is bf16's smallest subnormal -- so the bf16 tensor cores of the backward see
// the stored values exactly.  A block with a NaN or an infinity gets e = 255 and decodes to NaN.
// q [T, d_in] int8 and scales [T, d_in / 32], both row-major.
//
// Adapter gradients from it (k_act_gemm): the int8 tile is brought to shared memory by TMA and
// turned into the swizzled bf16 operand there, so no bf16 copy of X is ever in HBM:
//   dA^T[d_in, r] = X~^T (s G)       A operand MN-major (the tokens are K)
//   U[T, r]       = X~ A^T           A operand K-major
// The other operand comes as one or two bf16 matrices hi + lo (a value's bf16 rounding and the
// rounding of what is left: 16 significant bits), accumulated in the same fp32 tile, so that
// rounding G (or U) to the tensor cores' type costs 2^-18 of a gradient and not 2^-9.
#pragma once

#include "common.cuh"
#include "mxfp4.cuh"

namespace qlora {

// 2^(e - 133) as fp32: the value of one integer step; exact (subnormal for e < 7), NaN for 255.
__device__ __forceinline__ float act8_step(uint32_t e) {
    return __uint_as_float(e == 255u ? 0x7FFFFFFFu : (e >= 7u ? (e - 6u) << 23 : 1u << (e + 16u)));
}

// Four lanes per block of 32, eight elements per lane.
template <typename T>
__global__ void __launch_bounds__(256) k_act8_quantize(const T* __restrict__ X, int64_t n8,
                                                       int8_t* __restrict__ q, uint8_t* __restrict__ scales) {
    griddep_enter();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    // n8 is a multiple of 4 (whole blocks) and blockDim of 32: a quad is never split
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i - (threadIdx.x & 31) < n8;
         i += stride) {
        float x[8];
        uint32_t m = 0;
        const bool in = i < n8;
        if (in) m = load8(X + i * 8, x);
        const uint32_t e = quad_max(m) >> 23;
        if (!in) continue;
        // x 2^(133 - e) in two exact steps (2^133 is no fp32 value)
        const uint32_t ec = max(e, 6u);
        const float f = __uint_as_float((260u - ec) << 23);
        const float g = static_cast<float>(1u << (ec - e));
        uint32_t w[2] = {0, 0};
        if (e != 255u) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float y = fminf(fmaxf(rintf(__fmul_rn(__fmul_rn(x[k], f), g)), -127.f), 127.f);
                w[k >> 2] |= (static_cast<uint32_t>(static_cast<int>(y)) & 255u) << (8 * (k & 3));
            }
        }
        reinterpret_cast<uint2*>(q)[i] = make_uint2(w[0], w[1]);
        if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(e);
    }
}

// Four int8 to fp32: 2^23 + (q + 128) is put together from bits (no integer conversion), then
// 2^23 + 128 is taken off again; both steps are exact.
__device__ __forceinline__ void int8x4_to_f32(uint32_t q, float (&f)[4]) {
    const uint32_t u = q ^ 0x80808080u;
    f[0] = __uint_as_float(prmt(u, 0x4B000000u, 0x7650)) - 8388736.f;
    f[1] = __uint_as_float(prmt(u, 0x4B000000u, 0x7651)) - 8388736.f;
    f[2] = __uint_as_float(prmt(u, 0x4B000000u, 0x7652)) - 8388736.f;
    f[3] = __uint_as_float(prmt(u, 0x4B000000u, 0x7653)) - 8388736.f;
}

// Eight int8 times the block's step, as bf16 (exact).
__device__ __forceinline__ uint4 act8_decode8(uint32_t q0, uint32_t q1, float s) {
    float a[4], b[4];
    int8x4_to_f32(q0, a);
    int8x4_to_f32(q1, b);
    return make_uint4(pack_bf16x2(a[0] * s, a[1] * s), pack_bf16x2(a[2] * s, a[3] * s),
                      pack_bf16x2(b[0] * s, b[1] * s), pack_bf16x2(b[2] * s, b[3] * s));
}

template <typename T>
__global__ void __launch_bounds__(256) k_act8_dequant(const int8_t* __restrict__ q,
                                                      const uint8_t* __restrict__ scales, int64_t n8,
                                                      T* __restrict__ out) {
    griddep_enter();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n8;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(q) + i);
        const float s = act8_step(__ldg(scales + (i >> 2)));
        if constexpr (sizeof(T) == 4) {
            float a[4], b[4];
            int8x4_to_f32(v.x, a);
            int8x4_to_f32(v.y, b);
            float4* o = reinterpret_cast<float4*>(out) + 2 * i;
            o[0] = make_float4(a[0] * s, a[1] * s, a[2] * s, a[3] * s);
            o[1] = make_float4(b[0] * s, b[1] * s, b[2] * s, b[3] * s);
        } else {
            reinterpret_cast<uint4*>(out)[i] = act8_decode8(v.x, v.y, s);
        }
    }
}

// ------------------------------------------------------------------ adapter products

// How the A operand of k_act_gemm is stored.
enum : int {
    kActBf16Mn = 0,   // bf16 [K, M] (tokens are K): TMA straight into the MN-major operand
    kActInt8Mn = 1,   // int8 [K, M] with scales [K, M / 32]: decoded into the MN-major operand
    kActInt8K = 2     // int8 [M, K] with scales [M, K / 32]: decoded into the K-major operand
};

struct ActGemmArgs {
    int M, N;                // output rows (channels or tokens) and valid columns (the rank)
    int64_t K;               // contraction length
    int k_steps;             // ceil(K / 64)
    int split;               // split-K over grid.z
    int nb;                  // B matrices: 1, or 2 for hi + lo
    const uint8_t* scales;   // E8M0 bytes of the int8 operand
    int64_t ld_scales;       // blocks per stored row
    float* part;             // fp32 partials: [split][M][ldp], or transposed [split][N][M]
    int64_t ldp;
    int transposed;
    int* err;
    uint64_t wait_ns;
};

// RPT: the padded rank (B tile columns), 64 or 128.
template <int MODE, int RPT>
struct ActGemmSmem {
    static constexpr int kA = 128 * 64 * 2;                     // bf16 operand tile
    static constexpr int kRaw = MODE == kActBf16Mn ? 0 : 128 * 64;
    static constexpr int kB = RPT * 64 * 2;                     // one B matrix's tile
    static constexpr int kStage = kA + kRaw + 2 * kB;
    static constexpr int kStages = 4;
    static constexpr int kTotal = 1024 + kStages * kStage + 256;
    static_assert(kTotal <= 232448, "shared memory budget");
};

// D[M, RPT] = sum over K of A[M, K] (B0 + B1)[RPT, K], fp32 split-K partials.  Warp 0: TMA; warp 1:
// MMA; warps 2..9: int8 decode (one 32-element block per thread and stage), then the epilogue.
// B is MN-major ([K, rank] rows) for the Mn modes and K-major ([rank, K]) for kActInt8K.
// Memory-bound: per K step of 64 a tile reads 8 KB of int8 and 2 to 4 B tiles that stay in L2.
template <int MODE, int RPT>
__global__ void __launch_bounds__(320, 1)
    k_act_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
               const __grid_constant__ CUtensorMap tmB1, const ActGemmArgs args) {
    using L = ActGemmSmem<MODE, RPT>;
    constexpr int S = L::kStages;
    constexpr bool kMn = MODE != kActInt8K;
    constexpr bool kDecode = MODE != kActBf16Mn;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + S * L::kA;
    uint8_t* sR = sB + S * 2 * L::kB;
    uint64_t* full = reinterpret_cast<uint64_t*>(sR + S * L::kRaw);
    uint64_t* empty = full + S;
    uint64_t* decoded = empty + S;
    uint64_t* accf = decoded + S;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m0 = blockIdx.x * 128;
    const int z = blockIdx.y;
    const int per = (args.k_steps + args.split - 1) / args.split;
    const int k_begin = z * per;
    const int n_iters = max(0, min(args.k_steps, k_begin + per) - k_begin);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&decoded[s], 8);
        }
        mbar_init(accf, 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB0);
        if (args.nb > 1) tma_prefetch_desc(&tmB1);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, RPT);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_acc = *tmem_slot;
    griddep_enter();

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int it = 0; it < n_iters; ++it) {
                const int s = it % S;
                if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1, abort, args.wait_ns)) {
                    set_error(args.err, kErrTimeout);
                    *abort = 1;
                    break;
                }
                const int kx = (k_begin + it) * 64;
                mbar_arrive_expect_tx(&full[s], (kDecode ? L::kRaw : L::kA) + args.nb * L::kB);
                if (MODE == kActBf16Mn) {
                    tma_load_2d(sA + s * L::kA, &tmA, &full[s], m0, kx);
                    tma_load_2d(sA + s * L::kA + 8192, &tmA, &full[s], m0 + 64, kx);
                } else if (MODE == kActInt8Mn) {
                    tma_load_2d(sR + s * L::kRaw, &tmA, &full[s], m0, kx);
                } else {
                    tma_load_2d(sR + s * L::kRaw, &tmA, &full[s], kx, m0);
                }
                for (int b = 0; b < args.nb; ++b) {
                    const CUtensorMap* mb = b ? &tmB1 : &tmB0;
                    uint8_t* dst = sB + (s * 2 + b) * L::kB;
                    if (kMn) {
#pragma unroll
                        for (int c = 0; c < RPT / 64; ++c) tma_load_2d(dst + c * 8192, mb, &full[s], c * 64, kx);
                    } else {
                        tma_load_2d(dst, mb, &full[s], kx, 0);
                    }
                }
                issued = it + 1;
            }
            if (*abort)
                for (int it = max(0, issued - S); it < issued; ++it)
                    mbar_wait(&full[it % S], (it / S) & 1, nullptr, args.wait_ns);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = make_idesc_bf16(128, RPT, kMn, kMn);
            for (int it = 0; it < n_iters; ++it) {
                const int s = it % S;
                const uint32_t ph = (it / S) & 1;
                bool ok = mbar_wait(&full[s], ph, abort, args.wait_ns);
                if (ok && kDecode) ok = mbar_wait(&decoded[s], ph, abort, args.wait_ns);
                if (!ok) {
                    set_error(args.err, kErrTimeout);
                    *abort = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t a = smem_u32(sA + s * L::kA);
                for (int b = 0; b < args.nb; ++b) {
                    const uint32_t bb = smem_u32(sB + (s * 2 + b) * L::kB);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16_ss(tmem_acc,
                                     kMn ? make_sw128_desc(a + k * 2048, 8192, 1024) : make_sw128_desc(a + k * 32, 16, 1024),
                                     kMn ? make_sw128_desc(bb + k * 2048, 8192, 1024) : make_sw128_desc(bb + k * 32, 16, 1024),
                                     idesc, (it > 0 || b > 0 || k > 0) ? 1u : 0u);
                }
                umma_commit(&empty[s]);
            }
            umma_commit(accf);
        }
    } else {
        if (kDecode) {
            const int td = threadIdx.x - 64;                     // 0..255: the block of this thread
            const int row = kMn ? td >> 2 : td >> 1;              // row of the int8 tile
            const int b = kMn ? td & 3 : td & 1;                  // block within the row
            auto scale_at = [&](int it) -> uint32_t {
                const int64_t kx = static_cast<int64_t>(k_begin + it) * 64;
                const int64_t srow = kMn ? kx + row : m0 + row;
                const int64_t blk = (kMn ? m0 / 32 : kx / 32) + b;
                const int64_t rows = kMn ? args.K : args.M;
                if (it >= n_iters || srow >= rows || blk >= args.ld_scales) return 0u;
                return __ldg(args.scales + srow * args.ld_scales + blk);
            };
            uint32_t e_nxt = scale_at(0);
            for (int it = 0; it < n_iters; ++it) {
                const int s = it % S;
                const uint32_t e = e_nxt;
                e_nxt = scale_at(it + 1);
                if (!mbar_wait(&full[s], (it / S) & 1, abort, args.wait_ns)) {
                    set_error(args.err, kErrTimeout);
                    *abort = 1;
                    break;
                }
                // (elements outside the matrix were filled with 0 by the copy)
                const uint4* src = reinterpret_cast<const uint4*>(sR + s * L::kRaw + td * 32);
                const uint4 v0 = src[0], v1 = src[1];
                const float st = act8_step(e);
                uint8_t* dst = sA + s * L::kA + (kMn ? (b >> 1) * 8192 + row * 128 : row * 128);
                const int c0 = kMn ? (b & 1) * 4 : b * 4, sw = row & 7;
                *reinterpret_cast<uint4*>(dst + (((c0 + 0) ^ sw) << 4)) = act8_decode8(v0.x, v0.y, st);
                *reinterpret_cast<uint4*>(dst + (((c0 + 1) ^ sw) << 4)) = act8_decode8(v0.z, v0.w, st);
                *reinterpret_cast<uint4*>(dst + (((c0 + 2) ^ sw) << 4)) = act8_decode8(v1.x, v1.y, st);
                *reinterpret_cast<uint4*>(dst + (((c0 + 3) ^ sw) << 4)) = act8_decode8(v1.z, v1.w, st);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&decoded[s]);
            }
        }
        if (!mbar_wait(accf, 0, nullptr, args.wait_ns)) {
            set_error(args.err, kErrTimeout);
            *abort = 1;
        }
        tc_fence_after();
        if (!*abort) {
            const int q = warp & 3, half = (warp - 2) >> 2;
            const int64_t grow = static_cast<int64_t>(m0) + q * 32 + lane;
            float* out = args.part + static_cast<int64_t>(z) * (args.transposed ? args.N : args.M) *
                                         (args.transposed ? static_cast<int64_t>(args.M) : args.ldp);
#pragma unroll 1
            for (int c0 = half * (RPT / 2); c0 < (half + 1) * (RPT / 2) && c0 < args.N; c0 += 32) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(tmem_acc + (static_cast<uint32_t>(q * 32) << 16) + c0, r);
                tmem_ld_wait();
                if (grow < args.M) {
                    if (args.transposed) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j < args.N) out[static_cast<int64_t>(c0 + j) * args.M + grow] = __uint_as_float(r[j]);
                    } else {
                        // rows of ldp floats, ldp a multiple of 4: 16-byte stores up to the rank
                        float* o = out + grow * args.ldp + c0;
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            if (c0 + 4 * g < args.N)
                                *reinterpret_cast<uint4*>(o + 4 * g) =
                                    make_uint4(r[4 * g], r[4 * g + 1], r[4 * g + 2], r[4 * g + 3]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_acc, RPT);
    }
}

// Sum split-K partials P[z][t][j] (row stride ldp) in z order and write v = scale sum as the bf16 pair
// hi = bf16(v), lo = bf16(v - hi), each [T, ld] (columns j >= r are zero).
__global__ void __launch_bounds__(256) k_finalize_pair(const float* __restrict__ P, int split, int64_t T, int r,
                                                       int ldp, float scale, int ld,
                                                       __nv_bfloat16* __restrict__ hi,
                                                       __nv_bfloat16* __restrict__ lo) {
    griddep_enter();
    const int64_t n = T * ld, stride = T * ldp;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = i / ld;
        const int j = static_cast<int>(i - t * ld);
        float acc = 0.f;
        if (j < r)
            for (int z = 0; z < split; ++z) acc += P[z * stride + t * ldp + j];
        const float v = scale * acc;
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        const float rest = v - __bfloat162float(h);
        hi[i] = h;
        // an infinite or NaN v is carried by hi alone (inf - inf would turn it into NaN)
        lo[i] = __float2bfloat16_rn(fabsf(rest) < __int_as_float(0x7F800000) ? rest : 0.f);
    }
}

// out[i] = scale sum_z P[z][i] over n elements (partials of out's own layout), or added to out.
__global__ void __launch_bounds__(256) k_finalize_flat(const float* __restrict__ P, int split, int64_t n,
                                                       float scale, float* __restrict__ out, int accumulate) {
    griddep_enter();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        float acc = 0.f;
        for (int z = 0; z < split; ++z) acc += P[z * n + i];
        out[i] = accumulate ? out[i] + scale * acc : scale * acc;
    }
}

// out[m, j] = scale sum_z P[z][m][j] (row stride ldp), j < r, or added to out.
__global__ void __launch_bounds__(256) k_finalize_strided(const float* __restrict__ P, int split, int64_t M, int r,
                                                          int ldp, float scale, float* __restrict__ out,
                                                          int accumulate) {
    griddep_enter();
    const int64_t n = M * r, stride = M * ldp;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t m = i / r;
        float acc = 0.f;
        for (int z = 0; z < split; ++z) acc += P[z * stride + m * ldp + (i - m * r)];
        out[i] = accumulate ? out[i] + scale * acc : scale * acc;
    }
}

}  // namespace qlora
