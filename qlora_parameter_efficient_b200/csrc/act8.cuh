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
// The adapter products of a backward that reads it (k_act_gemm): the int8 tile is brought to shared
// memory by TMA and turned into the swizzled bf16 operand there, so no bf16 copy of X is ever in HBM:
//   dA^T[d_in, r] = X~^T (s G)       A operand MN-major (the tokens are K)
//   U[T, r]       = X~ A^T           A operand K-major
// and with bf16 operands G = dH B, dB = s dH^T U, and both of the above from a bf16 X.
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

struct ActGemmArgs {
    int M, N;                // output rows (channels or tokens) and valid columns (the rank)
    int64_t K;               // contraction length
    int k_steps;             // ceil(K / 64)
    int split;               // split-K over grid.y
    const uint8_t* scales;   // E8M0 bytes of the int8 operand, row-major
    int64_t ld_scales;       // blocks per stored row
    float* part;             // fp32 partials: [split][M][ldp], or transposed [split][N][M]
    int64_t ldp;
    int transposed;
    int* err;
    uint64_t wait_ns;
};

// RPT: the padded rank, 64 or 128 (B tile rows); NB: bf16 matrices whose sum B is, 1 or 3.
template <bool INT8, int RPT, int NB>
struct ActGemmSmem {
    static constexpr int kA = 128 * 64 * 2;                     // bf16 operand tile
    static constexpr int kRaw = INT8 ? 128 * 64 : 0;
    static constexpr int kB = RPT * 64 * 2;                     // one B matrix's tile
    static constexpr int kStage = kA + kRaw + NB * kB;
    static constexpr int kStages = 221184 / kStage < 6 ? 221184 / kStage : 6;
    static constexpr int kTotal = 1024 + kStages * kStage + 512;
    // K steps of 64 per accumulator segment (see the kernel)
    static constexpr int kSeg = NB == 1 ? 4 : 2;
    static_assert(kTotal <= 232448 && kStages >= 3, "shared memory budget");
};

// D[M, N] = sum over K of A[M, K] B[N, K], B the sum of NB bf16 matrices; fp32 split-K partials.
//   INT8   A is int8 with E8M0 scales, decoded to bf16 in shared memory (else bf16)
//   AMN    A is stored [K, M] (tokens are K) and consumed MN-major, else [M, K]
//   BMN    B is stored [K, N], else [N, K]; B's tensor map is three-dimensional, matrix outermost
// Warp 0: TMA; warp 1: MMA; warps 2..9: int8 decode (one 32-element block per thread and stage),
// accumulator drains, partials.
//
// Precision: the results are fp32 gradients.  (1) A value that was computed here (s G, a recomputed U)
// is given to the bf16 tensor cores as the three bf16 numbers that make up its 24 bits, so nothing is
// rounded off it.  (2) The tensor core's running fp32 sum is truncated at every MMA -- a bias that
// grows with the chain: 9e-6 of a gradient over 8192 tokens.  So the chain is cut into segments of
// 16 or 24 MMAs, whose sums warps 2..9 add up in registers, rounding to nearest, from two
// accumulator tiles in turn.
// Bound by memory: a K step of 64 reads 8 KB of int8 (or 16 KB of bf16) from HBM and the B tiles from
// L2; N is the rank rounded up to 16, so that the MMAs stay below that.
template <bool INT8, bool AMN, bool BMN, int RPT, int NB>
__global__ void __launch_bounds__(320, 1)
    k_act_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const ActGemmArgs args) {
    using L = ActGemmSmem<INT8, RPT, NB>;
    constexpr int S = L::kStages, kSeg = L::kSeg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + S * L::kA;
    uint8_t* sR = sB + S * NB * L::kB;
    uint64_t* full = reinterpret_cast<uint64_t*>(sR + S * L::kRaw);
    uint64_t* empty = full + S;
    uint64_t* decoded = empty + S;
    uint64_t* accf = decoded + S;         // [2] segment complete
    uint64_t* acc_free = accf + 2;        // [2] segment drained (8 warp arrivals)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_free + 2);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m0 = blockIdx.x * 128;
    const int z = blockIdx.y;
    const int per = (args.k_steps + args.split - 1) / args.split;
    const int k_begin = z * per;
    const int n_iters = max(0, min(args.k_steps, k_begin + per) - k_begin);
    const int n_seg = (n_iters + kSeg - 1) / kSeg;
    const int n_mma = (args.N + 15) & ~15;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&decoded[s], 8);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acc_free[b], 8);
        }
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 2 * RPT);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_enter();

    auto fail = [&]() {
        set_error(args.err, kErrTimeout);
        *abort = 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int it = 0; it < n_iters; ++it) {
                const int s = it % S;
                if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1, abort, args.wait_ns)) {
                    fail();
                    break;
                }
                const int kx = (k_begin + it) * 64;
                mbar_arrive_expect_tx(&full[s], (INT8 ? L::kRaw : L::kA) + NB * L::kB);
                uint8_t* a = INT8 ? sR + s * L::kRaw : sA + s * L::kA;
                if (AMN) {
                    tma_load_2d(a, &tmA, &full[s], m0, kx);
                    if (!INT8) tma_load_2d(a + 8192, &tmA, &full[s], m0 + 64, kx);
                } else {
                    tma_load_2d(a, &tmA, &full[s], kx, m0);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint8_t* dst = sB + (s * NB + b) * L::kB;
                    if (BMN) {
#pragma unroll
                        for (int c = 0; c < RPT / 64; ++c) tma_load_3d(dst + c * 8192, &tmB, &full[s], c * 64, kx, b);
                    } else {
                        tma_load_3d(dst, &tmB, &full[s], kx, 0, b);
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
            const uint32_t idesc = make_idesc_bf16(128, n_mma, AMN, BMN);
            for (int it = 0; it < n_iters; ++it) {
                const int s = it % S, seg = it / kSeg;
                const uint32_t ph = (it / S) & 1;
                bool ok = true;
                if (it % kSeg == 0 && seg >= 2)
                    ok = mbar_wait(&acc_free[seg & 1], ((seg >> 1) & 1) ^ 1, abort, args.wait_ns);
                if (ok) ok = mbar_wait(&full[s], ph, abort, args.wait_ns);
                if (ok && INT8) ok = mbar_wait(&decoded[s], ph, abort, args.wait_ns);
                if (!ok) {
                    fail();
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>((seg & 1) * RPT);
                const uint32_t a = smem_u32(sA + s * L::kA);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t bb = smem_u32(sB + (s * NB + b) * L::kB);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16_ss(d, AMN ? make_sw128_desc(a + k * 2048, 8192, 1024) : make_sw128_desc(a + k * 32, 16, 1024),
                                     BMN ? make_sw128_desc(bb + k * 2048, 8192, 1024) : make_sw128_desc(bb + k * 32, 16, 1024),
                                     idesc, (it % kSeg > 0 || b > 0 || k > 0) ? 1u : 0u);
                }
                umma_commit(&empty[s]);
                if (it % kSeg == kSeg - 1 || it == n_iters - 1) umma_commit(&accf[seg & 1]);
            }
        }
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;      // lane quarter, half of the columns
        constexpr int kHalf = RPT / 2;
        float acc[kHalf];
#pragma unroll
        for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;
        bool ok = true;
        auto drain = [&](int seg) {
            ok = mbar_wait_warp(&accf[seg & 1], (seg >> 1) & 1, abort, args.wait_ns);
            if (!ok) return;
            tc_fence_after();
            const uint32_t t = tmem + (static_cast<uint32_t>(q * 32) << 16) + (seg & 1) * RPT + half * kHalf;
#pragma unroll
            for (int c = 0; c < kHalf; c += 32)
                if (half * kHalf + c < args.N) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(t + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[c + j] += __uint_as_float(r[j]);
                }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_free[seg & 1]);
        };
        const int td = threadIdx.x - 64;                      // 0..255: the int8 block of this thread
        const int row = AMN ? td >> 2 : td >> 1;              // row of the int8 tile
        const int blk_in = AMN ? td & 3 : td & 1;             // block within the row
        auto scale_at = [&](int it) -> uint32_t {
            const int64_t kx = static_cast<int64_t>(k_begin + it) * 64;
            const int64_t srow = AMN ? kx + row : m0 + row;
            const int64_t blk = (AMN ? m0 / 32 : kx / 32) + blk_in;
            const int64_t rows = AMN ? args.K : args.M;
            if (it >= n_iters || srow >= rows || blk >= args.ld_scales) return 0u;
            return __ldg(args.scales + srow * args.ld_scales + blk);
        };
        uint32_t e_nxt = INT8 ? scale_at(0) : 0u;
        for (int seg = 0; ok && seg < n_seg; ++seg) {
            if (INT8) {
                for (int it = seg * kSeg; it < min(n_iters, (seg + 1) * kSeg); ++it) {
                    const int s = it % S;
                    const uint32_t e = e_nxt;
                    e_nxt = scale_at(it + 1);
                    ok = mbar_wait_warp(&full[s], (it / S) & 1, abort, args.wait_ns);
                    if (!ok) break;
                    // (elements outside the matrix were filled with 0 by the copy)
                    const uint4* src = reinterpret_cast<const uint4*>(sR + s * L::kRaw + td * 32);
                    const uint4 v0 = src[0], v1 = src[1];
                    const float st = act8_step(e);
                    uint8_t* dst = sA + s * L::kA + (AMN ? (blk_in >> 1) * 8192 + row * 128 : row * 128);
                    const int c0 = AMN ? (blk_in & 1) * 4 : blk_in * 4, sw = row & 7;
                    *reinterpret_cast<uint4*>(dst + (((c0 + 0) ^ sw) << 4)) = act8_decode8(v0.x, v0.y, st);
                    *reinterpret_cast<uint4*>(dst + (((c0 + 1) ^ sw) << 4)) = act8_decode8(v0.z, v0.w, st);
                    *reinterpret_cast<uint4*>(dst + (((c0 + 2) ^ sw) << 4)) = act8_decode8(v1.x, v1.y, st);
                    *reinterpret_cast<uint4*>(dst + (((c0 + 3) ^ sw) << 4)) = act8_decode8(v1.z, v1.w, st);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&decoded[s]);
                }
            }
            // one segment behind the decode, so that the MMAs of this one run meanwhile
            if (ok && seg >= 1) drain(seg - 1);
        }
        if (ok && n_seg > 0) drain(n_seg - 1);
        if (!ok) fail();
        const int64_t grow = static_cast<int64_t>(m0) + q * 32 + lane;
        if (ok && grow < args.M) {
            const int c0 = half * kHalf;
            if (args.transposed) {
                float* out = args.part + static_cast<int64_t>(z) * args.N * args.M + grow;
#pragma unroll
                for (int j = 0; j < kHalf; ++j)
                    if (c0 + j < args.N) out[static_cast<int64_t>(c0 + j) * args.M] = acc[j];
            } else {
                // rows of ldp floats (a multiple of 4): 16-byte stores up to the rank
                float* out = args.part + (static_cast<int64_t>(z) * args.M + grow) * args.ldp + c0;
#pragma unroll
                for (int j = 0; j < kHalf; j += 4)
                    if (c0 + j < args.N)
                        *reinterpret_cast<float4*>(out + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * RPT);
    }
}

// Sum split-K partials P[z][t][j] (row stride ld) in z order; v = scale sum is written as the three bf16
// numbers out[0] + out[1] + out[2] = v (8 significant bits each), matrices [T, ld], columns
// j >= r zero.  An infinite or NaN v is carried by the first alone (inf - inf would make it NaN).
__global__ void __launch_bounds__(256) k_finalize_triple(const float* __restrict__ P, int split, int64_t T, int r,
                                                         int ld, float scale, __nv_bfloat16* __restrict__ out) {
    griddep_enter();
    const int64_t n = T * ld;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int j = static_cast<int>(i % ld);
        float acc = 0.f;
        if (j < r)
            for (int z = 0; z < split; ++z) acc += P[z * n + i];
        float v = scale * acc;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const __nv_bfloat16 h = __float2bfloat16_rn(v);
            out[k * n + i] = h;
            const float rest = v - __bfloat162float(h);
            v = fabsf(rest) < __int_as_float(0x7F800000) ? rest : 0.f;
        }
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
