// mx_gemm.cuh -- block-scaled MXFP4 products of the layer's forward (sm_100a kind::mxf4).
//
//   H[T, d_out] = X4[T, d_in] W4[d_out, d_in]^T + sU[T, RP] B[d_out, RP]^T
//
// Both operands of the main K steps stay 4-bit: tcgen05.mma kind::mxf4.block_scale reads the E2M1
// codes from swizzled shared memory and the E8M0 scales from tensor memory, and accumulates the
// exact products of the stored values in fp32, so nothing is decoded.  The adapter enters as bf16
// kind::f16 K steps into the same accumulator.  A K stage is 256 elements: one 128-byte swizzled row
// of codes per matrix row, and per 128 rows two stored 512-byte scale tiles, which
// tcgen05.cp.32x128b.warpx4 copies into four tensor-memory columns each; an MMA (K = 64) takes half
// a tile, picked by the scale-factor id of its instruction descriptor.
//
// k_mx_stream: one CTA per 128 weight rows, the tokens as the (narrow) N operand, K split over the
//   ranks of a cluster whose partials meet in shared memory.  For token counts whose time is the
//   weight stream.
// k_pair_gemm: persistent pairs of CTAs (cta_group::2) on 256 x 256 tiles, for the rest; with bf16
//   operands also the backward's dX over a decoded weight.
#pragma once

#include "act8.cuh"
#include "common.cuh"
#include "mxfp4.cuh"
#include "nf4_gemm2.cuh"
#include "pair_schedule.cuh"

namespace qlora {

// ------------------------------------------------------------------ PTX

// Instruction descriptor of kind::mxf4: E2M1 x E2M1, E8M0 scales, fp32 D, K-major operands.
// a_id / b_id: which half (0 or 2) of the four scale bytes of a tensor-memory word is used.
__device__ __forceinline__ uint32_t make_idesc_mxf4(int M, int N, uint32_t a_id, uint32_t b_id) {
    return (b_id << 4)                                // B scale-factor id
           | (1u << 7)                                // A format E2M1
           | (1u << 10)                               // B format E2M1
           | (static_cast<uint32_t>(N >> 3) << 17)    // N / 8
           | (1u << 23)                               // scale format E8M0
           | (static_cast<uint32_t>(M >> 7) << 27)    // M / 128
           | (a_id << 29);                            // A scale-factor id
}

template <int CG>
__device__ __forceinline__ void umma_mxf4_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
                d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
                d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// Copy one 512-byte scale tile (32 lines of 16 bytes) to four tensor-memory columns, repeated for
// the four lane quarters.
// Its shared-memory descriptor: no swizzle, 8-line groups of 128 bytes, 128 bytes apart.
__device__ __forceinline__ uint64_t make_scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (8ull << 32) | (1ull << 46);
}
template <int CG>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// The adapter side of a decode-size call (T <= 16), beside which the weight stream already runs.  CTAs
// [0, r): one adapter row j each, U[:, j] = X A[j]^T in fp32, written unscaled to u_save (nullable,
// [T, r]) and s U as two bf16 terms to us [T, ext_ld(r)]; the rest: B copied to padded rows (only where r is
// not a multiple of 8).
// Bound by latency (out of HBM 5.1 us at one token of 4096, r = 16; 9.3 us at 13 tokens, r = 64), most
// of it behind the stream.
constexpr int kMxDecodeT = 16;
struct MxPrepArgs {
    const __nv_bfloat16 *X, *A;
    int T, r;
    int64_t d_in;
    float s;
    __nv_bfloat16 *u_save, *us;
    PadCopy pad;
};
__global__ void __launch_bounds__(256) k_mx_prepare(const MxPrepArgs a) {
    __shared__ float s_red[8][kMxDecodeT];
    griddep_launch_dependents();
    const int j = blockIdx.x;
    if (j >= a.r) {
        a.pad.run(j - a.r);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float acc[kMxDecodeT];
#pragma unroll
    for (int t = 0; t < kMxDecodeT; ++t) acc[t] = 0.f;
    for (int64_t c = threadIdx.x * 8; c < a.d_in; c += 256 * 8) {
        float w[8];
        load8(a.A + j * a.d_in + c, w);
#pragma unroll
        for (int t = 0; t < kMxDecodeT; ++t)
            if (t < a.T) {
                float x[8];
                load8(a.X + t * a.d_in + c, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[t] = fmaf(w[i], x[i], acc[t]);
            }
    }
#pragma unroll
    for (int t = 0; t < kMxDecodeT; ++t)
        if (t < a.T) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
            if (lane == 0) s_red[warp][t] = acc[t];
        }
    __syncthreads();
    if (threadIdx.x < a.T) {
        const int t = threadIdx.x;
        float u = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) u += s_red[w][t];
        if (a.u_save) a.u_save[t * a.r + j] = __float2bfloat16_rn(u);
        const int stride = act_triple(a.r).stride;
        __nv_bfloat16* us = a.us + t * ext_ld(a.r) + j;
        float x[4] = {a.s * u, 0.f, 0.f, 0.f};
        const uint2 hi = bf16_term(x), lo = bf16_term(x);
        us[0] = __ushort_as_bfloat16(static_cast<unsigned short>(hi.x));
        us[stride] = __ushort_as_bfloat16(static_cast<unsigned short>(lo.x));
        if (j == a.r - 1)
            for (int c = 1; j + c < ((a.r + 15) & ~15); ++c) us[c] = us[stride + c] = __float2bfloat16_rn(0.f);
    }
}

// Untiled copy of whole scale tiles (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// ------------------------------------------------------------------ weight-streaming kernel

struct MxStreamArgs {
    int T, d_out;
    int k64;                  // d_in / 64: MMAs of the whole contraction
    int col_tiles;            // scale tiles per row of tiles (d_in / 128, rounded up)
    int ranks;                // CTAs per cluster (1, 2 or 4), K split over them
    int stages;               // of the ring
    ExtSteps ext;             // the adapter's K steps, taken by the last rank
    const uint8_t* w_scales;
    const uint8_t* x_scales;  // MXFP4 X (NT > 16), or
    const __nv_bfloat16* X;   // X itself (NT = 16), quantized by the CTAs that use it
    int64_t d_in;
    __nv_bfloat16* out;       // [T, d_out]
    int* err;
    uint64_t wait_ns;
};

// Warps that quantize one stage of X at T <= 16: four rows each, 1, 2 or 4 of them.
__device__ __forceinline__ int quant_warps(int T) { return T <= 4 ? 1 : (T <= 8 ? 2 : 4); }

// NT: tokens per CTA (the MMA's N): 16 or 64 for calls of up to that many tokens, 128 (a whole scale
// tile) in several token tiles above.
template <int NT>
struct MxStreamCfg {
    static constexpr int kA = 128 * 128;            // codes of 128 weight rows, one stage
    static constexpr int kB = NT * 128;             // codes of the tokens
    static constexpr int kSf = 1024;                // two scale tiles (each operand)
    static constexpr int kStage = kA + kB + 2 * kSf;
    // stages of the ring where two CTAs share an SM, and where each has one to itself (200 tokens of an
    // 8192 x 8192 layer 28.6 us with three stages, 26.0 with four or more)
    static constexpr int kShared = NT <= 16 ? 5 : (NT <= 64 ? 4 : 3);
    static constexpr int kAlone = NT <= 16 ? 11 : (NT <= 64 ? 8 : 6);
    static constexpr int bytes(int stages) { return 1024 + stages * kStage + 256; }
    static constexpr bool kQuant = NT == 16;
    static constexpr int kRed = NT * 128 * 4; // partials of this rank's share of the rows (over the ring)
    static constexpr int kQuantWarps = 8, kQuantGroups = 4;
    static_assert(!kQuant || kQuantGroups <= kShared, "a group per ring stage at most");
    static constexpr int kThreads = kQuant ? 64 + 32 * kQuantWarps : 192;
    static constexpr int kAcc = NT < 32 ? 32 : NT;  // accumulator columns
    // and sets of 16 scale columns: with two, a stage waits for the last but one to complete
    static constexpr int kSets = 4;
    static constexpr uint32_t kTmem = NT <= 64 ? 128 : 256;
    static_assert(kAcc + 16 * kSets <= static_cast<int>(kTmem), "tensor memory");
    static_assert((bytes(kShared) + 1024) * 2 <= 233472 && bytes(kAlone) <= 232448 && kRed <= kStage * kShared,
                  "shared memory budget");
};

// Sum of the C ranks' partials of 128 / C weight rows from col0 on, red[rank][token][row], in the order
// of the ranks (= of K), and its output columns.  By all threads, two rows each and several at once: one
// element at a time by four warps took 3 us at 64 tokens, 10 us at 128.
template <int C, int NT, int THREADS>
__device__ __forceinline__ void mx_join(const float* red, int t_end, int col0, int t0, const MxStreamArgs& args) {
    constexpr int R = 128 / C;
    const bool pairs = !(args.d_out & 1);
#pragma unroll 4
    for (int i = 2 * threadIdx.x; i < R * t_end; i += 2 * THREADS) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float2 v = *reinterpret_cast<const float2*>(red + c * NT * R + i);
            x += v.x;
            y += v.y;
        }
        const int col = col0 + i % R;
        __nv_bfloat16* out = args.out + static_cast<int64_t>(t0 + i / R) * args.d_out + col;
        if (pairs) {
            if (col < args.d_out) *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(x, y);
        } else {
            if (col < args.d_out) out[0] = __float2bfloat16_rn(x);
            if (col + 1 < args.d_out) out[1] = __float2bfloat16_rn(y);
        }
    }
}

// grid: x = weight tile * ranks + rank, y = token tile; clusters of `ranks` along x.
// Bound: 24 to 34 KB a stage into one SM, 0.29 us (60 bytes a cycle) however many CTAs run, so K is split
// until every SM has a CTA: 64 tokens of a 4096 x 11008 layer 28.3 us on 32 SMs, 19.3 us on 128
// (whole forward, weight out of HBM).
// Launched with programmatic dependent launch: the weight's tiles are read before the kernel in front
// (which forms U and, for NT > 16, quantizes X) has finished; that kernel is launched without it, so
// whatever wrote the weight and X is done.  What it writes is read, and H written, after it has ended.
// NT = 16: warps 2..9 quantize this rank's part of X into the ring themselves, one block of 32 per
// thread and stage, so that the stream does not wait for another kernel before its last step.
template <int NT>
__global__ void __launch_bounds__(MxStreamCfg<NT>::kThreads)
    k_mx_stream(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ CUtensorMap tmBx, const __grid_constant__ CUtensorMap tmUx,
                const MxStreamArgs args) {
    using L = MxStreamCfg<NT>;
    const int S = args.stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + S * L::kA;
    uint8_t* sSa = sB + S * L::kB;
    uint8_t* sSb = sSa + S * L::kSf;
    float* red = reinterpret_cast<float*>(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * L::kStage);
    uint64_t* empty = full + S;
    uint64_t* accf = empty + S;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int C = args.ranks;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tile = blockIdx.x / C;
    const int n0 = tile * 128;
    const int t0 = blockIdx.y * NT;
    const int chunks = (args.k64 + 3) / 4;            // stages of 256 elements
    const int c_begin = static_cast<int>(static_cast<int64_t>(chunks) * rank / C);
    const int c_end = static_cast<int>(static_cast<int64_t>(chunks) * (rank + 1) / C);
    const int n_main = c_end - c_begin;
    const int n_iters = n_main + (rank == C - 1 ? args.ext.steps : 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], L::kQuant ? 1 + quant_warps(args.T) : 1);      // the copies, and the quantizing warps
            mbar_init(&empty[s], 1);
        }
        mbar_init(accf, 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, L::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();

    // MMAs (K = 64) and scale tiles of main stage `it`
    auto mmas_of = [&](int it) { return min(4, args.k64 - (c_begin + it) * 4); };
    // bytes of the scale tiles of stage `c` from row tile `rt` of `rows` rows on
    auto scales_at = [&](int rt, int c, uint32_t bytes, int rows) {
        const int64_t at = (static_cast<int64_t>(rt) * args.col_tiles + 2 * c) * kMxTileBytes;
        return dcheck(at + bytes <= static_cast<int64_t>((rows + 127) / 128) * args.col_tiles * kMxTileBytes, args.err) ? at : 0;
    };

    if (warp == 0) {
        auto load_w = [&](int it, int s) {
            const int c = c_begin + it;
            const uint32_t sf = static_cast<uint32_t>((mmas_of(it) + 1) / 2) * kMxTileBytes;
            mbar_arrive_expect_tx(&full[s], L::kQuant ? L::kA + sf : L::kA + L::kB + 2 * sf);
            tma_load_2d(sA + s * L::kA, &tmW, &full[s], c * 128, n0);
            bulk_load(sSa + s * L::kSf, args.w_scales + scales_at(tile, c, sf, args.d_out), sf, &full[s]);
        };
        auto load_x = [&](int it, int s) {
            if (L::kQuant) return;
            const int c = c_begin + it;
            const uint32_t sf = static_cast<uint32_t>((mmas_of(it) + 1) / 2) * kMxTileBytes;
            tma_load_2d(sB + s * L::kB, &tmX, &full[s], c * 128, t0);
            bulk_load(sSb + s * L::kSf, args.x_scales + scales_at(t0 >> 7, c, sf, args.T), sf, &full[s]);
        };
        const int ahead = min(S, n_main);
        if (elect_one())
            for (int it = 0; it < ahead; ++it) load_w(it, it);
        __syncwarp();
        if (!L::kQuant) {
            griddep_wait();
            if (elect_one())
                for (int it = 0; it < ahead; ++it) load_x(it, it);
            __syncwarp();
        }
        int issued = ahead;
        for (int it = ahead, s = ahead % S, ph = ahead / S; it < n_iters; ++it) {
            if (!mbar_wait_uniform(&empty[s], ph ^ 1, abort, args.wait_ns)) {
                set_error(args.err, kErrTimeout);
                *abort = 1;
                break;
            }
            if (L::kQuant && it == n_main) griddep_wait();
            if (elect_one()) {
                if (it < n_main) {
                    load_w(it, s);
                    load_x(it, s);
                } else {
                    const int e = it - n_main;
                    mbar_arrive_expect_tx(&full[s], L::kA + L::kB);
                    tma_load_2d(sA + s * L::kA, &tmBx, &full[s], args.ext.c_col(e), n0);
                    tma_load_2d(sB + s * L::kB, &tmUx, &full[s], e * 64, t0);
                }
            }
            __syncwarp();
            issued = it + 1;
            if (++s == S) s = 0, ph ^= 1;
        }
        if (*abort)
            for (int it = max(0, issued - S); it < issued; ++it)
                mbar_wait(&full[it % S], (it / S) & 1, nullptr, args.wait_ns);
    } else if (warp == 1) {
        const uint32_t idesc_x = make_idesc_bf16(128, NT, false, false);
        const uint32_t idesc0 = make_idesc_mxf4(128, NT, 0, 0), idesc2 = make_idesc_mxf4(128, NT, 2, 2);
        const uint64_t a_desc = make_sw128_desc(smem_u32(sA), 16, 1024), b_desc = make_sw128_desc(smem_u32(sB), 16, 1024);
        const uint64_t sa_desc = make_scale_desc(smem_u32(sSa)), sb_desc = make_scale_desc(smem_u32(sSb));
        // sets of scale columns are used in turn: that of step it - kSets is free once its MMAs are done
        // (a ring of no more stages than sets has waited for that already)
        int s2 = 0, ph2 = 0;
        for (int it = 0, s = 0, ph = 0; it < n_iters; ++it) {
            bool ok = mbar_wait_uniform(&full[s], ph, abort, args.wait_ns);
            if (ok && S > L::kSets && it >= L::kSets) {
                ok = mbar_wait_uniform(&empty[s2], ph2, abort, args.wait_ns);
                if (++s2 == S) s2 = 0, ph2 ^= 1;
            }
            if (!ok) {
                set_error(args.err, kErrTimeout);
                *abort = 1;
                break;
            }
            tc_fence_after();
            const uint64_t ad = a_desc + static_cast<uint32_t>(s * (L::kA >> 4));
            const uint64_t bd = b_desc + static_cast<uint32_t>(s * (L::kB >> 4));
            if (it < n_main) {
                const uint32_t sfa = tmem + L::kAcc + (it % L::kSets) * 16, sfb = sfa + 8;
                const uint64_t sad = sa_desc + static_cast<uint32_t>(s * (L::kSf >> 4));
                const uint64_t sbd = sb_desc + static_cast<uint32_t>(s * (L::kSf >> 4));
                const int nk = mmas_of(it);
                if (elect_one()) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (2 * h < nk) {
                            tmem_cp_scales<1>(sfa + 4 * h, sad + h * (kMxTileBytes >> 4));
                            tmem_cp_scales<1>(sfb + 4 * h, sbd + h * (kMxTileBytes >> 4));
                        }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < nk)
                            umma_mxf4_ss<1>(tmem, ad + 2 * k, bd + 2 * k, (k & 1) ? idesc2 : idesc0, sfa + 4 * (k >> 1),
                                            sfb + 4 * (k >> 1), (it > 0 || k > 0) ? 1u : 0u);
                    umma_commit(&empty[s]);
                }
            } else {
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = args.ext.c16(it - n_main, k);
                        if (c >= 0) umma_bf16_ss(tmem, ad + 2 * c, bd + 2 * k, idesc_x, (it > 0 || k > 0) ? 1u : 0u);
                    }
                    umma_commit(&empty[s]);
                }
            }
            __syncwarp();
            if (++s == S) s = 0, ph ^= 1;
        }
        if (elect_one()) umma_commit(accf);
    } else if constexpr (L::kQuant) {
        // Groups of just the warps whose rows there are (four rows each), every group its own stages in
        // turn: quantizing one takes a warp longer (0.6 us) than the stream brings one.  No more groups
        // than ring stages: the wait for a slot tells its last two uses apart, so a group may ask for it
        // only after having seen the use before the last one end.  Token `row`, block `blk` of a
        // stage's 256 columns; rows past T are left as they are (they reach the output columns past T only).
        const int G = quant_warps(args.T), groups = min(L::kQuantGroups, L::kQuantWarps / G), qw = warp - 2;
        const int row = qw % G * 4 + (lane >> 3), blk = lane & 7;
        const bool in = row < args.T;
        const __nv_bfloat16* src = args.X + row * args.d_in + static_cast<int64_t>(c_begin) * 256 + blk * 32;
        auto fetch = [&](int it, Raw8<__nv_bfloat16> (&raw)[4]) {
            const bool there = in && it < n_main && static_cast<int64_t>(c_begin + it) * 256 + blk * 32 < args.d_in;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (there) raw[c].load(src + static_cast<int64_t>(it) * 256 + c * 8);
                else raw[c].zero();
            }
        };
        Raw8<__nv_bfloat16> nxt[4];
        int it = qw / G < groups ? qw / G : n_iters, s = it, ph = 0;
        fetch(it, nxt);
        for (; it < n_iters; it += groups, s += groups) {
            while (s >= S) s -= S, ph ^= 1;
            Raw8<__nv_bfloat16> cur[4] = {nxt[0], nxt[1], nxt[2], nxt[3]};
            fetch(it + groups, nxt);
            if (!mbar_wait_warp(&empty[s], ph ^ 1, abort, args.wait_ns)) {
                set_error(args.err, kErrTimeout);
                *abort = 1;
                break;
            }
            if (it < n_main && in) {
                uint32_t e, q[4];
                mxfp4_block32(cur, e, q);
                *reinterpret_cast<uint4*>(sB + s * L::kB + row * 128 + ((blk ^ (row & 7)) << 4)) =
                    make_uint4(q[0], q[1], q[2], q[3]);
                sSb[s * L::kSf + (blk >> 2) * kMxTileBytes + row * 16 + (blk & 3)] = static_cast<uint8_t>(e);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
        }
    }
    __syncwarp();

    // ------------------------------------------------------------ join the ranks, store
    const int q = warp & 3;                            // tensor-memory lane quarter of this warp
    const int row = n0 + q * 32 + lane;                // weight row = output column
    const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int t_end = min(NT, args.T - t0);
    const bool store = warp >= 2 && warp < 6;          // one warp for each quarter
    if (store) {
        if (!mbar_wait_warp(accf, 0, nullptr, args.wait_ns)) {
            set_error(args.err, kErrTimeout);
            *abort = 1;
        }
        tc_fence_after();
    }
    if (C == 1) {
        griddep_wait();          // earlier kernels of the stream may still read or write H
        if (store && !*abort) {
#pragma unroll 1
            for (int c0 = 0; c0 < t_end; c0 += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(tbase + c0, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (row < args.d_out && c0 + j < t_end)
                        args.out[static_cast<int64_t>(t0 + c0 + j) * args.d_out + row] =
                            __float2bfloat16_rn(__uint_as_float(r[j]));
            }
        }
    } else {
        // rank o sums the weight rows [o R, (o + 1) R): every rank sends it its partials of them,
        // red[source rank][token][row], once every rank's MMAs are done with the ring underneath; a
        // warp's 32 rows go as one line
        const int R = 128 / C;
        cluster_barrier();
        if (store && !*abort) {
            const int lr = q * 32 + lane;
            const uint32_t dst = mapa_shared(smem_u32(red + rank * NT * R + lr % R), static_cast<uint32_t>(lr / R));
#pragma unroll 1
            for (int c0 = 0; c0 < t_end; c0 += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(tbase + c0, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c0 + j < t_end)
                        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(dst + (c0 + j) * R * 4), "r"(r[j]) : "memory");
            }
        }
        cluster_barrier();
        griddep_wait();
        if (!*abort) {
            if (C == 2) mx_join<2, NT, L::kThreads>(red, t_end, n0 + 64 * rank, t0, args);
            else mx_join<4, NT, L::kThreads>(red, t_end, n0 + 32 * rank, t0, args);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmem);
    }
}

// ------------------------------------------------------------------ persistent 2-SM kernel

// 2-D tiled load into this CTA's shared memory that completes on a barrier of either CTA of the
// pair (bar: cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int32_t x,
                                                 int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

// Limit, after a wait has run out, of that for the copies still in flight (ns).
constexpr uint64_t kLandNs = 1000000;

struct PairGemmArgs {
    int M, N;                 // output rows (tokens) and columns
    int k_steps;              // main stages: 256 MXFP4 or 64 bf16 elements of K
    int k_mma_last;           // MMAs of the last main stage (1..4)
    ExtSteps ext;             // the adapter's K stages
    int m_tiles, n_tiles;     // 256 x BN tiles
    int a_sf_tiles, b_sf_tiles;   // MXFP4: scale tiles per row of tiles (both operands share d_in)
    int split;                // ways the tail tiles are split along K (1: not)
    int tail_tiles;           // trailing tiles that are split
    float* part;              // [tail_tiles][2 ranks][4 warps][split][BN * 8 float4] fp32 partials
    int* cnt;                 // [tail_tiles][2 ranks][4 warps] tickets, zero at launch
    __nv_bfloat16* out;
    int64_t ld_out;
    int* err;
    uint64_t wait_ns;
};

__device__ __forceinline__ uint4 shfl_xor4(const uint4& a, int m) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, a.x, m), __shfl_xor_sync(0xffffffffu, a.y, m),
                      __shfl_xor_sync(0xffffffffu, a.z, m), __shfl_xor_sync(0xffffffffu, a.w, m));
}
template <int M>
__device__ __forceinline__ void quad_swap(uint4& a, uint4& b, bool hi) {
    const uint4 x = shfl_xor4(hi ? a : b, M);
    a = hi ? x : a;
    b = hi ? b : x;
}
// v[g] of lane 4 i + p becomes v[p] of lane 4 i + g.
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4], int lane) {
    quad_swap<1>(v[0], v[1], lane & 1);
    quad_swap<1>(v[2], v[3], lane & 1);
    quad_swap<2>(v[0], v[2], lane & 2);
    quad_swap<2>(v[1], v[3], lane & 2);
}

// r[e] of lane l becomes r[l] of lane e.
template <int M>
__device__ __forceinline__ void warp_swap(uint32_t (&r)[32], int lane) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (!(e & M)) {
            const uint32_t x = __shfl_xor_sync(0xffffffffu, (lane & M) ? r[e] : r[e + M], M);
            if (lane & M) r[e] = x;
            else r[e + M] = x;
        }
}
__device__ __forceinline__ void warp_transpose(uint32_t (&r)[32], int lane) {
    warp_swap<1>(r, lane);
    warp_swap<2>(r, lane);
    warp_swap<4>(r, lane);
    warp_swap<8>(r, lane);
    warp_swap<16>(r, lane);
}

// BN: columns of a tile, 256, or for bf16 also 128.
template <bool MX, int BN>
struct PairGemmSmem {
    static constexpr int kA = 128 * 128;               // this CTA's A half: 128 rows of 128 bytes
    static constexpr int kB = BN / 2 * 128;            // its B half
    static constexpr int kSfA = MX ? 1024 : 0;         // scales of its 128 A rows
    static constexpr int kSfB = MX ? 2048 : 0;         // scales of all 256 B rows
    static constexpr int kStage = kA + kB + kSfA + kSfB;
    static constexpr int kStages = MX ? 6 : BN == 256 ? 7 : 9;
    static constexpr int kTotal = 1024 + kStages * kStage + 512;
    static constexpr int kThreads = 192;
    // Accumulator columns of the second buffer.  MXFP4 keeps the scales in columns 448..511, so its
    // two accumulators share 64 columns, which the epilogue reads first.
    static constexpr int kAcc1 = MX ? 192 : BN;
    static constexpr int kSfCol = 448;
    static_assert(kTotal <= 232448, "shared memory budget");
};

// MX:  out[T, d_out] = X4 W4^T + sU B^T   (kind::mxf4, all operands K-major)
// !MX: out[T, d_in]  = dH W + sG A        (kind::f16, W bf16 [K, N] and A [r, N] consumed MN-major)
//
// A pair of CTAs computes 256 x 256 tiles with cta_group::2 MMAs of M = N = 256 issued by the leader;
// each CTA loads half of both operands (and, for MXFP4, the scales of its own A rows and of all B
// rows).  Both CTAs' copies complete on the leader's full[s], so one wait covers the pair; a stage
// is released to both by the MMAs' commit.  Persistent: pair p takes tiles p, p + pairs, ...; the tiles
// of an incomplete last wave (all of them when there are fewer tiles than pairs) may be split along K
// over `split` pairs each (bf16 only: an MXFP4 tile is over before a join would be).  Every epilogue
// warp of a split tile writes its fp32 partial and takes a ticket; the last adds all partials in K
// order, so the result does not depend on which is last, and no CTA waits for another.
// Bound by the tensor cores (256 x 256 x 256 MXFP4 or x 64 bf16 in 512 cycles) where K is long and the
// waves are full: 8192 tokens of 11008 x 4096 in 458 to 484 us (bf16, 1.6 PFLOP/s, tensor pipe 95 % busy).  4096^3 takes
// 82 to 94 us in bf16 (76 % busy) and 33 to 36 in MXFP4 (3.9 PFLOP/s, 47 %): 3.46 waves in 4, 620 cycles a stage
// (the 35 KB of its loads come at 55 bytes a cycle), and between two tiles the time to read the columns
// that their accumulators share.
template <bool MX, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairGemmSmem<MX, BN>::kThreads, 1)
    k_pair_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmSa, const __grid_constant__ CUtensorMap tmSb,
                const __grid_constant__ CUtensorMap tmAx, const __grid_constant__ CUtensorMap tmBx,
                const PairGemmArgs args) {
    using L = PairGemmSmem<MX, BN>;
    constexpr int S = L::kStages;
    static_assert(!MX || BN == 256, "MXFP4 tiles are 256 wide");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + S * L::kA;
    uint8_t* sSa = sB + S * L::kB;
    uint8_t* sSb = sSa + S * L::kSfA;
    uint64_t* full = reinterpret_cast<uint64_t*>(sSb + S * L::kSfB);   // leader: both halves landed
    uint64_t* empty = full + S;             // both: stage consumed
    uint64_t* accf = empty + S;             // [2] both: accumulator complete
    uint64_t* acc_free = accf + 2;          // [2] leader: accumulator (MX: its shared columns) read
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_free + 2);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int n_tiles_total = args.m_tiles * args.n_tiles;
    const int iters_per_tile = args.k_steps + args.ext.steps;
    const int tail_base = n_tiles_total - args.tail_tiles;
    // this pair's units: whole tiles pair, pair + npairs, ... < tail_base, then at most one part of a
    // tail tile (part p: main stages [p k / split, (p + 1) k / split), the last part also the adapter's)
    const int n_full = pair < tail_base ? (tail_base - pair + npairs - 1) / npairs : 0;
    const bool has_part = pair < args.tail_tiles * args.split;
    const int part_tile = has_part ? pair / args.split : 0, part = has_part ? pair % args.split : 0;
    const int n_units = n_full + (has_part ? 1 : 0);
    auto unit = [&](int u, int& tile, int& k0, int& k1) {
        if (u < n_full) {
            tile = pair + u * npairs;
            k0 = 0;
            k1 = iters_per_tile;
        } else {
            tile = tail_base + part_tile;
            k0 = args.k_steps * part / args.split;
            k1 = part == args.split - 1 ? iters_per_tile : args.k_steps * (part + 1) / args.split;
        }
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
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
        tma_prefetch_desc(&tmAx);
        tma_prefetch_desc(&tmBx);
        if (MX) {
            tma_prefetch_desc(&tmSa);
            tma_prefetch_desc(&tmSb);
        }
    }
    if (warp == 1) {
        tmem_alloc_2sm(tmem_slot, 512);
        tmem_relinquish_2sm();
    }
    tc_fence_before();
    cluster_barrier();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_enter();

    auto fail = [&]() {
        set_error(args.err, kErrTimeout);
        *abort = 1;
    };

    if (warp == 0) {
        const uint32_t full_leader = mapa_shared(smem_u32(&full[0]), 0);
        int s = 0, ph = 0, issued = 0;
        bool ok = true;
        for (int u = 0; ok && u < n_units; ++u) {
            int tile, k0, k1;
            unit(u, tile, k0, k1);
            const int m0 = (tile % args.m_tiles) * 256 + static_cast<int>(rank) * 128;
            const int nt = tile / args.m_tiles;
            const int n0 = nt * BN + static_cast<int>(rank) * (BN / 2);
            for (int it = k0; it < k1; ++it) {
                ok = mbar_wait_uniform(&empty[s], ph ^ 1, abort, args.wait_ns);
                if (!ok) break;
                const uint32_t bar = full_leader + static_cast<uint32_t>(s * 8);
                uint8_t* a = sA + s * L::kA;
                uint8_t* b = sB + s * L::kB;
                if (elect_one()) {
                    if (it < args.k_steps) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * L::kStage);
                        if (MX) {
                            tma_load_2d_pair(a, &tmA, bar, it * 128, m0);
                            tma_load_2d_pair(b, &tmB, bar, it * 128, n0);
                            tma_load_2d_pair(sSa + s * L::kSfA, &tmSa, bar, 0, (m0 >> 7) * args.a_sf_tiles + 2 * it);
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                tma_load_2d_pair(sSb + s * L::kSfB + h * 1024, &tmSb, bar, 0,
                                                 (2 * nt + h) * args.b_sf_tiles + 2 * it);
                        } else {
                            tma_load_2d_pair(a, &tmA, bar, it * 64, m0);
                            tma_load_2d_pair(b, &tmB, bar, n0, it * 64);
                            if (BN == 256) tma_load_2d_pair(b + 8192, &tmB, bar, n0 + 64, it * 64);
                        }
                    } else {
                        const int e = it - args.k_steps, c = args.ext.c_col(e);
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (L::kA + L::kB));
                        tma_load_2d_pair(a, &tmAx, bar, e * 64, m0);
                        if (MX) {
                            tma_load_2d_pair(b, &tmBx, bar, c, n0);
                        } else {
                            tma_load_2d_pair(b, &tmBx, bar, n0, c);
                            if (BN == 256) tma_load_2d_pair(b + 8192, &tmBx, bar, n0 + 64, c);
                        }
                    }
                }
                __syncwarp();
                ++issued;
                if (++s == S) s = 0, ph ^= 1;
            }
        }
        if (!ok) fail();
        // given up: the copies in flight land before the teardown lets shared memory go.  They complete on
        // the leader's barriers, its peer's too; a stage whose other half was never issued ends the wait by its
        // limit, far above what a copy takes
        if (rank == 0 && *abort)
            for (int it = max(0, issued - S); it < issued; ++it) mbar_wait(&full[it % S], (it / S) & 1, nullptr, kLandNs);
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t idesc = make_idesc_bf16(256, BN, false, !MX);
            const uint32_t idesc0 = make_idesc_mxf4(256, 256, 0, 0), idesc2 = make_idesc_mxf4(256, 256, 2, 2);
            const uint64_t a_desc = make_sw128_desc(smem_u32(sA), 16, 1024);
            const uint64_t b_desc = make_sw128_desc(smem_u32(sB), MX ? 16 : 8192, 1024);
            const uint64_t sa_desc = make_scale_desc(smem_u32(sSa)), sb_desc = make_scale_desc(smem_u32(sSb));
            constexpr uint32_t kBStep = MX ? 2 : 2048 >> 4;
            int git = 0, s = 0, ph = 0, s2 = 0, ph2 = 0;
            bool ok = true;
            for (int u = 0; ok && u < n_units; ++u) {
                int tile, k0, k1;
                unit(u, tile, k0, k1);
                // MX: the shared columns of unit u - 1 have been read; else: all of unit u - 2
                const int prev = u - (MX ? 1 : 2);
                if (prev >= 0) ok = mbar_wait_uniform(&acc_free[prev & 1], (prev >> 1) & 1, abort, args.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>((u & 1) * L::kAcc1);
                for (int it = k0; it < k1; ++it, ++git) {
                    ok = mbar_wait_uniform(&full[s], ph, abort, args.wait_ns);
                    // two sets of scale columns in turn: those of stage git - 2 are free once its MMAs are done
                    if (MX && ok && git >= 2) {
                        ok = mbar_wait_uniform(&empty[s2], ph2, abort, args.wait_ns);
                        if (++s2 == S) s2 = 0, ph2 ^= 1;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = a_desc + static_cast<uint32_t>(s * (L::kA >> 4));
                    const uint64_t bd = b_desc + static_cast<uint32_t>(s * (L::kB >> 4));
                    const bool first = it == k0;
                    if (MX && it < args.k_steps) {
                        const uint32_t sfa = tmem + L::kSfCol + (git & 1) * 24, sfb = sfa + 8;
                        const uint64_t sad = sa_desc + static_cast<uint32_t>(s * (L::kSfA >> 4));
                        const uint64_t sbd = sb_desc + static_cast<uint32_t>(s * (L::kSfB >> 4));
                        const int nk = it == args.k_steps - 1 ? args.k_mma_last : 4;
                        if (elect_one()) {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (2 * h < nk) {
                                    tmem_cp_scales<2>(sfa + 4 * h, sad + h * 32);
                                    tmem_cp_scales<2>(sfb + 8 * h, sbd + h * 32);
                                    tmem_cp_scales<2>(sfb + 8 * h + 4, sbd + 64 + h * 32);
                                }
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < nk)
                                    umma_mxf4_ss<2>(d, ad + 2 * k, bd + 2 * k, (k & 1) ? idesc2 : idesc0,
                                                    sfa + 4 * (k >> 1), sfb + 8 * (k >> 1), (!first || k > 0) ? 1u : 0u);
                            umma_commit_2sm_both(&empty[s]);
                        }
                    } else if (it < args.k_steps) {
                        const int nk = it == args.k_steps - 1 ? args.k_mma_last : 4;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < nk)
                                    umma_bf16_ss_2sm(d, ad + 2 * k, bd + kBStep * k, idesc, (!first || k > 0) ? 1u : 0u);
                            umma_commit_2sm_both(&empty[s]);
                        }
                    } else {
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int c = args.ext.c16(it - args.k_steps, k);
                                if (c >= 0)
                                    umma_bf16_ss_2sm(d, ad + 2 * k, bd + kBStep * c, idesc, (!first || k > 0) ? 1u : 0u);
                            }
                            umma_commit_2sm_both(&empty[s]);
                        }
                    }
                    __syncwarp();
                    if (++s == S) s = 0, ph ^= 1;
                }
                if (ok && elect_one()) umma_commit_2sm_both(&accf[u & 1]);
                __syncwarp();
            }
            if (!ok) fail();
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3;
        const uint32_t free_leader = mapa_shared(smem_u32(&acc_free[0]), 0);
        const bool vec_rows = !MX || (args.ld_out & 7) == 0;
        for (int u = 0; u < n_units; ++u) {
            int tile, k0, k1;
            unit(u, tile, k0, k1);
            const int buf = u & 1;
            if (!mbar_wait_warp(&accf[buf], (u >> 1) & 1, abort, args.wait_ns)) {
                fail();
                break;
            }
            tc_fence_after();
            const int64_t grow = static_cast<int64_t>(tile % args.m_tiles) * 256 + rank * 128 + q * 32 + lane;
            const int gc0 = (tile / args.m_tiles) * BN;
            const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * L::kAcc1;
            const bool split = !MX && u >= n_full && args.split > 1;
            bool last = true;
            const float4* parts = nullptr;
            if (split) {
                const int64_t slot = (static_cast<int64_t>(part_tile) * 2 + rank) * 4 + q;
                parts = reinterpret_cast<const float4*>(args.part) + slot * args.split * (BN * 8);
                float4* mine = const_cast<float4*>(parts) + part * (BN * 8);
#pragma unroll 1
                for (int c = 0; c < BN / 32; ++c) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tbase + c * 32, r);
                    tmem_ld_wait();
                    if (grow < args.M && dcheck(part_tile < args.tail_tiles && part < args.split, args.err)) {
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            mine[g2_part_idx(c, g, lane)] =
                                make_float4(__uint_as_float(r[4 * g]), __uint_as_float(r[4 * g + 1]),
                                            __uint_as_float(r[4 * g + 2]), __uint_as_float(r[4 * g + 3]));
                    }
                }
                __threadfence();
                __syncwarp();
                int ticket = 0;
                if (lane == 0) ticket = atomicAdd(args.cnt + slot, 1);
                last = __shfl_sync(0xffffffffu, ticket, 0) == args.split - 1;
                if (last) __threadfence();
            }
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_async_payload(free_leader + static_cast<uint32_t>(buf * 8));
            };
            // 32 columns of this warp's 32 rows.  Whole ones change hands among four lanes first, so that a store
            // covers 64 bytes of eight rows, not 16 of 32 (the last tile's stores have nothing beside them; 4096
            // tokens of 11008 x 4096 89.2 us against 91.8, of 4096 x 4096 backward 121.4 against 122.6).
            auto store = [&](int c, const uint32_t (&r)[32]) {
                const int gc = gc0 + c * 32;
                if (gc >= args.N) return;
                // (dX has whole rows of 64 columns)
                if (!MX || (vec_rows && gc + 32 <= args.N)) {
                    uint4 v[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        v[g].x = pack_bf16x2(__uint_as_float(r[8 * g + 0]), __uint_as_float(r[8 * g + 1]));
                        v[g].y = pack_bf16x2(__uint_as_float(r[8 * g + 2]), __uint_as_float(r[8 * g + 3]));
                        v[g].z = pack_bf16x2(__uint_as_float(r[8 * g + 4]), __uint_as_float(r[8 * g + 5]));
                        v[g].w = pack_bf16x2(__uint_as_float(r[8 * g + 6]), __uint_as_float(r[8 * g + 7]));
                    }
                    quad_transpose(v, lane);
                    const int p = lane & 3;
                    const int64_t row0 = grow - p;
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        if (row0 + g < args.M) *reinterpret_cast<uint4*>(args.out + (row0 + g) * args.ld_out + gc + 8 * p) = v[g];
                    return;
                }
                if constexpr (MX) {
                    // rows that are no whole 16-byte units, or end here: one column per lane, row by row (1024 tokens
                    // of 1001 x 2048 24.7 us, as one row per lane 49.4)
                    uint32_t t[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) t[e] = r[e];
                    warp_transpose(t, lane);
                    const int64_t row0 = grow - lane;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (row0 + e < args.M && gc + lane < args.N)
                            args.out[(row0 + e) * args.ld_out + gc + lane] = __float2bfloat16_rn(__uint_as_float(t[e]));
                }
            };
            if constexpr (MX) {
                // the 64 columns that the other accumulator shares (the last of buffer 0, the first of
                // buffer 1) are read first, and the next tile's MMAs released before anything is stored
                const int c0 = buf == 0 ? 6 : 0;
                uint32_t r0[32], r1[32];
                tmem_ld_32x32b_x32(tbase + c0 * 32, r0);
                tmem_ld_32x32b_x32(tbase + c0 * 32 + 32, r1);
                tmem_ld_wait();
                release();
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    const int c = (c0 + i) & 7;
                    if (i >= 2) {
                        tmem_ld_32x32b_x32(tbase + c * 32, r0);
                        tmem_ld_wait();
                    }
                    store(c, r0);
                    if (i == 0) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) r0[e] = r1[e];
                    }
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < BN / 32; ++c) {
                    uint32_t r[32];
                    if (split && last) {
                        // all other parts' values of the chunk in flight at once, added in K order whichever
                        // part is last
                        float4 o[kPairMaxSplit][8];
#pragma unroll
                        for (int p = 0; p < kPairMaxSplit; ++p)
                            if (p < args.split && p != part && grow < args.M)
#pragma unroll
                                for (int g = 0; g < 8; ++g) o[p][g] = __ldcg(parts + p * (BN * 8) + g2_part_idx(c, g, lane));
                        tmem_ld_32x32b_x32(tbase + c * 32, r);
                        tmem_ld_wait();
                        float4 v[8];
#pragma unroll
                        for (int p = 0; p < kPairMaxSplit; ++p)
                            if (p < args.split)
#pragma unroll
                                for (int g = 0; g < 8; ++g) {
                                    const float4 x = p == part ? make_float4(__uint_as_float(r[4 * g]), __uint_as_float(r[4 * g + 1]),
                                                                             __uint_as_float(r[4 * g + 2]), __uint_as_float(r[4 * g + 3]))
                                                               : o[p][g];
                                    v[g] = p == 0 ? x : make_float4(v[g].x + x.x, v[g].y + x.y, v[g].z + x.z, v[g].w + x.w);
                                }
#pragma unroll
                        for (int g = 0; g < 8; ++g) {
                            r[4 * g] = __float_as_uint(v[g].x);
                            r[4 * g + 1] = __float_as_uint(v[g].y);
                            r[4 * g + 2] = __float_as_uint(v[g].z);
                            r[4 * g + 3] = __float_as_uint(v[g].w);
                        }
                    } else if (last) {
                        tmem_ld_32x32b_x32(tbase + c * 32, r);
                        tmem_ld_wait();
                    }
                    if (c == BN / 32 - 1) release();
                    if (last) store(c, r);
                }
            }
        }
    }

    __syncwarp();
    if (*abort) __nanosleep(100000);   // (copies of a peer that ran ahead of the leader)
    tc_fence_before();
    cluster_barrier();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_2sm(tmem, 512);
    }
}

}  // namespace qlora
