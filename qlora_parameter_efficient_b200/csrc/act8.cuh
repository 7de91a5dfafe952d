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
#include "nf4.cuh"
#include "ring.cuh"

namespace qlora {

// 2^(e - 133) as fp32: the value of one integer step; exact (subnormal for e < 7), NaN for 255.
__device__ __forceinline__ float act8_step(uint32_t e) {
    return __uint_as_float(e == 255u ? 0x7FFFFFFFu : (e >= 7u ? (e - 6u) << 23 : 1u << (e + 16u)));
}

// Four lanes per block of 32, eight elements per lane, kAct8Unroll chunks of 256 lanes per CTA whose
// loads are issued together.  n8 (elements / 8) is a multiple of 8, so a block is never split.
// 4096 x 4096 bf16 in 11.7 us (51 MB, 4.3 TB/s, two thirds of what a copy gets; the decoder below, with the
// same loads and stores the other way round, 6.3): what is left is its arithmetic, two products, two clamps and an
// addition per element.
constexpr int kAct8Unroll = 4;
template <typename T>
__global__ void __launch_bounds__(256) k_act8_quantize(const T* __restrict__ X, int64_t n8,
                                                       int8_t* __restrict__ q, uint8_t* __restrict__ scales) {
    griddep_enter();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * kAct8Unroll) + threadIdx.x;
    Raw8<T> raw[kAct8Unroll];
#pragma unroll
    for (int u = 0; u < kAct8Unroll; ++u) {
        if (i0 + u * 256 < n8) raw[u].load(X + (i0 + u * 256) * 8);
        else raw[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kAct8Unroll; ++u) {
        const int64_t i = i0 + u * 256;
        float x[8];
        const uint32_t e = quad_max(raw[u].values(x)) >> 23;
        // x 2^(133 - e) in two exact steps (2^133 is no fp32 value)
        const uint32_t ec = max(e, 6u);
        const float f = __uint_as_float((260u - ec) << 23);
        const float g = static_cast<float>(1u << (ec - e));
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // rounded by adding 1.5 2^23 (to nearest even, the integer in the low bits)
            const float y = fminf(fmaxf(__fmul_rn(__fmul_rn(x[k], f), g), -127.f), 127.f) + 12582912.f;
            w[k >> 2] |= (__float_as_uint(y) & 255u) << (8 * (k & 3));
        }
        if (i < n8) {
            reinterpret_cast<uint2*>(q)[i] = e == 255u ? make_uint2(0, 0) : make_uint2(w[0], w[1]);
            if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(e);
        }
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

// The same split; 4096 x 4096 to bf16 in 8.1 us (51 MB, 6.3 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) k_act8_dequant(const int8_t* __restrict__ q,
                                                      const uint8_t* __restrict__ scales, int64_t n8,
                                                      T* __restrict__ out) {
    griddep_enter();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * kAct8Unroll) + threadIdx.x;
    uint2 v[kAct8Unroll];
    uint32_t e[kAct8Unroll];
#pragma unroll
    for (int u = 0; u < kAct8Unroll; ++u) {
        const int64_t i = i0 + u * 256;
        v[u] = make_uint2(0, 0);
        e[u] = 0;
        if (i < n8) {
            v[u] = __ldg(reinterpret_cast<const uint2*>(q) + i);
            e[u] = __ldg(scales + (i >> 2));
        }
    }
#pragma unroll
    for (int u = 0; u < kAct8Unroll; ++u) {
        const int64_t i = i0 + u * 256;
        if (i >= n8) break;
        const float s = act8_step(e[u]);
        if constexpr (sizeof(T) == 4) {
            float a[4], b[4];
            int8x4_to_f32(v[u].x, a);
            int8x4_to_f32(v[u].y, b);
            float4* o = reinterpret_cast<float4*>(out) + 2 * i;
            o[0] = make_float4(a[0] * s, a[1] * s, a[2] * s, a[3] * s);
            o[1] = make_float4(b[0] * s, b[1] * s, b[2] * s, b[3] * s);
        } else {
            reinterpret_cast<uint4*>(out)[i] = act8_decode8(v[u].x, v[u].y, s);
        }
    }
}

// ------------------------------------------------------------------ adapter products

// A matrix of fp32 values [T, r] as a tensor-core operand: three bf16 terms per value, whose sum is the
// value (8 significant bits each), as column groups of one matrix.  Up to rank 64 the groups are
// `stride` = the rank rounded up to 16 apart, so that one MMA takes all three (N = 3 stride, each
// group with accumulator columns of its own); above, 128 apart, one MMA each into the same columns.
struct ActTriple {
    int stride, ld;
};
__host__ __device__ __forceinline__ ActTriple act_triple(int r) {
    ActTriple t;
    t.stride = r <= 64 ? (r + 15) & ~15 : 128;
    t.ld = (3 * t.stride + 63) & ~63;
    return t;
}

// The K steps of 64 by which a layer's product F C^T takes its adapter term: F[., r] is s U or s G and C[., r]
// is B or A.  F comes as the first two terms of its triple: rounded to one bf16 number it would cost
// 2^-8 of the adapter term, as much as the rounding of the result (errors of H and dX 2.15e-3 against the 1.66e-3
// of that alone, Frobenius norm); two carry 16 bits.  C is exact.  Up to rank 64 a step holds 64 of the
// 2 stride columns of F and all of C, and an MMA of 16 of F's columns takes those of C that belong to them:
// up to rank 32 one step as with one term.  Above, a step holds half a term and half of C.
struct ExtSteps {
    int steps;
    int n16;      // MMAs per term
    int wide;     // rank above 64
    // first of the columns of C that step e holds
    __host__ __device__ __forceinline__ int c_col(int e) const { return wide ? (e & 1) * 64 : 0; }
    // which 16 of them go with columns 16 k of F's tile; -1: no MMA
    __host__ __device__ __forceinline__ int c16(int e, int k) const {
        if (wide) return 4 * (e & 1) + k < n16 ? k : -1;
        const int g = 4 * e + k;
        return g < n16 ? g : g < 2 * n16 ? g - n16 : -1;
    }
};
__host__ __device__ __forceinline__ ExtSteps ext_steps_of(int r) {
    ExtSteps x;
    x.n16 = (r + 15) / 16;
    x.wide = r > 64;
    x.steps = x.wide ? 4 : (2 * x.n16 + 3) / 4;
    return x;
}
// F alone: [., ld], the two terms `stride` apart, columns past the rank up to 16 n16 of both 0.
__host__ __device__ __forceinline__ int ext_ld(int r) { return (2 * act_triple(r).stride + 63) & ~63; }

// Two bf16 terms of four values, the second of what the first leaves.  An infinite or NaN value is carried by
// the first alone (inf - inf would make it NaN); so for a triple.
__device__ __forceinline__ uint2 bf16_term(float (&x)[4]) {
    uint2 w;
    w.x = pack_bf16x2(x[0], x[1]);
    w.y = pack_bf16x2(x[2], x[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t h = e < 2 ? w.x : w.y;
        const float rest = x[e] - __uint_as_float((e & 1) ? h & 0xFFFF0000u : h << 16);
        x[e] = fabsf(rest) < __int_as_float(0x7F800000) ? rest : 0.f;
    }
    return w;
}

// What becomes of the sum D[M, N] of a product.
enum : int {
    kActTriple = 0,   // scale D as three bf16 terms (ActTriple layout)
    kActCols = 1,     // fp32 out[j, m] = scale D[m, j]  (dA)
    kActRows = 2,     // fp32 out[m, j] = scale D[m, j]  (dB)
    kActU = 3,        // scale D as two bf16 terms (row stride ext_ld) and bf16 out2[m, j] = D[m, j] (nullable)
    kActDx = 4        // bf16 out[j, m] = D[m, j]  (dX of few tokens)
};

// The products of a launch.  One kernel for all of them would be too long for the instruction cache (and
// measured 10 to 25% slower).
enum : int {
    kRoleU = 0,       // forward: U from bf16 X [T, d_in] (and the MXFP4 of X), kActU
    kRoleUG = 1,      // backward: G from dH, U from X or its checkpoint, kActTriple
    kRoleAB = 2,      // backward: dA from X or its checkpoint (kActCols), dB from dH (kActRows)
    kRoleDx = 3       // backward of few tokens: dX from the weight, kActDx
};

// How the A operand is stored; all but bf16 are decoded to it in shared memory.
enum : int {
    kOpBf16 = 0,
    kOpInt8 = 1,      // 8-bit checkpoint
    kOpMxfp4 = 2,     // the weight of a backward for few tokens, [K, M] (its rows are K)
    kOpNf4 = 3
};

// One product of a launch: D[M, N] = sum over K of A[M, K] B[N, K], B bf16 or a bf16 triple.
struct ActJob {
    int M, N;                // output rows (channels or tokens) and columns (the rank)
    int64_t K;               // contraction length
    int k_steps;             // ceil(K / 64)
    int op;                  // how A is stored
    int bmn;                 // kRoleUG: B is stored [K, N], else [N, K]
    int triple;              // B is an ActTriple (kRoleAB)
    const uint8_t* scales;   // E8M0 bytes (int8: row-major, MXFP4: tiled) or NF4's uint8 constants
    const float* c2;         // NF4's group constants
    int64_t ld_scales;       // scales per stored row (MXFP4: scale tiles)
    ExtSteps ext;            // kActDx: the adapter's K steps, taken by the last rank
    int mode;                // kRoleAB: kActCols or kActRows
    float scale;
    int accumulate;          // kActCols, kActRows: add to out
    void* out;
    __nv_bfloat16* out2;
    // Forward: A (bf16 [M, K]) is also quantized to MXFP4 on its way through shared memory (null: not)
    uint8_t *mx_codes, *mx_scales;
};
// Copy of a matrix whose rows are no whole 16-byte units to zero-padded rows.
struct PadCopy {
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    int64_t rows;
    int cols, ld, ctas;
    __device__ __forceinline__ void run(int cta) const {
        const int64_t n = rows * ld;
        for (int64_t i = static_cast<int64_t>(cta) * blockDim.x + threadIdx.x; i < n;
             i += static_cast<int64_t>(ctas) * blockDim.x) {
            const int64_t row = i / ld;
            const int col = static_cast<int>(i - row * ld);
            dst[i] = col < cols ? src[row * cols + col] : __float2bfloat16_rn(0.f);
        }
    }
};
struct ActGemmArgs {
    ActJob job[2];
    int tiles0, tiles;       // M tiles of job 0, of both
    int ranks;               // CTAs per cluster, K split over them
    // Done by the CTAs past the tiles (each range a multiple of ranks): a padded copy, and the MXFP4 of X
    // [qx_rows, qx_cols], one scale tile per CTA, where the products' own CTAs are too few for it
    PadCopy pad;
    int qx_ctas, qx_tiles;
    const __nv_bfloat16* qx;
    int64_t qx_rows, qx_cols;
    uint8_t *qx_codes, *qx_scales;
    int* err;
    uint64_t wait_ns;
};

// RPT: the padded rank, 64 or 128 (B tile rows).
template <int RPT>
struct ActGemmSmem {
    static constexpr int kA = 128 * 64 * 2;                     // bf16 operand tile
    static constexpr int kRaw = 128 * 64;                       // int8 tile
    static constexpr int kChunk = 64 * 64 * 2;                  // 64 columns (or rows) of the B tile
    static constexpr int kRing = 221184;
    static constexpr int kMaxStages = 6;
    static constexpr int kAcc = 4;                              // accumulator tiles, at most
    static constexpr int kTotal = 1024 + kRing + 512;
    // groups of eight decoding warps (one at rank > 64, whose drains need the registers)
    static constexpr int kGroups = RPT == 64 ? 2 : 1;
    static constexpr int kThreads = 32 * (2 + 8 * kGroups);
    static constexpr int kLdRed = RPT + 4;                      // floats per row of the joining buffer
    static_assert(kTotal <= 232448 && 128 * kLdRed * 4 <= kRing, "shared memory budget");
    static_assert(3 * (kA + kRaw + 3 * RPT / 64 * kChunk) <= kRing, "three stages at least");
    static_assert(kGroups <= 3, "no more groups than stages (ring_landed)");
};

// Warp 0: TMA; warp 1: MMA; warps 2..9 and, up to rank 64, 10..17: int8 decode or MXFP4 quantization, one
// 32-element block per thread and stage, the groups taking stages in turn (one group alone is
// bound by the latency of its own chain, 1100 cycles a stage); warps 2..9 also drain the accumulators.
// A cluster's ranks split K; their sums meet in shared memory, each rank adding and writing 128 / ranks
// rows in rank order, so no partial goes through memory.  Up to two products share a launch (U and G; dA
// and dB).
//
// Precision: the results are fp32 gradients.  (1) A value that was computed here (s G, a recomputed U)
// is given to the bf16 tensor cores as the three bf16 numbers that make up its 24 bits, so nothing is
// rounded off it.  (2) The tensor core's running fp32 sum is truncated at every MMA -- a bias that
// grows with the chain: 9e-6 of a gradient over 8192 tokens.  So the chain is cut into segments of
// 16 or 24 MMAs, whose sums warps 2..9 add up in registers, rounding to nearest, from two to four
// accumulator tiles in turn.
// A K step of 64 reads 8 KB of int8 (or 16 KB of bf16) from HBM and the B tiles from L2.  Bound by the
// decoding or quantizing of those in the CTA (about 0.6 us a step for one group of warps; DRAM at 21 to 26 % with
// 4096 tokens, 56 % for U and G of 8192) and, with few tiles, by latency.  With few tokens dX^T = W^T dH^T is such a product too (kActDx): M = d_in, N = tokens, the weight
// decoded once per CTA and split along d_out over the SMs.  An MMA of M = 128 takes about 75 cycles
// however small N is (it reads its A tile), hence one of N = 3 stride for a triple and not three.
// Measured out of HBM: U and G of 4096 tokens, 4096 x 4096, r = 16, from the checkpoint, 14 us (50 MB), dA and
// dB of the same 25 us; of 8192 tokens, 11008 x 4096, r = 64, 37 and 73 us (214 MB); U and X's MXFP4 of 200
// tokens, 8192 wide, 11.4 us, of 4096 tokens, 4096 wide, 17.7 us.
template <int RPT, int ROLE>
__global__ void __launch_bounds__(ActGemmSmem<RPT>::kThreads, 1)
    k_act_gemm(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmB0,
               const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmB1,
               const __grid_constant__ ActGemmArgs args) {      // (kActDx: tmA1, tmB1 are the adapter's)
    using L = ActGemmSmem<RPT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kRing);
    uint64_t* empty = full + L::kMaxStages;
    uint64_t* decoded = empty + L::kMaxStages;
    uint64_t* accf = decoded + L::kMaxStages;   // [kAcc] segment complete
    uint64_t* acc_free = accf + L::kAcc;        // [kAcc] segment drained (8 warp arrivals)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_free + L::kAcc);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int C = args.ranks;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tile = blockIdx.x / C;
    if (ROLE == kRoleU && tile >= args.tiles) {
        griddep_enter();
        const int b = static_cast<int>(blockIdx.x) - args.tiles * C;
        if (b >= args.qx_ctas) {
            args.pad.run(b - args.qx_ctas);
        } else if (b < args.qx_tiles) {
            const int64_t kts = mx_col_tiles(args.qx_cols);
            mxfp4_quantize_tile(args.qx, args.qx_rows, args.qx_cols, b / kts, b % kts, args.qx_codes, args.qx_scales,
                                smem_raw);
        }
        return;
    }
    const int ji = (ROLE == kRoleUG || ROLE == kRoleAB) && tile >= args.tiles0 ? 1 : 0;
    const ActJob& job = args.job[ji];
    const CUtensorMap* tmA = ji ? &tmA1 : &tmA0;
    const CUtensorMap* tmB = ji ? &tmB1 : &tmB0;
    const int tj = tile - (ji ? args.tiles0 : 0);
    const int m0 = tj * 128;
    const int N = job.N;
    const int op = job.op;
    const bool dec = ROLE == kRoleDx || (ROLE != kRoleU && op != kOpBf16);
    // A is stored [K, M] (its rows are K: tokens, weight rows) and consumed MN-major, else [M, K]
    constexpr bool amn = ROLE == kRoleAB || ROLE == kRoleDx;
    const bool bmn = ROLE == kRoleAB || (ROLE == kRoleUG && job.bmn);
    const bool quant = ROLE == kRoleU && job.mx_codes != nullptr;
    const int unit = quant ? 2 : 1;             // K steps a range is made of (quantizing: whole scale tiles)
    const int64_t units = (job.k_steps + unit - 1) / unit;
    const int k_begin = static_cast<int>(units * rank / C) * unit;
    const int n_main = min(job.k_steps, static_cast<int>(units * (rank + 1) / C) * unit) - k_begin;
    const int n_iters = n_main + (ROLE == kRoleDx && rank == C - 1 ? job.ext.steps : 0);
    const ActTriple tr = act_triple(job.N);
    const bool triple = ROLE == kRoleAB && job.triple;
    const int terms = RPT == 64 && triple ? 3 : 1;             // column groups of an accumulator tile
    const int groups = RPT == 128 && triple ? 3 : 1;           // MMAs per 16 of K
    const int n_mma = terms == 3 ? 3 * tr.stride : (N + 15) & ~15;
    const int chunks = triple ? tr.ld / 64 : RPT / 64;         // of the B tile
    const int acc_cols = terms == 3 ? tr.ld : RPT;
    const int NA = min(L::kAcc, 512 / acc_cols);               // accumulator tiles
    const int seg_len = groups == 3 ? 2 : 4;                   // K steps of 64 per accumulator segment
    const int n_seg = (n_iters + seg_len - 1) / seg_len;
    // ring: A tiles, B tiles, tiles as stored
    const int b_bytes = chunks * L::kChunk;
    const int raw_bytes = !dec ? 0 : ROLE == kRoleDx ? L::kRaw / 2 : L::kRaw;
    const int stage = L::kA + b_bytes + raw_bytes;
    const int S = min(L::kMaxStages, L::kRing / stage);
    uint8_t* sA = smem;
    uint8_t* sB = sA + S * L::kA;
    uint8_t* sR = sB + S * b_bytes;

    if (warp == 2) {
        if (lane < L::kMaxStages) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], quant ? 9 : 1);     // the MMAs, and the warps that quantize
            mbar_init(&decoded[lane], 8);
        }
        if (lane < L::kAcc) {
            mbar_init(&accf[lane], 1);
            mbar_init(&acc_free[lane], 8);
        }
        if (lane == 0) *abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(tmA);
        tma_prefetch_desc(tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
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
    // warps 2..9: this thread's row and half of the columns
    const bool drains = warp >= 2 && warp < 10;
    const int group = (warp - 2) >> 3;                      // of the decoding warps
    const int q = warp & 3, half = ((warp - 2) >> 2) & 1;
    constexpr int kHalf = RPT / 2;
    float acc[kHalf];
#pragma unroll
    for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;

    if (warp == 0) {
        int issued = 0;
        for (int it = 0, s = 0, ph = 0; it < n_iters; ++it) {
            if (!mbar_wait_uniform(&empty[s], ph ^ 1, abort, args.wait_ns)) {
                fail();
                break;
            }
            uint8_t* a = sA + s * L::kA;
            uint8_t* dst = sB + s * b_bytes;
            if (elect_one()) {
                if (ROLE != kRoleDx || it < n_main) {
                    const int kx = (k_begin + it) * 64;
                    mbar_arrive_expect_tx(&full[s], (dec ? raw_bytes : L::kA) + b_bytes);
                    if (ROLE == kRoleDx) {
                        tma_load_2d(sR + s * raw_bytes, tmA, &full[s], m0 / 2, kx);
                    } else if (dec) {
                        tma_load_2d(sR + s * raw_bytes, tmA, &full[s], amn ? m0 : kx, amn ? kx : m0);
                    } else if (amn) {
                        tma_load_2d(a, tmA, &full[s], m0, kx);
                        tma_load_2d(a + 8192, tmA, &full[s], m0 + 64, kx);
                    } else {
                        tma_load_2d(a, tmA, &full[s], kx, m0);
                    }
                    if (bmn) {
                        for (int c = 0; c < chunks; ++c) tma_load_2d(dst + c * L::kChunk, tmB, &full[s], c * 64, kx);
                    } else {
                        tma_load_2d(dst, tmB, &full[s], kx, 0);
                    }
                } else {
                    const int e = it - n_main, c = job.ext.c_col(e);
                    mbar_arrive_expect_tx(&full[s], L::kA + b_bytes);
                    tma_load_2d(a, &tmA1, &full[s], m0, c);
                    tma_load_2d(a + 8192, &tmA1, &full[s], m0 + 64, c);
                    tma_load_2d(dst, &tmB1, &full[s], e * 64, 0);
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
        const uint32_t idesc = make_idesc_bf16(128, n_mma, amn, bmn);
        const uint32_t a_step = amn ? 2048 : 32, b_step = bmn ? 2048 : 32;
        const uint64_t a_desc = make_sw128_desc(smem_u32(sA), amn ? 8192 : 16, 1024);
        const uint64_t b_desc = make_sw128_desc(smem_u32(sB), bmn ? 8192 : 16, 1024);
        int in_seg = 0, acc_i = 0, acc_ph = 1;      // accumulator tile of the segment, phase of its release
        for (int it = 0, s = 0, ph = 0; it < n_iters; ++it) {
            bool ok = true;
            if (in_seg == 0) ok = mbar_wait_uniform(&acc_free[acc_i], acc_ph, abort, args.wait_ns);
            if (ok && dec) ok = mbar_wait_uniform(&decoded[s], ph, abort, args.wait_ns);
            if (ok) ok = mbar_wait_uniform(&full[s], ph, abort, args.wait_ns);
            if (!ok) {
                fail();
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + static_cast<uint32_t>(acc_i * acc_cols);
            // (descriptors hold addresses in 16-byte units; shared memory ends below their field's 256 KB)
            const uint64_t ad = a_desc + static_cast<uint32_t>(s * (L::kA >> 4));
            const uint64_t bd = b_desc + static_cast<uint32_t>(s * (b_bytes >> 4));
            const bool last = in_seg + 1 == seg_len || it == n_iters - 1;
            if (ROLE == kRoleDx && it >= n_main) {
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = job.ext.c16(it - n_main, k);
                        if (c >= 0)
                            umma_bf16_ss(d, ad + ((c * a_step) >> 4), bd + ((k * b_step) >> 4), idesc,
                                         (in_seg > 0 || k > 0) ? 1u : 0u);
                    }
                    umma_commit(&empty[s]);
                    if (last) umma_commit(&accf[acc_i]);
                }
            } else if (elect_one()) {
                for (int b = 0; b < groups; ++b) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16_ss(d, ad + ((k * a_step) >> 4), bd + ((b * 2 * L::kChunk + k * b_step) >> 4), idesc,
                                     (in_seg > 0 || b > 0 || k > 0) ? 1u : 0u);
                }
                umma_commit(&empty[s]);
                if (last) umma_commit(&accf[acc_i]);
            }
            __syncwarp();
            ++in_seg;
            if (last) {
                in_seg = 0;
                if (++acc_i == NA) acc_i = 0, acc_ph ^= 1;
            }
            if (++s == S) s = 0, ph ^= 1;
        }
    } else {
        bool ok = true;
        int acc_i = 0, acc_ph = 0;
        auto drain = [&]() {
            ok = mbar_wait_warp(&accf[acc_i], acc_ph, abort, args.wait_ns);
            if (!ok) return;
            tc_fence_after();
            const uint32_t t = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc_i * acc_cols + half * kHalf;
#pragma unroll
            for (int c = 0; c < kHalf; c += 16)
                if (half * kHalf + c < N) {
                    uint32_t r0[16];
                    tmem_ld_32x32b_x16(t + c, r0);
                    if (RPT == 64 && terms == 3) {
                        // the smallest terms first (columns past a group are the next one's: never used)
                        uint32_t r1[16], r2[16];
                        tmem_ld_32x32b_x16(t + c + tr.stride, r1);
                        tmem_ld_32x32b_x16(t + c + 2 * tr.stride, r2);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            acc[c + j] += __uint_as_float(r0[j]) + (__uint_as_float(r1[j]) + __uint_as_float(r2[j]));
                    } else {
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[c + j] += __uint_as_float(r0[j]);
                    }
                }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_free[acc_i]);
            if (++acc_i == NA) acc_i = 0, acc_ph ^= 1;
        };
        // every kGroups-th stage, two per turn of the loop
        RingPos at(S, group);
        auto landed = [&]() {
            return ring_landed<L::kGroups>(
                at, [&](int i, int par) { return mbar_wait_warp(&empty[i], par, abort, args.wait_ns); },
                [&](int i, int par) { return mbar_wait_warp(&full[i], par, abort, args.wait_ns); });
        };
        int drained = 0;
        // after the pair at it0: the segments whose MMAs are behind it (those of the next rounds then find
        // their accumulator tiles free)
        auto drain_behind = [&](int it0) {
            for (const int end = (it0 + 4) / seg_len - NA / 2; ok && drained < end && drained < n_seg; ++drained) drain();
        };
        if constexpr (ROLE == kRoleDx) {
            // 32 columns of one weight row per thread and stage (the adapter's steps need no decode)
            const int td = (threadIdx.x - 64) & 255, row = td >> 2, blk_in = td & 3, sw = row & 7;
            const int64_t mblk = m0 / 32 + blk_in;
            uint32_t e[2] = {0, 0};
            float c2[2] = {0.f, 0.f};
            const int64_t k0 = static_cast<int64_t>(k_begin) * 64, ld = job.ld_scales;
            const int lim = mblk * 32 >= job.M ? 0 : min(static_cast<int64_t>(n_main), (job.K - k0 - row + 63) / 64);
            const uint8_t* sc = job.scales;
            const float* gc = job.c2;
            auto fetch = [&](int it, uint32_t& ev, float& cv) {
                if (it >= lim) return;
                const int64_t wrow = k0 + it * 64 + row;
                if (!dcheck(wrow < job.K && mblk * 32 < job.M, args.err)) return;
                if (op == kOpMxfp4) {
                    ev = __ldg(sc + mx_scale_offset(wrow, mblk, ld));
                } else {
                    const int64_t blk = wrow * ld + mblk / 2;
                    ev = __ldg(sc + blk);
                    cv = __ldg(gc + blk / kGroup);
                }
            };
            const int dst_off = (blk_in >> 1) * 8192 + row * 128, c0 = (blk_in & 1) * 4;
#pragma unroll
            for (int u = 0; u < 2; ++u) fetch(group + u * L::kGroups, e[u], c2[u]);
            for (int it0 = group; ok && it0 < n_iters; it0 += 2 * L::kGroups) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int it = it0 + u * L::kGroups;
                    if (!ok || it >= n_iters) break;
                    const uint32_t ev = e[u];
                    const float cv = c2[u];
                    fetch(it + 2 * L::kGroups, e[u], c2[u]);
                    ok = landed();
                    if (!ok) break;
                    const int s = at.s;
                    if (it < n_main) {
                        // (codes outside the weight are 0: the value 0 in MXFP4; NF4's is not, but meets only
                        // rows of dH that are 0 or columns past d_in)
                        const uint4 q = *reinterpret_cast<const uint4*>(sR + s * raw_bytes + row * 64 + blk_in * 16);
                        const uint32_t qs[4] = {q.x, q.y, q.z, q.w};
                        uint8_t* dst = sA + s * L::kA + dst_off;
                        if (op == kOpMxfp4) {
                            const float sc = e8m0_value(ev);
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                *reinterpret_cast<uint4*>(dst + (((c0 + c) ^ sw) << 4)) = e2m1_scale8_bf16(qs[c], sc);
                        } else {
                            const Nf4Planes pl = nf4_make_planes(nf4_block_scale(ev, cv));
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                *reinterpret_cast<uint4*>(dst + (((c0 + c) ^ sw) << 4)) = nf4_decode8(qs[c], pl);
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&decoded[s]);
                    at.skip(L::kGroups);
                }
                if (drains) drain_behind(it0);
            }
        } else if ((ROLE == kRoleUG || ROLE == kRoleAB) && dec) {
            const int td = (threadIdx.x - 64) & 255;              // the int8 block of this thread
            const int row = amn ? td >> 2 : td >> 1;              // row of the int8 tile
            const int blk_in = amn ? td & 3 : td & 1;             // block within the row
            // this thread's scales: `lim` of them (0 past the matrix), `step` bytes apart
            const int64_t ld = job.ld_scales, k0 = static_cast<int64_t>(k_begin) * 64;
            const int64_t step = amn ? 64 * ld : 2;
            const uint8_t* sc = job.scales + (amn ? (k0 + row) * ld + m0 / 32 : (m0 + row) * ld + k0 / 32) + blk_in;
            const bool there = amn ? m0 / 32 + blk_in < ld : m0 + row < job.M;
            const int lim = !there ? 0 : min(static_cast<int64_t>(n_iters), amn ? (job.K - k0 - row + 63) / 64 : n_iters);
            const int64_t n_scales = (amn ? job.K : job.M) * ld;
            auto scale_at = [&](int it) -> uint32_t {
                return it < lim && dcheck(sc + it * step < job.scales + n_scales, args.err) ? __ldg(sc + it * step) : 0u;
            };
            const int dst_off = amn ? (blk_in >> 1) * 8192 + row * 128 : row * 128;
            const int c0 = amn ? (blk_in & 1) * 4 : blk_in * 4, sw = row & 7;
            // the scales of this group's next two stages are in flight while it decodes (a load takes longer than
            // a step)
            uint32_t e[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) e[u] = scale_at(group + u * L::kGroups);
            for (int it0 = group; ok && it0 < n_iters; it0 += 2 * L::kGroups) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int it = it0 + u * L::kGroups;
                    if (!ok || it >= n_iters) break;
                    const float st = act8_step(e[u]);
                    e[u] = scale_at(it + 2 * L::kGroups);
                    ok = landed();
                    if (!ok) break;
                    const int s = at.s;
                    // (elements outside the matrix were filled with 0 by the copy)
                    const uint4* src = reinterpret_cast<const uint4*>(sR + s * L::kRaw + td * 32);
                    const uint4 v0 = src[0], v1 = src[1];
                    uint8_t* dst = sA + s * L::kA + dst_off;
                    *reinterpret_cast<uint4*>(dst + (((c0 + 0) ^ sw) << 4)) = act8_decode8(v0.x, v0.y, st);
                    *reinterpret_cast<uint4*>(dst + (((c0 + 1) ^ sw) << 4)) = act8_decode8(v0.z, v0.w, st);
                    *reinterpret_cast<uint4*>(dst + (((c0 + 2) ^ sw) << 4)) = act8_decode8(v1.x, v1.y, st);
                    *reinterpret_cast<uint4*>(dst + (((c0 + 3) ^ sw) << 4)) = act8_decode8(v1.z, v1.w, st);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&decoded[s]);
                    at.skip(L::kGroups);
                }
                if (drains) drain_behind(it0);
            }
        } else if (quant) {
            // one block of 32 per thread and stage, from the swizzled operand tile
            const int td = (threadIdx.x - 64) & 255, row = td >> 1, b = td & 1, sw = row & 7;
            const int64_t grow = static_cast<int64_t>(m0) + row;
            const bool in = grow < job.M;
            uint8_t* codes = job.mx_codes + grow * (job.K / 2) + b * 16;
            // a stage fills half a scale word of the row; its tile advances by 512 bytes every other stage
            uint8_t* word = job.mx_scales + mx_scale_offset(grow, k_begin * 2, mx_col_tiles(job.K));
            for (int it0 = group; ok && it0 < n_iters; it0 += 2 * L::kGroups) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int it = it0 + u * L::kGroups;
                    if (!ok || it >= n_iters) break;
                    ok = landed();
                    if (!ok) break;
                    const int s = at.s;
                    const uint8_t* src = sA + s * L::kA + row * 128;
                    Raw8<__nv_bfloat16> raw[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        raw[c].v = *reinterpret_cast<const uint4*>(src + (((4 * b + c) ^ sw) << 4));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[s]);       // the tile has been read
                    uint32_t e, v[4];
                    mxfp4_block32(raw, e, v);
                    if (in && dcheck(static_cast<int64_t>(k_begin + it) * 64 + b * 32 < job.K, args.err))
                        *reinterpret_cast<uint4*>(codes + static_cast<int64_t>(k_begin + it) * 32) =
                            make_uint4(v[0], v[1], v[2], v[3]);
                    e |= __shfl_xor_sync(0xffffffffu, e, 1) << 8;        // (of the even lane: both blocks' bytes)
                    if (in && b == 0 && dcheck(static_cast<int64_t>(k_begin + it) * 64 < job.K, args.err))
                        *reinterpret_cast<uint16_t*>(word + (it >> 1) * kMxTileBytes + (it & 1) * 2) = static_cast<uint16_t>(e);
                    at.skip(L::kGroups);
                }
                if (drains) drain_behind(it0);
            }
        }
        if (drains)
            for (; ok && drained < n_seg; ++drained) drain();
        if (!ok) fail();
    }
    __syncwarp();

    // ------------------------------------------------------------ join the ranks, write
    // The ring becomes red[source rank][row of this rank's share][kLdRed]: every MMA of every rank is
    // done before a rank writes into another's.
    const int R = 128 / C;
    if (C > 1) cluster_barrier();
    else __syncthreads();
    const bool dead = *abort != 0;
    if (drains && !dead) {
        const int row = q * 32 + lane;
        const uint32_t dst = mapa_shared(smem_u32(smem), static_cast<uint32_t>(C > 1 ? row / R : 0)) +
                             static_cast<uint32_t>(((rank * R + row % R) * L::kLdRed + half * kHalf) * 4);
#pragma unroll
        for (int j = 0; j < kHalf; j += 4)
            if (half * kHalf + j < N)
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + j * 4), "f"(acc[j]),
                             "f"(acc[j + 1]), "f"(acc[j + 2]), "f"(acc[j + 3])
                             : "memory");
    }
    if (C > 1) cluster_barrier();
    else __syncthreads();
    if (drains && !dead) {
        const float* red = reinterpret_cast<const float*>(smem);
        const int row0 = m0 + rank * R;
        const int rows = min(R, job.M - row0);
        auto total = [&](int rl, int j) {
            float v = 0.f;
            for (int c = 0; c < C; ++c) v += red[(c * R + rl) * L::kLdRed + j];
            return v;
        };
        const int td = threadIdx.x - 64;
        const int mode = ROLE == kRoleU ? kActU : ROLE == kRoleUG ? kActTriple : ROLE == kRoleDx ? kActDx : job.mode;
        const float scale = job.scale;
        if (mode == kActDx || mode == kActCols) {
            // column by column: consecutive threads on consecutive rows (R a power of two)
            const int sh = 31 - __clz(R);
            const bool add = job.accumulate != 0;
            for (int i = td; i < R * N; i += 256) {
                const int j = i >> sh, rl = i & (R - 1);
                if (rl >= rows) continue;
                const int64_t at = static_cast<int64_t>(j) * job.M + row0 + rl;
                if (!dcheck(j < N && row0 + rl < job.M, args.err)) continue;
                const float v = total(rl, j);
                if (mode == kActDx) static_cast<__nv_bfloat16*>(job.out)[at] = __float2bfloat16_rn(v);
                else static_cast<float*>(job.out)[at] = add ? static_cast<float*>(job.out)[at] + scale * v : scale * v;
            }
        } else {
            // row by row, four columns per thread (the joining buffer's rows are 16-byte units)
            const int n4 = mode == kActTriple ? tr.stride / 4 : mode == kActU ? 4 * ((N + 15) / 16) : (N + 3) / 4;
            for (int rl = td / n4, g = td - rl * n4; rl < rows;) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (4 * g < N)
                    for (int c = 0; c < C; ++c) {
                        const float4 o = *reinterpret_cast<const float4*>(red + (c * R + rl) * L::kLdRed + 4 * g);
                        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                    }
                const int64_t row = row0 + rl;
                if (!dcheck(row < job.M && g < n4, args.err)) break;
                const int j = 4 * g, left = N - j;           // columns of this group that exist
                float x[4] = {v.x, left > 1 ? v.y : 0.f, left > 2 ? v.z : 0.f, left > 3 ? v.w : 0.f};
                if (mode == kActTriple) {
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(job.out) + row * tr.ld + j;
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] *= scale;
#pragma unroll
                    for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2*>(out + k * tr.stride) = bf16_term(x);
                } else if (mode == kActU) {
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(job.out) + row * ext_ld(N) + j;
                    if (job.out2) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (e < left) job.out2[row * N + j + e] = __float2bfloat16_rn(x[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] *= scale;
#pragma unroll
                    for (int k = 0; k < 2; ++k) *reinterpret_cast<uint2*>(out + k * tr.stride) = bf16_term(x);
                } else {
                    float* out = static_cast<float*>(job.out) + row * N + j;
                    const bool add = job.accumulate != 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left) out[e] = add ? out[e] + scale * x[e] : scale * x[e];
                }
                // (no division in the loop: 256 threads further on)
                for (g += 256; g >= n4; g -= n4) ++rl;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// What a backward has to lay out before its products: the weight decoded to bf16 (MXFP4 or NF4, eight
// elements per thread), copies of matrices whose rows are no whole 16-byte units to zero-padded rows (dH, B,
// a given U), and cleared ticket counters.  Each part has its own range of CTAs.  It reads nothing that the
// kernel in front writes and writes nothing that it reads, so it runs beside it and waits for it last: a
// kernel behind then still finds both finished.  Bound by HBM: 4096 x 4096 from MXFP4 in 10.7 us, 11008 x 4096
// from NF4 in 21.7 us (113 MB, 5.2 TB/s, four fifths of it writes).
struct BwdPrepArgs {
    const uint8_t* codes;
    const uint8_t* mx_scales;     // MXFP4 weight (one scale tile per CTA), or
    const uint8_t* absmax_q;      // NF4 weight (eight elements per thread and step)
    const float* c2;
    int64_t d_out, d_in;
    __nv_bfloat16* w;
    int ctas_w;
    PadCopy pad[3];
    int* zero;
    int n_zero;
};
constexpr int kPrepUnroll = 4;
__global__ void __launch_bounds__(256) k_bwd_prepare(const __grid_constant__ BwdPrepArgs a) {
    griddep_launch_dependents();
    int b = blockIdx.x;
    if (b < a.ctas_w && a.mx_scales) {
        __shared__ __align__(16) uint8_t s_sc[kMxTileBytes];
        const int64_t kts = mx_col_tiles(a.d_in);
        mxfp4_dequantize_tile(a.codes, a.mx_scales, a.d_out, a.d_in, b / kts, b % kts, a.w, s_sc);
        griddep_wait();
        return;
    }
    if (b < a.ctas_w) {
        const int64_t i0 = static_cast<int64_t>(b) * (256 * kPrepUnroll) + threadIdx.x, n8 = a.d_out * a.d_in / 8;
        uint32_t q[kPrepUnroll], e[kPrepUnroll];
        float c[kPrepUnroll];
#pragma unroll
        for (int u = 0; u < kPrepUnroll; ++u) {
            const int64_t i = i0 + u * 256;
            if (i < n8) {
                q[u] = __ldg(reinterpret_cast<const uint32_t*>(a.codes) + i);
                e[u] = __ldg(a.absmax_q + (i >> 3));
                c[u] = __ldg(a.c2 + (i >> 3) / kGroup);
            }
        }
#pragma unroll
        for (int u = 0; u < kPrepUnroll; ++u) {
            const int64_t i = i0 + u * 256;
            if (i < n8)
                reinterpret_cast<uint4*>(a.w)[i] = nf4_decode8(q[u], nf4_make_planes(nf4_block_scale(e[u], c[u])));
        }
        griddep_wait();
        return;
    }
    b -= a.ctas_w;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        if (b >= 0 && b < a.pad[p].ctas) a.pad[p].run(b);
        b -= a.pad[p].ctas;
    }
    if (b == 0)
        for (int i = threadIdx.x; i < a.n_zero; i += 256) a.zero[i] = 0;
    griddep_wait();
}

}  // namespace qlora
