// mx_api.cuh -- host side of the microscaled entry points (included by qlora_api.cu): planning,
// argument checks and launch sequences of the MXFP4 layer, the 8-bit activation checkpoints and the
// backward passes that read them.
#pragma once

namespace {

// ======================================================================= planning

constexpr int pad8(int64_t n) { return static_cast<int>((n + 7) / 8 * 8); }   // whole 16-byte units of bf16
constexpr int64_t kMaxDim = 1LL << 30;
// Up to this many tokens the MXFP4 forward streams the weight past tiles of 128 tokens, above it computes
// 256 x 256 tiles.  Stream against tiles (us): 300 tokens of 11008 x 4096 21.2, 28.4; of 4096 x 4096 18.1,
// 19.3; of 8192 x 8192 29.3, 28.2; 400 of the same layers 28.9, 29.0; 18.9, 19.7; 33.3, 31.1.
constexpr int64_t kMxStreamMaxT = 384;
// Up to this many tokens (one tile of k_act_gemm) dX decodes the weight in the CTA, above it reads the
// weight decoded to bf16 beforehand.  The whole backward that way and that (us): 64 tokens of 4096 x 4096
// 29, 33; of 8192 x 8192 58, 77; of 2048 x 2048 23.4, 22.7; 128 tokens (two tiles) 36, 35; 79, 80; 27, 22.7.
constexpr int64_t kDxFewT = 64;

qlora_status mx_check_dims(int64_t rows, int64_t cols) {
    if (rows < 1 || rows > kMaxDim || cols < 64 || cols % 64 || cols > kMaxDim) return QLORA_ERR_UNSUPPORTED;
    if (cdiv(rows, 128) * mx_col_tiles(cols) > (1LL << 28)) return QLORA_ERR_UNSUPPORTED;   // grids
    return QLORA_OK;
}
inline size_t mx_scale_bytes(int64_t rows, int64_t cols) {
    return static_cast<size_t>(cdiv(rows, 128)) * mx_col_tiles(cols) * kMxTileBytes;
}
qlora_status check_mxfp4(const qlora_mxfp4* w) {
    if (!w || !aligned16(w->codes) || !aligned16(w->scales)) return QLORA_ERR_INVALID_ARG;
    return mx_check_dims(w->d_out, w->d_in);
}

// CTAs of the checkpoint's format kernels: 256 threads, kAct8Unroll steps of 8 elements each.
unsigned act8_ctas(int64_t n8) { return static_cast<unsigned>(cdiv(n8, 256 * kAct8Unroll)); }

// Routes of the MXFP4 forward by the number of tokens.
enum MxRoute { kMxDecode, kMxStream64, kMxStream128, kMxPair };
MxRoute mx_route(int64_t T) {
    if (T <= kMxDecodeT) return kMxDecode;
    if (T <= 64) return kMxStream64;
    return T <= kMxStreamMaxT ? kMxStream128 : kMxPair;
}

// Ranks of a weight-stream cluster: as many of 4, 2, 1 as K has stages for and `slots` can take at once,
// two CTAs per SM at T <= 16 (whose rings are small), one above.  8 ranks of half the length measured 8.4
// against 7.7 us at one token of a 4096 x 4096 layer, the same at 64 tokens of it.
int mx_ranks(int64_t ctas, int64_t chunks, int64_t slots) {
    for (int c = 4; c > 1; c >>= 1)
        if (chunks >= c && ctas * c <= slots) return c;
    return 1;
}

struct MxFwdPlan {
    int RP = 0;
    size_t codes = 0, scales = 0, us = 0, b_pad = 0, total = 0;
    PairSched sched;
};
MxFwdPlan mx_fwd_plan(int64_t T, int64_t d_out, int64_t d_in, int r) {
    MxFwdPlan p;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = align256(off + bytes);
        return o;
    };
    p.RP = pad_rank(r);
    if (mx_route(T) != kMxDecode) {
        p.codes = take(static_cast<size_t>(T) * d_in / 2);
        p.scales = take(mx_scale_bytes(T, d_in));
    }
    p.us = take(static_cast<size_t>(T) * ext_ld(r) * 2);
    if (r % 8) p.b_pad = take(static_cast<size_t>(d_out) * pad8(r) * 2);
    if (mx_route(T) == kMxPair) {
        p.sched = pair_schedule(T, d_out, cdiv(d_in, 256), true, kSmsForSplit / 2);
    }
    p.total = off;
    return p;
}

// The backward of an MXFP4 or NF4 base from a bf16 activation or an 8-bit checkpoint.
struct MxBwdPlan {
    int RP = 0;
    size_t b_pad = 0, dh_pad = 0, u3 = 0, g3 = 0, w = 0, pair = 0, total = 0;
    PairSched sched;
};
MxBwdPlan mx_bwd_plan(int64_t T, int64_t d_out, int64_t d_in, int r) {
    MxBwdPlan p;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = align256(off + bytes);
        return o;
    };
    p.RP = pad_rank(r);
    if (r % 8) p.b_pad = take(static_cast<size_t>(d_out) * pad8(r) * 2);
    if (d_out % 8) p.dh_pad = take(static_cast<size_t>(T) * ((d_out + 7) / 8 * 8) * 2);
    const size_t triple = static_cast<size_t>(T) * act_triple(r).ld * 2;
    p.u3 = take(triple);           // U and s G, three bf16 terms each (or a given U in padded rows)
    p.g3 = take(triple);
    if (T > kDxFewT) {
        p.w = take(static_cast<size_t>(d_out) * d_in * 2);  // the decoded weight
        p.sched = pair_schedule(T, d_in, cdiv(d_out, 64), false, kSmsForSplit / 2);
        p.pair = take(p.sched.bytes());
    }
    p.total = off;
    return p;
}

size_t mx_workspace_bytes(int op, qlora_dtype dtype, int64_t T, int64_t d_out, int64_t d_in, int32_t r) {
    if (dtype != QLORA_BF16 || T < 1 || T > kMaxDim || r < 1 || r > 128) return 0;
    if (mx_check_dims(d_out, d_in) != QLORA_OK) return 0;
    if (op == QLORA_OP_FWD_MXFP4)
        return mx_check_dims(T, d_in) == QLORA_OK ? mx_fwd_plan(T, d_out, d_in, r).total : 0;
    return mx_bwd_plan(T, d_out, d_in, r).total;
}

// ======================================================================= launchers

template <typename K>
qlora_status allow_smem(K kern, int bytes, std::atomic<uint64_t>& configured) {
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return QLORA_ERR_CUDA;
        configured.fetch_or(bit);
    }
    return QLORA_OK;
}

template <int NT>
qlora_status launch_mx_stream(const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tb,
                              const CUtensorMap& tu, MxStreamArgs g, cudaStream_t st) {
    using L = MxStreamCfg<NT>;
    static std::atomic<uint64_t> configured{0};
    QL_TRY(allow_smem(k_mx_stream<NT>, L::bytes(L::kAlone), configured));
    const int64_t tiles = cdiv(g.d_out, 128), tok = cdiv(g.T, NT), chunks = cdiv(g.k64, 4);
    g.ranks = mx_ranks(tiles * tok, chunks, L::kQuant ? 2 * kSmsForSplit : kSmsForSplit);
    // a ring of all of the shared memory where each CTA has an SM to itself, no longer than its K
    g.stages = L::kShared;
    if (tiles * g.ranks * tok <= kSmsForSplit)
        g.stages = static_cast<int>(std::min<int64_t>(L::kAlone, std::max<int64_t>(L::kShared, cdiv(chunks, g.ranks) + g.ext.steps)));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(g.ranks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * g.ranks), static_cast<unsigned>(tok));
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(L::bytes(g.stages));
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = g.ranks > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, k_mx_stream<NT>, tw, tx, tb, tu, g) != cudaSuccess) return QLORA_ERR_CUDA;
    QL_LAUNCH_CHECK();
    return QLORA_OK;
}

// One launch of one or two adapter products.  The cluster size (K ranks) is the one with the shortest
// schedule by the measured costs: a K step of a bf16 product 1 (0.33 us), of a triple 1.3, of one whose
// operand is decoded or quantized on the way 1.8, a CTA besides 8.  One CTA fills an SM, and clusters do not
// fill the card: 33 clusters of four and 15 of eight run at once (cudaOccupancyMaxActiveClusters; dX of 16 tokens,
// 2048 x 2048, as 16 clusters of eight 25.2 us with the rest, as 16 of four 21.5).
struct ActLaunch {
    ActGemmArgs g{};
    CUtensorMap a[2], b[2];
    int n = 0;
    bool pdl = true;         // launched with programmatic dependent launch
    ActJob& add(int64_t M, int N, int64_t K) {
        ActJob& j = g.job[n++];
        j.M = static_cast<int>(M);
        j.N = N;
        j.K = K;
        j.k_steps = static_cast<int>(cdiv(K, 64));
        j.scale = 1.f;
        return j;
    }
};
template <int RPT, int ROLE>
qlora_status launch_act_gemm(ActLaunch& l, int* err, cudaStream_t st) {
    using L = ActGemmSmem<RPT>;
    auto kern = k_act_gemm<RPT, ROLE>;
    static std::atomic<uint64_t> configured{0};
    QL_TRY(allow_smem(kern, L::kTotal, configured));
    if (l.n == 1 && !l.g.job[0].ext.steps) {
        l.a[1] = l.a[0];
        l.b[1] = l.b[0];
    }
    int64_t tiles = 0;
    int steps = 1 << 30;
    for (int i = 0; i < l.n; ++i) {
        tiles += cdiv(l.g.job[i].M, 128);
        steps = std::min(steps, l.g.job[i].mx_codes ? (l.g.job[i].k_steps + 1) / 2 : l.g.job[i].k_steps);
    }
    double best = 0;
    for (int c = 1; c <= 8 && c <= steps; c *= 2) {
        // one wave ends with its longest CTA, several of equal CTAs are whole; others end, on average, half a CTA
        // after an even share
        const double slots = c == 8 ? 120 : c == 4 ? 132 : kSmsForSplit;
        double total = 8.0 * l.g.qx_tiles, longest = 0;
        for (int i = 0; i < l.n; ++i) {
            const ActJob& j = l.g.job[i];
            const double one = cdiv(j.k_steps, c) * ((j.op != kOpBf16 || j.mx_codes) ? 1.8 : j.triple ? 1.3 : 1.0) + 8;
            total += one * cdiv(j.M, 128) * c;
            longest = std::max(longest, one);
        }
        const int64_t ctas = tiles * c + l.g.qx_tiles;
        const double cost = ctas <= slots                     ? longest
                            : l.n == 1 && l.g.qx_tiles == 0 ? std::ceil(static_cast<double>(ctas) / slots) * longest
                                                              : total / slots + longest / 2;
        if (c == 1 || cost < best) {
            best = cost;
            l.g.ranks = c;
        }
    }
    l.g.tiles0 = static_cast<int>(cdiv(l.g.job[0].M, 128));
    l.g.tiles = static_cast<int>(tiles);
    l.g.pad.ctas = static_cast<int>(cdiv(l.g.pad.ctas, l.g.ranks)) * l.g.ranks;
    l.g.qx_ctas = static_cast<int>(cdiv(l.g.qx_tiles, l.g.ranks)) * l.g.ranks;
    l.g.err = err;
    l.g.wait_ns = kWaitNs;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(l.g.ranks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * l.g.ranks + l.g.qx_ctas + l.g.pad.ctas));
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = L::kTotal;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = l.pdl ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, l.a[0], l.b[0], l.a[1], l.b[1], l.g) != cudaSuccess) return QLORA_ERR_CUDA;
    QL_LAUNCH_CHECK();
    return QLORA_OK;
}
template <int ROLE>
qlora_status act_gemm(int rpt, ActLaunch& l, int* err, cudaStream_t st) {
    return rpt == 64 ? launch_act_gemm<64, ROLE>(l, err, st) : launch_act_gemm<128, ROLE>(l, err, st);
}

template <bool MX, int BN>
qlora_status launch_pair_gemm(const CUtensorMap (&t)[6], PairGemmArgs g, const PairSched& sch, void* ws, int* err,
                              cudaStream_t st) {
    using L = PairGemmSmem<MX, BN>;
    auto kern = k_pair_gemm<MX, BN>;
    g.split = sch.split;
    g.tail_tiles = sch.tail;
    if (sch.split > 1) {
        g.part = static_cast<float*>(ws);
        g.cnt = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + sch.part_bytes);
    }
    g.err = err;
    g.wait_ns = kWaitNs;
    static std::atomic<uint64_t> configured{0};
    QL_TRY(allow_smem(kern, L::kTotal, configured));
    if (launch_pdl(kern, dim3(2 * sch.pairs), dim3(L::kThreads), L::kTotal, st, t[0], t[1], t[2], t[3], t[4],
                   t[5], g) != cudaSuccess)
        return QLORA_ERR_CUDA;
    QL_LAUNCH_CHECK();
    return QLORA_OK;
}

// Scale tiles as rows of 128 words, two tiles (256 elements of K) per box.
qlora_status tmap_scales(CUtensorMap* m, const void* base, int64_t rows, int64_t cols) {
    QL_TRY(get_encoder());
    cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(cdiv(rows, 128) * mx_col_tiles(cols))};
    cuuint64_t strides[1] = {kMxTileBytes};
    cuuint32_t box[2] = {128, 2};
    cuuint32_t es[2] = {1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? QLORA_OK : QLORA_ERR_CUDA;
}

// dX = dH W + (sG) A over the weight decoded to bf16 in the workspace.
qlora_status dx_gemm(const void* W, const void* dH, int64_t dh_ld, int64_t T, int64_t d_out, int64_t d_in,
                     const void* sG, const void* A, int r, void* dX, const PairSched& sch, void* pair_ws,
                     int* err, cudaStream_t st) {
    CUtensorMap t[6];
    QL_TRY(tmap_bf16(&t[0], dH, T, d_out, dh_ld, 128));
    QL_TRY(tmap_bf16(&t[1], W, d_out, d_in, d_in, 64));
    QL_TRY(tmap_bf16(&t[4], sG, T, 2 * act_triple(r).stride, act_triple(r).ld, 128));
    QL_TRY(tmap_bf16(&t[5], A, r, d_in, d_in, 64));
    t[2] = t[3] = t[0];
    PairGemmArgs g{};
    g.M = static_cast<int>(T);
    g.N = static_cast<int>(d_in);
    g.k_steps = static_cast<int>(cdiv(d_out, 64));
    g.k_mma_last = static_cast<int>(cdiv(d_out - 64 * (g.k_steps - 1), 16));
    g.ext = ext_steps_of(r);
    g.m_tiles = static_cast<int>(cdiv(T, 256));
    g.n_tiles = static_cast<int>(cdiv(d_in, sch.bn));
    g.out = static_cast<__nv_bfloat16*>(dX);
    g.ld_out = d_in;
    return sch.bn == 256 ? launch_pair_gemm<false, 256>(t, g, sch, pair_ws, err, st)
                         : launch_pair_gemm<false, 128>(t, g, sch, pair_ws, err, st);
}

PadCopy pad_copy(const void* src, void* dst, int64_t rows, int64_t cols, int64_t ld, int most_ctas) {
    PadCopy p{};
    p.src = static_cast<const __nv_bfloat16*>(src);
    p.dst = static_cast<__nv_bfloat16*>(dst);
    p.rows = rows;
    p.cols = static_cast<int>(cols);
    p.ld = static_cast<int>(ld);
    p.ctas = static_cast<int>(std::min<int64_t>(cdiv(rows * ld, 1024), most_ctas));
    return p;
}

// ======================================================================= sequences

qlora_status mx_fwd(const qlora_mxfp4* w, const void* X, int64_t T, const void* A, const void* B, int r, float s,
                    void* H, void* U_save, void* ws, int* err, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const int64_t d_out = w->d_out, d_in = w->d_in;
    const MxFwdPlan p = mx_fwd_plan(T, d_out, d_in, r);
    const MxRoute route = mx_route(T);
    const int RP = p.RP;
    auto* codes = at<uint8_t>(ws, p.codes);
    auto* scales = at<uint8_t>(ws, p.scales);
    auto* us = at<bf>(ws, p.us);
    // B as the extension operand: the caller's where its rows are whole 16-byte units (the tensor
    // map fills the rank padding with 0), else a padded copy
    const bool direct = r % 8 == 0;
    const void* b_src = direct ? B : at<void>(ws, p.b_pad);
    const int b_ld = pad8(r);
    // The first kernel is launched without programmatic dependent launch: whatever wrote the weight
    // and whatever used this workspace has finished before it starts.
    if (route == kMxDecode) {
        MxPrepArgs a{};
        a.X = static_cast<const bf*>(X);
        a.A = static_cast<const bf*>(A);
        a.T = static_cast<int>(T);
        a.r = r;
        a.d_in = d_in;
        a.s = s;
        a.u_save = static_cast<bf*>(U_save);
        a.us = us;
        if (!direct) a.pad = pad_copy(B, at<void>(ws, p.b_pad), d_out, r, b_ld, kSmsForSplit);
        k_mx_prepare<<<static_cast<unsigned>(r + a.pad.ctas), 256, 0, st>>>(a);
        QL_LAUNCH_CHECK();
    } else {
        // U = X A^T and the MXFP4 of X, in one pass over X
        ActLaunch l;
        l.pdl = false;
        ActJob& ju = l.add(T, r, d_in);
        ju.scale = s;
        ju.out = us;
        ju.out2 = static_cast<bf*>(U_save);
        const int64_t qx_tiles = cdiv(T, 128) * mx_col_tiles(d_in);
        if (cdiv(T, 128) > 5) {
            ju.mx_codes = codes;
            ju.mx_scales = scales;
        } else {
            // few token tiles: their CTAs (8 at most for each) would be slow at it, the other SMs are free (640
            // tokens of 8192 x 8192 44.3 us against 44.7, of 4096 x 4096 20.0 against 22.4; 768 tokens 47.2
            // against 45.0, 22.9 against 22.5)
            l.g.qx = static_cast<const bf*>(X);
            l.g.qx_rows = T;
            l.g.qx_cols = d_in;
            l.g.qx_codes = codes;
            l.g.qx_scales = scales;
            l.g.qx_tiles = static_cast<int>(qx_tiles);
        }
        if (!direct) l.g.pad = pad_copy(B, at<void>(ws, p.b_pad), d_out, r, b_ld, kSmsForSplit / 2);
        QL_TRY(tmap_bf16(&l.a[0], X, T, d_in, d_in, 128));
        QL_TRY(tmap_bf16(&l.b[0], A, r, d_in, d_in, static_cast<uint32_t>(RP)));
        QL_TRY(act_gemm<kRoleU>(RP, l, err, st));
    }
    if (route == kMxPair) {
        CUtensorMap t[6];
        QL_TRY(tmap_u8_sw128(&t[0], codes, T, d_in / 2, d_in / 2, 128));
        QL_TRY(tmap_u8_sw128(&t[1], w->codes, d_out, d_in / 2, d_in / 2, 128));
        QL_TRY(tmap_scales(&t[2], scales, T, d_in));
        QL_TRY(tmap_scales(&t[3], w->scales, d_out, d_in));
        QL_TRY(tmap_bf16(&t[4], us, T, 2 * act_triple(r).stride, ext_ld(r), 128));
        QL_TRY(tmap_bf16(&t[5], b_src, d_out, r, b_ld, 128));
        PairGemmArgs g{};
        g.M = static_cast<int>(T);
        g.N = static_cast<int>(d_out);
        g.k_steps = static_cast<int>(cdiv(d_in, 256));
        g.k_mma_last = static_cast<int>(d_in / 64 - 4 * (g.k_steps - 1));
        g.ext = ext_steps_of(r);
        g.m_tiles = static_cast<int>(cdiv(T, 256));
        g.n_tiles = static_cast<int>(cdiv(d_out, 256));
        g.a_sf_tiles = g.b_sf_tiles = static_cast<int>(mx_col_tiles(d_in));
        g.out = static_cast<bf*>(H);
        g.ld_out = d_out;
        return launch_pair_gemm<true, 256>(t, g, p.sched, nullptr, err, st);
    }
    CUtensorMap tw, tx, tb, tu;
    const uint32_t nt = route == kMxDecode ? 16 : (route == kMxStream64 ? 64 : 128);
    QL_TRY(tmap_u8_sw128(&tw, w->codes, d_out, d_in / 2, d_in / 2, 128));
    if (route == kMxDecode) tx = tw;       // (X is quantized in the kernel)
    else QL_TRY(tmap_u8_sw128(&tx, codes, T, d_in / 2, d_in / 2, nt));
    QL_TRY(tmap_bf16(&tb, b_src, d_out, r, b_ld, 128));
    QL_TRY(tmap_bf16(&tu, us, T, 2 * act_triple(r).stride, ext_ld(r), nt));
    MxStreamArgs g{};
    g.T = static_cast<int>(T);
    g.d_out = static_cast<int>(d_out);
    g.k64 = static_cast<int>(d_in / 64);
    g.col_tiles = static_cast<int>(mx_col_tiles(d_in));
    g.ext = ext_steps_of(r);
    g.w_scales = w->scales;
    g.x_scales = scales;
    g.X = static_cast<const bf*>(X);
    g.d_in = d_in;
    g.out = static_cast<bf*>(H);
    g.err = err;
    g.wait_ns = kWaitNs;
    if (route == kMxDecode) return launch_mx_stream<16>(tw, tx, tb, tu, g, st);
    if (route == kMxStream64) return launch_mx_stream<64>(tw, tx, tb, tu, g, st);
    return launch_mx_stream<128>(tw, tx, tb, tu, g, st);
}

// The base weight of a backward: exactly one of the two.
struct MxBase {
    const qlora_nf4* nf4;
    const qlora_mxfp4* mx;
};

// X (bf16) or X8 (8-bit checkpoint), exactly one of the two, is the layer's activation.
qlora_status mx_bwd(MxBase base, const void* X, const qlora_act8* X8, const void* dH, int64_t T, const void* A,
                    const void* B, int r, float s, const void* U_saved, void* dX, float* dA, float* dB, void* ws,
                    int acc, BwdPhase phase, int* err, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const int64_t d_out = base.mx ? base.mx->d_out : base.nf4->d_out;
    const int64_t d_in = base.mx ? base.mx->d_in : base.nf4->d_in;
    const MxBwdPlan p = mx_bwd_plan(T, d_out, d_in, r);
    const int RP = p.RP;
    auto* u3 = at<bf>(ws, p.u3);
    auto* g3 = at<bf>(ws, p.g3);
    auto* W = at<bf>(ws, p.w);
    const bool grads = phase != kBwdDx, want_dx = dX && phase != kBwdGrads;
    const int64_t dh_ld = (d_out + 7) / 8 * 8;
    const void* b_src = B;
    const void* u_src = U_saved ? U_saved : u3;
    const ActTriple tr = act_triple(r);
    int b_ld = r, u_ld = U_saved ? r : tr.ld;
    // The call's first kernel is launched without programmatic dependent launch, so that whatever used
    // the workspace before has ended; the others start their prologue, or all of it where they depend on
    // nothing of this call, beside the one in front.
    bool first = true;
    auto prepare = [&](BwdPrepArgs& a) -> qlora_status {
        const int ctas = a.ctas_w + a.pad[0].ctas + a.pad[1].ctas + a.pad[2].ctas + (a.n_zero ? 1 : 0);
        if (!ctas) return QLORA_OK;
        if (first) k_bwd_prepare<<<ctas, 256, 0, st>>>(a);
        else if (launch_pdl(k_bwd_prepare, dim3(ctas), dim3(256), 0, st, a) != cudaSuccess) return QLORA_ERR_CUDA;
        QL_LAUNCH_CHECK();
        first = false;
        return QLORA_OK;
    };
    {
        // rows that are no whole 16-byte units cannot be read by a tensor map
        BwdPrepArgs a{};
        if (d_out % 8) {
            a.pad[0] = pad_copy(dH, at<void>(ws, p.dh_pad), T, d_out, dh_ld, 4 * kSmsForSplit);
            dH = at<void>(ws, p.dh_pad);
        }
        if (r % 8 && grads) {
            a.pad[1] = pad_copy(B, at<void>(ws, p.b_pad), d_out, r, pad8(r), kSmsForSplit);
            b_src = at<void>(ws, p.b_pad);
            b_ld = pad8(r);
            if (U_saved) {
                a.pad[2] = pad_copy(U_saved, u3, T, r, pad8(r), kSmsForSplit);
                u_src = u3;
                u_ld = pad8(r);
            }
        }
        QL_TRY(prepare(a));
    }
    if (grads) {
        // s G = s dH B, and U = X~ A^T unless the forward kept it
        ActLaunch l;
        ActJob& jg = l.add(T, r, d_out);
        jg.bmn = 1;
        jg.scale = s;
        jg.out = g3;
        QL_TRY(tmap_bf16(&l.a[0], dH, T, d_out, dh_ld, 128));
        QL_TRY(tmap_bf16(&l.b[0], b_src, d_out, r, b_ld, 64));
        if (!U_saved) {
            ActJob& ju = l.add(T, r, d_in);
            ju.out = u3;
            if (X8) {
                ju.op = kOpInt8;
                ju.scales = X8->scales;
                ju.ld_scales = d_in / 32;
                QL_TRY(tmap_u8(&l.a[1], X8->q, T, d_in, d_in, 64, 128));
            } else {
                QL_TRY(tmap_bf16(&l.a[1], X, T, d_in, d_in, 128));
            }
            QL_TRY(tmap_bf16(&l.b[1], A, r, d_in, d_in, static_cast<uint32_t>(RP)));
        }
        l.pdl = !first;
        first = false;
        QL_TRY(act_gemm<kRoleUG>(RP, l, err, st));
    }
    if (want_dx && T > kDxFewT) {
        BwdPrepArgs a{};
        a.codes = base.mx ? base.mx->codes : base.nf4->codes;
        if (base.mx) {
            a.mx_scales = base.mx->scales;
        } else {
            a.absmax_q = base.nf4->absmax_q;
            a.c2 = base.nf4->c2;
        }
        a.d_out = d_out;
        a.d_in = d_in;
        a.w = W;
        a.ctas_w = static_cast<int>(base.mx ? cdiv(d_out, 128) * mx_col_tiles(d_in) : cdiv(d_out * d_in / 8, 256 * kPrepUnroll));
        a.zero = at<int>(ws, p.pair + p.sched.part_bytes);
        a.n_zero = p.sched.n_cnt;
        QL_TRY(prepare(a));
    }
    // dX = dH W + (sG) A, s G as the first two terms of its triple
    if (want_dx && T <= kDxFewT) {
        ActLaunch l;
        ActJob& j = l.add(d_in, static_cast<int>(T), d_out);
        j.ext = ext_steps_of(r);
        j.out = dX;
        if (base.mx) {
            j.op = kOpMxfp4;
            j.scales = base.mx->scales;
            j.ld_scales = mx_col_tiles(d_in);
        } else {
            j.op = kOpNf4;
            j.scales = base.nf4->absmax_q;
            j.c2 = base.nf4->c2;
            j.ld_scales = d_in / 64;
        }
        QL_TRY(tmap_u8(&l.a[0], base.mx ? base.mx->codes : base.nf4->codes, d_out, d_in / 2, d_in / 2, 64, 64));
        QL_TRY(tmap_bf16(&l.b[0], dH, T, d_out, dh_ld, 64));
        QL_TRY(tmap_bf16(&l.a[1], A, r, d_in, d_in, 64));
        QL_TRY(tmap_bf16(&l.b[1], g3, T, 2 * tr.stride, tr.ld, 64));
        l.pdl = !first;
        QL_TRY((launch_act_gemm<64, kRoleDx>(l, err, st)));
    } else if (want_dx) QL_TRY(dx_gemm(W, dH, dh_ld, T, d_out, d_in, g3, A, r, dX, p.sched, at<void>(ws, p.pair), err, st));
    if (grads) {
        // dA^T[d_in, r] = X~^T (s G) and dB[d_out, r] = s dH^T U
        ActLaunch l;
        ActJob& ja = l.add(d_in, r, T);
        ja.triple = 1;
        ja.mode = kActCols;
        ja.accumulate = acc;
        ja.out = dA;
        if (X8) {
            ja.op = kOpInt8;
            ja.scales = X8->scales;
            ja.ld_scales = d_in / 32;
            QL_TRY(tmap_u8(&l.a[0], X8->q, T, d_in, d_in, 128, 64));
        } else {
            QL_TRY(tmap_bf16(&l.a[0], X, T, d_in, d_in, 64));
        }
        QL_TRY(tmap_bf16(&l.b[0], g3, T, tr.ld, tr.ld, 64));
        ActJob& jb = l.add(d_out, r, T);
        jb.triple = !U_saved;
        jb.mode = kActRows;
        jb.scale = s;
        jb.accumulate = acc;
        jb.out = dB;
        QL_TRY(tmap_bf16(&l.a[1], dH, T, d_out, dh_ld, 64));
        QL_TRY(tmap_bf16(&l.b[1], u_src, T, U_saved ? r : tr.ld, u_ld, 64));
        QL_TRY(act_gemm<kRoleAB>(RP, l, err, st));
    }
    return QLORA_OK;
}

constexpr uint32_t kBwdFlags = QLORA_BWD_ACCUMULATE | QLORA_BWD_GRADS_ONLY | QLORA_BWD_DX_FROM_WS;

// Checks shared by the two backward entries; X or X8 is the activation (checked by the caller's
// rule), then the launch sequence.
qlora_status mx_bwd_entry(MxBase base, const void* X, const qlora_act8* X8, const void* dH, int64_t T, const void* A,
                          const void* B, int32_t r, float alpha, const void* U_saved, void* dX, float* dA, float* dB,
                          void* ws, size_t ws_bytes, uint32_t flags, cudaStream_t st) {
    if (T < 1 || T > kMaxDim || r < 1 || r > 128) return QLORA_ERR_UNSUPPORTED;
    if (flags & ~kBwdFlags) return QLORA_ERR_INVALID_ARG;
    const bool grads_only = flags & QLORA_BWD_GRADS_ONLY, dx_only = flags & QLORA_BWD_DX_FROM_WS;
    if (grads_only && dx_only) return QLORA_ERR_INVALID_ARG;
    if (X8 ? (X != nullptr || !aligned16(X8->q) || !aligned16(X8->scales)) : !aligned16(X)) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(dH) || !aligned16(A) || !aligned16(B) || !aligned16_or_null(U_saved)) return QLORA_ERR_INVALID_ARG;
    if (dx_only ? !aligned16(dX) : (!aligned16(dA) || !aligned16(dB))) return QLORA_ERR_INVALID_ARG;
    if (!grads_only && !aligned16_or_null(dX)) return QLORA_ERR_INVALID_ARG;
    const int64_t d_out = base.mx ? base.mx->d_out : base.nf4->d_out;
    const int64_t d_in = base.mx ? base.mx->d_in : base.nf4->d_in;
    QL_TRY(check_ws(ws, ws_bytes, mx_bwd_plan(T, d_out, d_in, r).total));
    int* err = nullptr;
    QL_TRY(err_word(&err, st));
    return mx_bwd(base, X, X8, dH, T, A, B, r, alpha / static_cast<float>(r), U_saved, dX, dA, dB, ws,
                  (flags & QLORA_BWD_ACCUMULATE) ? 1 : 0, grads_only ? kBwdGrads : (dx_only ? kBwdDx : kBwdAll), err, st);
}

}  // namespace

// ======================================================================= C ABI

extern "C" {

qlora_status qlora_mxfp4_sizes(int64_t rows, int64_t cols, size_t* codes_bytes, size_t* scale_bytes) {
    if (!codes_bytes || !scale_bytes) return QLORA_ERR_INVALID_ARG;
    QL_TRY(mx_check_dims(rows, cols));
    *codes_bytes = static_cast<size_t>(rows) * cols / 2;
    *scale_bytes = mx_scale_bytes(rows, cols);
    return QLORA_OK;
}

qlora_status mxfp4_quantize(const void* W, qlora_dtype w_dtype, int64_t rows, int64_t cols, uint8_t* codes,
                            uint8_t* scales, cudaStream_t stream) {
    if (!aligned16(W) || !aligned16(codes) || !aligned16(scales)) return QLORA_ERR_INVALID_ARG;
    if (w_dtype != QLORA_F32 && w_dtype != QLORA_BF16) return QLORA_ERR_INVALID_ARG;
    QL_TRY(mx_check_dims(rows, cols));
    const unsigned tiles = static_cast<unsigned>(cdiv(rows, 128) * mx_col_tiles(cols));
    if (w_dtype == QLORA_F32)
        k_mxfp4_quantize<float><<<tiles, 256, 0, stream>>>(static_cast<const float*>(W), rows, cols, codes, scales);
    else
        k_mxfp4_quantize<__nv_bfloat16><<<tiles, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(W), rows, cols,
                                                                   codes, scales);
    QL_LAUNCH_CHECK();
    return QLORA_OK;
}

qlora_status mxfp4_dequantize(const qlora_mxfp4* w, void* W_out, qlora_dtype out_dtype, cudaStream_t stream) {
    if (!aligned16(W_out) || (out_dtype != QLORA_F32 && out_dtype != QLORA_BF16)) return QLORA_ERR_INVALID_ARG;
    QL_TRY(check_mxfp4(w));
    const dim3 grid(static_cast<unsigned>(cdiv(w->d_out, 128) * mx_col_tiles(w->d_in)));
    if (out_dtype == QLORA_F32)
        k_mxfp4_dequant<float><<<grid, 256, 0, stream>>>(w->codes, w->scales, w->d_out, w->d_in,
                                                         static_cast<float*>(W_out));
    else
        k_mxfp4_dequant<__nv_bfloat16><<<grid, 256, 0, stream>>>(w->codes, w->scales, w->d_out, w->d_in,
                                                                 static_cast<__nv_bfloat16*>(W_out));
    QL_LAUNCH_CHECK();
    return QLORA_OK;
}

qlora_status qlora_linear_fwd_mxfp4(const qlora_mxfp4* w, const void* X, int64_t T, const void* A, const void* B,
                                    int32_t r, float alpha, void* H, void* U_save, void* ws, size_t ws_bytes,
                                    cudaStream_t stream) {
    QL_TRY(check_mxfp4(w));
    QL_TRY(mx_check_dims(T, w->d_in));
    if (r < 1 || r > 128) return QLORA_ERR_UNSUPPORTED;
    if (!aligned16(X) || !aligned16(A) || !aligned16(B) || !aligned16(H) || !aligned16_or_null(U_save))
        return QLORA_ERR_INVALID_ARG;
    QL_TRY(check_ws(ws, ws_bytes, mx_fwd_plan(T, w->d_out, w->d_in, r).total));
    int* err = nullptr;
    QL_TRY(err_word(&err, stream));
    return mx_fwd(w, X, T, A, B, r, alpha / static_cast<float>(r), H, U_save, ws, err, stream);
}

qlora_status qlora_linear_bwd_mxfp4(const qlora_mxfp4* w, const void* X, const qlora_act8* X8, const void* dH,
                                    int64_t T, const void* A, const void* B, int32_t r, float alpha,
                                    const void* U_saved, void* dX, float* dA, float* dB, void* ws, size_t ws_bytes,
                                    uint32_t flags, cudaStream_t stream) {
    QL_TRY(check_mxfp4(w));
    return mx_bwd_entry(MxBase{nullptr, w}, X, X8, dH, T, A, B, r, alpha, U_saved, dX, dA, dB, ws, ws_bytes, flags,
                        stream);
}

qlora_status qlora_linear_bwd_act8(const qlora_nf4* w, const qlora_act8* X8, const void* dH, int64_t T, const void* A,
                                   const void* B, int32_t r, float alpha, const void* U_saved, void* dX, float* dA,
                                   float* dB, void* ws, size_t ws_bytes, uint32_t flags, cudaStream_t stream) {
    QL_TRY(check_nf4(w));
    if (!X8) return QLORA_ERR_INVALID_ARG;
    return mx_bwd_entry(MxBase{w, nullptr}, nullptr, X8, dH, T, A, B, r, alpha, U_saved, dX, dA, dB, ws, ws_bytes,
                        flags, stream);
}

qlora_status qlora_act8_sizes(int64_t T, int64_t d_in, size_t* q_bytes, size_t* scale_bytes) {
    if (!q_bytes || !scale_bytes) return QLORA_ERR_INVALID_ARG;
    if (T < 1 || T > kMaxDim || d_in < 64 || d_in % 64 || d_in > kMaxDim) return QLORA_ERR_UNSUPPORTED;
    if (cdiv(T * d_in, 8192) > 0x7FFFFFFFLL) return QLORA_ERR_UNSUPPORTED;                  // grids
    *q_bytes = static_cast<size_t>(T) * d_in;
    *scale_bytes = static_cast<size_t>(T) * d_in / 32;
    return QLORA_OK;
}

qlora_status qlora_act8_quantize(const void* X, qlora_dtype x_dtype, int64_t T, int64_t d_in, int8_t* q,
                                 uint8_t* scales, cudaStream_t stream) {
    if (!aligned16(X) || !aligned16(q) || !aligned16(scales)) return QLORA_ERR_INVALID_ARG;
    if (x_dtype != QLORA_F32 && x_dtype != QLORA_BF16) return QLORA_ERR_INVALID_ARG;
    size_t qb, sb;
    QL_TRY(qlora_act8_sizes(T, d_in, &qb, &sb));
    const int64_t n8 = T * d_in / 8;
    if (x_dtype == QLORA_F32)
        k_act8_quantize<float><<<act8_ctas(n8), 256, 0, stream>>>(static_cast<const float*>(X), n8, q, scales);
    else
        k_act8_quantize<__nv_bfloat16><<<act8_ctas(n8), 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(X), n8, q,
                                                                       scales);
    QL_LAUNCH_CHECK();
    return QLORA_OK;
}

qlora_status qlora_act8_dequantize(const qlora_act8* a, int64_t T, int64_t d_in, void* X_out, qlora_dtype out_dtype,
                                   cudaStream_t stream) {
    if (!a || !aligned16(a->q) || !aligned16(a->scales) || !aligned16(X_out)) return QLORA_ERR_INVALID_ARG;
    if (out_dtype != QLORA_F32 && out_dtype != QLORA_BF16) return QLORA_ERR_INVALID_ARG;
    size_t qb, sb;
    QL_TRY(qlora_act8_sizes(T, d_in, &qb, &sb));
    const int64_t n8 = T * d_in / 8;
    if (out_dtype == QLORA_F32)
        k_act8_dequant<float><<<act8_ctas(n8), 256, 0, stream>>>(a->q, a->scales, n8, static_cast<float*>(X_out));
    else
        k_act8_dequant<__nv_bfloat16><<<act8_ctas(n8), 256, 0, stream>>>(a->q, a->scales, n8,
                                                                      static_cast<__nv_bfloat16*>(X_out));
    QL_LAUNCH_CHECK();
    return QLORA_OK;
}

}  // extern "C"
