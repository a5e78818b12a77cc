// ffn_prefill.cu -- expert FFN for the compute-bound regime (moe_expert_ffn,
// MOE_MODE_PREFILL): grouped GEMMs on the 5th-generation tensor cores.
//
// Computes what the decode path computes -- gate/up GEMM -> SwiGLU -> down
// GEMM -> affinity scale over the expert-sorted rows -- in the shape of the
// sorted grouped-GEMM prefill of the Nemotron-H layer
// (spark_model/layers/nemotron_moe.rs, `prefill` step 5) and the fused
// prefill producer of the aiter gfx950 PR (gate/up, SiLU, down and the
// routing-weight multiply in one pipeline), with the block-scaled E4M3FN
// weights of the FP8 MoE decode kernel page decoded tile by tile to 16-bit
// MMA operands: f16 in the gate/up GEMM, bf16 in the down GEMM.
//
// gate/up runs on f16 operands, which take one conversion instruction and one
// f16x2 multiply per code pair.  A pre-pass (x16_kernel) copies x to f16 with
// each row scaled by a power of two 2^k_t that puts its largest magnitude in
// [2^14, 2^15) (exact: f16 has 11 significant bits to bf16's 8); the weights
// become f16(e4m3 * s * 2^ka), ka a power of two per row block chosen from its
// largest block scale so that every product is an f16 normal.  The epilogue
// multiplies the accumulators by 2^-ka * 2^-k_t before SwiGLU.  Both
// roundings (s * 2^ka to f16, the product to f16) are of 2^-12 relative, finer
// than the bf16(e4m3 * s) of the down GEMM.
//
// One persistent kernel per GEMM (gate/up, then down); each CTA owns one SM
// and walks a list of output tiles built on the device from the expert
// offsets (no host sync; under MOE_MODE_HYBRID the experts with at most
// FfnArgs::row_split rows are left to the weight-streaming kernels).  A tile
// is 128 weight rows x up to 192 token rows:
//  * swap-AB: the weights are the M=128 operand A, the tokens the N operand B,
//    so the FP8 decode writes tensor memory, not shared memory;
//  * warp 0: the weight tile's FP8 bytes by TMA into a 64 KB ring of four
//    stages: 64 reduction columns for gate/up (64-byte rows and swizzle), 128
//    for down (128-byte rows and swizzle);
//  * the token rows into the 128-byte-swizzled K-major layout the MMA reads:
//    gate/up gathers rows of the f16 copy of x through sorted_route with
//    cp.async on warps 2-7
//    (the per-SM gather rate grows with the number of issuing warps; each
//    thread keeps its rows' token indices in registers for the whole tile and
//    arrives on the stage's mbarrier when its copies land); down loads
//    contiguous rows of h as one 2-D TMA tile from warp 2 -- up to 4 stages
//    ahead;
//  * transform warps 8-15: each thread owns one TMEM lane (one weight row);
//    gate/up: warps 8-11 decode M-tile 0 and 12-15 M-tile 1, all 64 columns
//    of a step; down: two warps per lane quarter, half the columns each.  A
//    thread decodes its FP8 codes (gate/up: f16(e4m3 * s * 2^ka); down:
//    bf16(e4m3 * s)) as soon as the weight stage lands, then waits for its A
//    slot and stores them with tcgen05.st (A operand, two 16-bit values per
//    column) into a ring of four 32-column
//    units (two gate/up steps or four down steps, one barrier pair per step);
//  * warp 1 issues tcgen05.mma warp-uniformly, one elected lane per four
//    MMAs (kind::f16, A in TMEM, B in shared memory, fp32 accumulator D in
//    TMEM: gate/up uses both 192-column regions for one tile's two M-tiles,
//    down alternates between them so the epilogue of one output block
//    overlaps the MMAs of the next);
//  * epilogue warps 4-7 (in gate/up, between their gathers: after issuing the
//    next item's first stages): tcgen05.ld 16x256b of D; in each 32-lane
//    quarter of a gate/up M-tile, lanes 0-15 hold the gate rows and lanes
//    16-31 the up rows of the same 16 features, so a thread receives gate and
//    up of the same (feature, token) pairs and applies SwiGLU in place; the
//    down epilogue multiplies by the route weight.  bf16 results go through
//    a 128-byte-swizzled staging tile (stmatrix.trans, one row per token) and
//    leave as 32-row TMA tensor stores, the last rows as 16-byte stores.
// Every mbarrier wait is bounded; an expired wait sets a CTA-wide abort flag
// and every role runs to the end without waiting, so the CTA always reaches
// the TMEM de-allocation.
#include <algorithm>
#include <cstring>

#include "device_common.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int kSB = 4;                      // token stages
constexpr int kNMax = 192;                  // token rows per tile (MMA N)
constexpr int kBStage = kNMax * 128;        // token rows x 64 bf16 (128-byte swizzle)
constexpr int kWRing = 64 * 1024;           // FP8 weight ring (128 reduction columns per TMA stage)
constexpr int kOHalf = kNMax * 128;         // staging tile: two halves of 64 features (128-byte swizzled rows)
constexpr int kOStoreRows = 32;             // rows per TMA store of the staging tile
// Per mode: M-tiles (128 weight rows each) per step, weight stage bytes and
// depths of the weight ring and of the bf16 A ring in TMEM.  The A ring holds
// kSA units of 32 columns (one M-tile's 64 reduction columns); a gate/up step
// fills two units, a down step one, and the kSS = kSA / MT step slots each
// have one full/done barrier pair (one wait and one commit per step for the
// MMA warp, which shares its scheduler with transform warps).
template <int MODE> struct Cfg;
// Warp roles (transform and epilogue warps sit on their TMEM lane quarter, warp % 4):
// 0 weight TMA, 1 MMA, 2-7 token rows (gate/up) or 2 token TMA (down), 4-7
// epilogue, 8-15 FP8 transform.
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpTok = 2, kWarpEpi = 4, kWarpXform = 8;
// gate/up: the token rows are gathered by warps 2-7 (the epilogue warps 4-7
// gather too: one cp.async stream per warp caps the per-SM gather rate).
constexpr int kGatherThreads = 192;
constexpr int kNumWarps = 16;
constexpr int kThreads = kNumWarps * 32;
constexpr int kXformWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kDRegion = kNMax;        // two accumulator regions of kNMax columns
constexpr uint32_t kACol = 2 * kNMax;       // A ring: the remaining columns
constexpr int kARing = (kTmemCols - kACol) / 32;  // A units of 32 columns (4 with 192-row tiles)
constexpr int kDownGroup = 16;                  // output blocks sharing a resident token tile (down)
constexpr int kScales = 512;                    // staged block scales per item (floats)

enum Mode { kGateUp = 0, kDown = 1 };

// gate/up: a step feeds two M-tiles (gate and up rows of 128 features, two
// accumulator regions); down: one M-tile per step, regions double-buffered.
// A weight stage holds 128 reduction columns (128-byte rows) and feeds two
// 64-column MMA steps.
// kWCols: reduction columns (bytes of a row) per weight stage.  gate/up uses
// 64-column stages (one MMA step each, 64-byte swizzle), so that three of the
// ring's four stages are in flight while one is decoded: the weights of a
// gate/up step are consumed at twice the rate of a down step.
template <> struct Cfg<0> {
    static constexpr int MT = 2, kWCols = 64, kWStage = 2 * 128 * kWCols, kSW = kWRing / kWStage, kSA = kARing,
                         kSS = kSA / MT;
};
template <> struct Cfg<1> {
    static constexpr int MT = 1, kWCols = 128, kWStage = 128 * kWCols, kSW = kWRing / kWStage, kSA = kARing,
                         kSS = kSA / MT;
};
constexpr int kSWMax = 8, kSAMax = kARing;
static_assert(Cfg<0>::kSW <= kSWMax && Cfg<1>::kSW <= kSWMax, "weight ring depth");

struct Barriers {
    uint64_t w_full[kSWMax], w_empty[kSWMax];
    uint64_t b_full[kSB], b_done[kSB];
    uint64_t a_full[kSAMax], a_done[kSAMax];
    uint64_t d_full[2], d_empty[2], final_bar;
    uint32_t tmem_base;
    int abort_flag;
};

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// Tensor maps of one launch, indexed by part: [0] the routed experts, [1] the
// shared expert.
struct PrefillMaps {
    CUtensorMap w0[2];   // gate (gate/up launch) or down (down launch) weights
    CUtensorMap w1[2];   // up weights (gate/up launch)
    CUtensorMap act[2];  // rows of h (down launch)
    CUtensorMap out[2];  // staging-tile stores: h (gate/up) or y (down)
};

// Shape of one part (routed or shared) in one launch.
struct PartCfg {
    int I;         // intermediate size
    int KB;        // MMA steps (64 columns) per output block
    int KB128;     // 128-column scale blocks per output block
    int FB;        // output blocks of 128 features (gate/up: their gate and up rows)
    int GFB;       // output blocks per item
    bool resident; // down: the token tile stays in the ring across the item
};

template <int MODE>
__device__ __forceinline__ PartCfg part_cfg(const FfnArgs& a, int pt) {
    PartCfg c;
    c.I = pt ? a.sh.inter : a.ex.inter;
    const int Kred = MODE == kGateUp ? a.H : c.I;
    c.KB = Kred / 64;
    c.KB128 = Kred / 128;
    c.FB = MODE == kGateUp ? c.I / 128 : a.H / 128;
    // The down GEMM keeps its token tile resident across a group of output
    // blocks when the whole reduction fits in the token ring.
    c.resident = MODE == kDown && c.KB <= kSB;
    c.GFB = c.resident ? kDownGroup : 1;
    return c;
}

// One work item: a token tile of one expert and a group of consecutive
// output blocks (128 weight rows each) that share that token tile.
struct Tile {
    int e;    // expert within its part
    int pt;   // part: 0 routed, 1 shared
    long p0;  // first row (sorted position, or token for the shared expert)
    int n;    // rows in the tile (<= kNMax)
    int fb0;  // first output block
    int nfb;  // output blocks in the group
};

// Number of items of an expert with n_e rows.
__device__ __forceinline__ int items_of(long n_e, int groups) {
    return static_cast<int>((n_e + kNMax - 1) / kNMax) * groups;
}

// Rows of expert e of the combined list (e == E: the shared expert).
__device__ __forceinline__ long expert_len(const FfnArgs& a, int e, long R, bool* bad) {
    if (e >= a.ex.n) return a.T;
    const long b = a.offsets[e], f = a.offsets[e + 1];
    if (b < 0 || f < b || f > R) {
        *bad = true;
        return 0;
    }
    return f - b;
}

// Rows of expert e this launch processes: none for a routed expert left to
// the decode form (at most a.row_split rows when a.row_split > 0).
__device__ __forceinline__ long expert_rows_here(const FfnArgs& a, int e, long R, bool* bad) {
    const long n = expert_len(a, e, R, bad);
    return (a.row_split > 0 && e < a.ex.n && n <= a.row_split) ? 0 : n;
}

__device__ __forceinline__ int num_experts(const FfnArgs& a) { return a.ex.n + (a.sh.n ? 1 : 0); }

// Item list over the routed experts then the shared one: pre[] holds the
// exclusive prefix of items over experts.  Returns the total.
__device__ int build_tiles(const FfnArgs& a, int groups_r, int groups_s, int* pre) {
    const int E = num_experts(a);
    const long R = static_cast<long>(a.T) * a.K;
    const int per = (E + blockDim.x - 1) / blockDim.x;
    const int e0 = min(E, static_cast<int>(threadIdx.x) * per), e1 = min(E, e0 + per);
    int local = 0;
    bool bad = false;
    for (int e = e0; e < e1; ++e) local += items_of(expert_rows_here(a, e, R, &bad), e < a.ex.n ? groups_r : groups_s);
    if (bad) report_status(a.status, MOE_STATUS_BAD_MAP);
    // Block exclusive scan of `local`.
    __shared__ int warp_sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int x = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    int run = (warp ? warp_sums[warp - 1] : 0) + x - local;
    for (int e = e0; e < e1; ++e) {
        pre[e] = run;
        run += items_of(expert_rows_here(a, e, R, &bad), e < a.ex.n ? groups_r : groups_s);
    }
    const int total = warp_sums[nw - 1];
    if (threadIdx.x == 0) pre[E] = total;
    __syncthreads();
    return total;
}

template <int MODE>
__device__ __forceinline__ Tile tile_of(const FfnArgs& a, const int* pre, int item) {
    int lo = 0, hi = num_experts(a) - 1;  // last e with pre[e] <= item
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= item)
            lo = mid;
        else
            hi = mid - 1;
    }
    Tile t;
    t.pt = lo >= a.ex.n ? 1 : 0;
    t.e = t.pt ? 0 : lo;
    const PartCfg c = part_cfg<MODE>(a, t.pt);
    const int groups = (c.FB + c.GFB - 1) / c.GFB;
    const int local = item - pre[lo];
    const int tt = local / groups;
    const int fg = local - tt * groups;
    const long base = t.pt ? 0 : a.offsets[lo];
    const long n_e = t.pt ? a.T : a.offsets[lo + 1] - base;
    t.p0 = base + static_cast<long>(tt) * kNMax;
    t.n = static_cast<int>(min(static_cast<long>(kNMax), n_e - static_cast<long>(tt) * kNMax));
    t.fb0 = fg * c.GFB;
    t.nfb = min(c.GFB, c.FB - t.fb0);
    return t;
}

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Barriers* B, int32_t* status) {
    return mbar_wait_or_abort(bar, parity, &B->abort_flag, status);
}

// bf16(e4m3 * s) for two codes (down GEMM).
__device__ __forceinline__ uint32_t decode_scaled(uint16_t codes, float s) {
    const uint32_t h = e4m3x2_to_f16x2(codes);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf16x2(f.x * s, f.y * s);
}

// f16(e4m3 * s2) for two codes (gate/up GEMM): the exact conversion of the
// codes to f16, then one f16x2 multiply by the scale pair s2 (a power-of-two
// multiple of the block scale, so every product is an f16 normal).
__device__ __forceinline__ uint32_t decode_scaled_f16(uint16_t codes, uint32_t s2) {
    const uint32_t h = e4m3x2_to_f16x2(codes);
    __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&s2));
    return *reinterpret_cast<uint32_t*>(&r);
}

// Power-of-two exponent ka of a gate/up weight row block whose largest block
// scale is smax: 448 * smax * 2^ka lies in [2^14, 2^15), so the f16 operands
// e4m3 * s * 2^ka of every block stay below the f16 maximum, and those of
// blocks whose scale is at least 2^-10 smax stay f16 normals (the smallest
// nonzero E4M3FN magnitude is 2^-9, the largest 448).  The transform and the
// epilogue compute it from the same scales, so they agree exactly.
__device__ __forceinline__ int f16_row_exponent(float smax) {
    const float m = 448.f * smax;
    if (!(m > 0.f) || !(m < INFINITY)) return 0;
    const int e = (__float_as_int(m) >> 23) & 0xFF;  // biased exponent (0 for a subnormal m)
    return max(-120, min(120, 141 - e));
}

__device__ __forceinline__ float exp2_int(int k) {  // 2^k for -126 <= k <= 127
    return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// Largest |x| bit pattern (sign cleared) among the 8 bf16 of a 16-byte vector.
__device__ __forceinline__ uint32_t absmax_bf16x8_bits(const uint4& v) {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16);
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2_times(uint32_t w, float up) {
    __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
    return *reinterpret_cast<uint32_t*>(&h);
}

// x16[t] = f16(x[t] * 2^k_t), xinv[t] = 2^-k_t, with k_t putting the row's
// largest magnitude in [2^14, 2^15) (k_t = 0 for an all-zero row).  f16 has
// 11 significant bits to bf16's 8, so every element within 2^-28 of its
// row's largest is copied exactly; the gate/up epilogue multiplies by xinv.
// One warp per row, 16-byte loads and stores.
__global__ void __launch_bounds__(256) x16_kernel(const uint16_t* __restrict__ x, int T, int H,
                                                  uint16_t* __restrict__ x16, float* __restrict__ xinv) {
    const int t = static_cast<int>((static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= T) return;
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(t) * H);
    uint4* dst = reinterpret_cast<uint4*>(x16 + static_cast<size_t>(t) * H);
    const int nv = H >> 3;
    uint32_t amax = 0;
    for (int v = lane; v < nv; v += 32) amax = max(amax, absmax_bf16x8_bits(__ldg(src + v)));
    amax = __reduce_max_sync(0xffffffffu, amax);
    int k = 0;
    if (amax) {
        const int eb = static_cast<int>(amax >> 7);  // biased exponent of the largest magnitude (0: subnormal)
        k = min(127, 14 - (eb ? eb - 127 : -127));
    }
    const float up = exp2_int(k);
    if (lane == 0) xinv[t] = ldexpf(1.f, -k);
    for (int v = lane; v < nv; v += 32) {
        uint4 w = __ldg(src + v);
        w.x = bf16x2_to_f16x2_times(w.x, up);
        w.y = bf16x2_to_f16x2_times(w.y, up);
        w.z = bf16x2_to_f16x2_times(w.z, up);
        w.w = bf16x2_to_f16x2_times(w.w, up);
        dst[v] = w;
    }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ PrefillMaps M, const FfnArgs a) {
    using C = Cfg<MODE>;
    constexpr int MT = C::MT, kSW = C::kSW, kSA = C::kSA, kWStage = C::kWStage;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = align1024(smem_raw);
    uint8_t* w_ring = sm;                              // kSW x kWStage (64 KB)
    uint8_t* b_ring = w_ring + kWRing;                 // kSB x 24 KB
    uint8_t* otile = b_ring + kSB * kBStage;           // 2 x [kNMax][128 B] bf16 output staging
    Barriers* B = reinterpret_cast<Barriers*>(otile + 2 * kOHalf);
    int* row_tok = reinterpret_cast<int*>(B + 1);      // [kNMax] activation row of each tile row
                                                       // (down with out_acc: token of each column)
    float* col_w = reinterpret_cast<float*>(row_tok + kNMax);  // [kNMax] route weight of each column (down)
    float* sc_sm = col_w + kNMax;                              // [kScales] block scales of the item
    int* pre = reinterpret_cast<int*>(sc_sm + kScales);        // [E + 2]

    const int H = a.H;
    const bool has_sh = a.sh.n != 0;
    const long R = static_cast<long>(a.T) * a.K;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kSW; ++s) {
            mbar_init(&B->w_full[s], 1);
            mbar_init(&B->w_empty[s], kXformWarps);
        }
        for (int s = 0; s < kSB; ++s) {
            mbar_init(&B->b_full[s], MODE == kGateUp ? kGatherThreads : 1);
            mbar_init(&B->b_done[s], 1);
        }
        for (int s = 0; s < C::kSS; ++s) {
            // One barrier pair per step slot (the MT units of one step): all
            // eight transform warps fill it, one commit frees it.
            mbar_init(&B->a_full[s], kXformWarps);
            mbar_init(&B->a_done[s], 1);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(&B->d_full[d], 1);
            mbar_init(&B->d_empty[d], 4);
        }
        mbar_init(&B->final_bar, 1);
        B->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(&B->tmem_base, kTmemCols);
        tc_fence_before();
    }
    int total;
    {
        const PartCfg cr = part_cfg<MODE>(a, 0), cs = part_cfg<MODE>(a, 1);
        total = build_tiles(a, (cr.FB + cr.GFB - 1) / cr.GFB, has_sh ? (cs.FB + cs.GFB - 1) / cs.GFB : 1,
                            pre);  // contains __syncthreads
    }
    tc_fence_after();
    const uint32_t tmem = B->tmem_base;
    if (MODE == kGateUp && threadIdx.x == 0) grid_dependency_launch();

    if (warp == kWarpTma) {
        // ------------------------------------------------ FP8 weight tiles (TMA, evict-first)
        if (lane == 0) {
            for (int pt = 0; pt < (has_sh ? 2 : 1); ++pt) {
                tma_prefetch_desc(&M.w0[pt]);
                if (MODE == kGateUp) tma_prefetch_desc(&M.w1[pt]);
            }
            const uint64_t policy = l2_evict_first_policy();
            long g = 0;  // weight stages (128 columns)
            for (int item = blockIdx.x; item < total; item += gridDim.x) {
                const Tile t = tile_of<MODE>(a, pre, item);
                const PartCfg pc = part_cfg<MODE>(a, t.pt);
                for (int f = 0; f < t.nfb; ++f) {
                    const int fb = t.fb0 + f;
                    const int nstages = (MODE == kGateUp ? H : pc.I) / C::kWCols;
                    for (int kw = 0; kw < nstages; ++kw, ++g) {
                        const int s = static_cast<int>(g % kSW);
                        if (g >= kSW) wait_bar(&B->w_empty[s], static_cast<uint32_t>((g / kSW - 1) & 1), B, a.status);
                        uint8_t* dst = w_ring + s * kWStage;
                        mbar_arrive_expect_tx(&B->w_full[s], kWStage);
                        if (MODE == kGateUp) {
                            const int row = t.e * pc.I + fb * 128;  // 128 gate rows, 128 up rows
                            tma_load_2d_hint(dst, &M.w0[t.pt], &B->w_full[s], kw * C::kWCols, row, policy);
                            tma_load_2d_hint(dst + kWStage / 2, &M.w1[t.pt], &B->w_full[s], kw * C::kWCols, row,
                                             policy);
                        } else {
                            tma_load_2d_hint(dst, &M.w0[t.pt], &B->w_full[s], kw * C::kWCols, t.e * H + fb * 128,
                                             policy);
                        }
                    }
                }
            }
        }
    } else if (warp >= kWarpTok && warp < kWarpXform) {
        // ------------------------------------------------ token rows (warps 2-7) and epilogue (warps 4-7)
        // gate/up: rows of x gathered through sorted_route by cp.async (16 bytes
        // per copy) by warps 2-7, each thread arriving on the stage barrier when
        // its copies land; warps 4-7 then run the item's epilogue.  down:
        // contiguous rows of h as one 2-D TMA tile (warp 2), epilogue on warps 4-7.
        // Padding rows of the last MMA column group are left stale: column j of
        // D depends on token row j only, and the epilogue drops those columns.
        const bool epi_warp = warp >= kWarpEpi;
        const int q = warp & 3;
        const int et = threadIdx.x - kWarpEpi * 32;  // 0..127
        const uint32_t otile_u32 = smem_u32(otile);
        int uses[2] = {0, 0};
        int tc = 0;
        // Epilogue of one item (warps 4-7).
        auto epilogue = [&](const Tile& t) {
            const PartCfg pc = part_cfg<MODE>(a, t.pt);
            // gate/up: D of a gate (up) row is 2^ka_g (2^ka_u) x 2^k_t times the
            // true sum (scaled weights, scaled x rows): fg, fu undo the first,
            // col_w[c] = xinv of column c's token the second.
            float fg = 1.f, fu = 1.f;
            if (MODE == kGateUp) {
                const ExpertsView& ev = t.pt ? a.sh : a.ex;
                const size_t off = (static_cast<size_t>(t.e) * (pc.I / 128) + t.fb0) * pc.KB128;
                float mg = 0.f, mu = 0.f;
                for (int i = lane; i < pc.KB128; i += 32) {
                    mg = fmaxf(mg, __ldg(ev.s_gate + off + i));
                    mu = fmaxf(mu, __ldg(ev.s_up + off + i));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    mg = fmaxf(mg, __shfl_xor_sync(0xffffffffu, mg, o));
                    mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, o));
                }
                fg = exp2_int(-f16_row_exponent(mg));
                fu = exp2_int(-f16_row_exponent(mu));
                named_barrier_sync(4, 128);
                for (int c = et; c < t.n; c += 128) {
                    int tk = 0;
                    if (t.pt) {
                        tk = static_cast<int>(t.p0 + c);
                    } else {
                        const int rt = a.sorted_route[t.p0 + c];
                        tk = (rt >= 0 && rt < R) ? rt / a.K : 0;
                    }
                    col_w[c] = __ldg(a.xinv + tk);
                }
                named_barrier_sync(4, 128);
            }
            if (MODE == kDown) {
                // Route weight of every column of the item, staged once (1 for
                // the shared expert).
                named_barrier_sync(4, 128);
                for (int c = et; c < t.n; c += 128) {
                    float wv = 1.f;
                    int tk = static_cast<int>(t.p0 + c);
                    if (!t.pt) {
                        const int rt = a.sorted_route[t.p0 + c];
                        const bool okr = rt >= 0 && rt < R;
                        wv = okr ? a.topk_w[rt] : 0.f;
                        tk = okr ? rt / a.K : -1;
                    }
                    col_w[c] = wv;
                    if (a.out_acc) row_tok[c] = tk;
                }
                named_barrier_sync(4, 128);
            }
            for (int f = 0; f < t.nfb; ++f, ++tc) {
                for (int mt = 0; mt < MT; ++mt) {
                    const int r = MODE == kGateUp ? mt : (tc & 1);  // accumulator region
                    const bool ok = wait_bar(&B->d_full[r], static_cast<uint32_t>(uses[r] & 1), B, a.status);
                    ++uses[r];
                    tc_fence_after();
                    if (mt == 0) {
                        // The staging tile is free once the previous block's row
                        // copies have read it.
                        bulk_wait_read0();
                        named_barrier_sync(4, 128);
                    }
                    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q) << 16) + r * kDRegion;
                    for (int c0 = 0; c0 < t.n; c0 += 32) {
                        if (MODE == kGateUp) {
                            // Lanes 32q+0..15 hold the gate rows, 32q+16..31 the up rows of
                            // features 16q..16q+15 of the M-tile: thread t gets gate and up
                            // of the same (feature, token) pairs.
                            uint32_t gv[16], uv[16];
                            tmem_ld16x256b_x4(tl + c0, gv);
                            tmem_ld16x256b_x4(tl + (16u << 16) + c0, uv);
                            tmem_ld_wait();
                            if (!ok) continue;
                            // Column scales of this thread's tokens c0 + 8g + 2(t%4) + {0, 1}.
                            float2 cs[4];
#pragma unroll
                            for (int gq = 0; gq < 4; ++gq)
                                cs[gq] = *reinterpret_cast<const float2*>(col_w + c0 + 8 * gq + 2 * (lane & 3));
                            uint32_t pk[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                float hv[2];
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const float cc = j ? cs[k >> 1].y : cs[k >> 1].x;
                                    const float z = __uint_as_float(gv[2 * k + j]) * (fg * cc);
                                    const float u = __uint_as_float(uv[2 * k + j]) * (fu * cc);
                                    hv[j] = __fdividef(z, 1.0f + __expf(-z)) * u;
                                }
                                pk[k] = pack_bf16x2(hv[0], hv[1]);
                            }
                            // Features mt*64 + 16q + 8(i&1) + 0..7 of matrix i: half mt, 16-byte
                            // chunk 2q + (i&1) of the token's 128-byte row.
                            const int row = c0 + 8 * (lane >> 4) + (lane & 7);
                            const uint32_t o = otile_u32 + mt * kOHalf + row * 128;
                            const uint32_t fc = 2 * q + ((lane >> 3) & 1);
                            stmatrix_x4_trans(o + ((fc ^ (row & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
                            stmatrix_x4_trans(o + 16 * 128 + ((fc ^ (row & 7)) << 4), pk[4], pk[5], pk[6], pk[7]);
                        } else {
                            uint32_t dv[2][16];
                            tmem_ld16x256b_x4(tl + c0, dv[0]);
                            tmem_ld16x256b_x4(tl + (16u << 16) + c0, dv[1]);
                            tmem_ld_wait();
                            if (!ok) continue;
                            // Route weights of this thread's tokens c0 + 8g + 2(t%4) + {0, 1}.
                            float2 wv[4];
#pragma unroll
                            for (int gq = 0; gq < 4; ++gq)
                                wv[gq] = *reinterpret_cast<const float2*>(col_w + c0 + 8 * gq + 2 * (lane & 3));
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                uint32_t pk[8];
#pragma unroll
                                for (int gq = 0; gq < 4; ++gq) {
                                    const uint32_t* d = dv[hf] + 4 * gq;
                                    pk[2 * gq] = pack_bf16x2(__uint_as_float(d[0]) * wv[gq].x,
                                                             __uint_as_float(d[1]) * wv[gq].y);
                                    pk[2 * gq + 1] = pack_bf16x2(__uint_as_float(d[2]) * wv[gq].x,
                                                                 __uint_as_float(d[3]) * wv[gq].y);
                                }
                                // Features 32q + 16hf + 8(i&1) + 0..7: half q/2, chunk
                                // 4(q&1) + 2hf + (i&1).
                                const int row = c0 + 8 * (lane >> 4) + (lane & 7);
                                const uint32_t o = otile_u32 + (q >> 1) * kOHalf + row * 128;
                                const uint32_t fc = 4 * (q & 1) + 2 * hf + ((lane >> 3) & 1);
                                stmatrix_x4_trans(o + ((fc ^ (row & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
                                stmatrix_x4_trans(o + 16 * 128 + ((fc ^ (row & 7)) << 4), pk[4], pk[5], pk[6],
                                                  pk[7]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B->d_empty[r]);
                }
                const int fb = t.fb0 + f;
                if (MODE == kDown && a.out_acc) {
                    // Fused combine: each row's 128 features (bf16, route weight
                    // applied) are added into its token's fp32 output row, 8
                    // features per thread as two vector reductions.
                    named_barrier_sync(4, 128);
                    for (int i = et; i < t.n * 16; i += 128) {
                        const int rr = i >> 4, hh = (i >> 3) & 1, c8 = i & 7;
                        const int tk = row_tok[rr];
                        if (tk < 0) continue;
                        const uint4 v =
                            *reinterpret_cast<const uint4*>(otile + hh * kOHalf + rr * 128 + ((c8 ^ (rr & 7)) << 4));
                        float* dst = a.out_acc + static_cast<size_t>(tk) * H + fb * 128 + hh * 64 + c8 * 8;
                        red_add_f32x4(dst, __uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                                      __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
                        red_add_f32x4(dst + 4, __uint_as_float(v.z << 16), __uint_as_float(v.z & 0xFFFF0000u),
                                      __uint_as_float(v.w << 16), __uint_as_float(v.w & 0xFFFF0000u));
                    }
                    continue;  // the next block's barrier orders these reads before its staging writes
                }
                // Staging tile -> global: TMA tensor stores of 32 rows x 64 features,
                // and 16-byte thread stores for the rows past the last full group.
                fence_proxy_async_smem();
                named_barrier_sync(4, 128);
                const int n32 = t.n / kOStoreRows;
                if (et < 2 * n32) {
                    const int hh = et & 1, k = et >> 1;
                    tma_store_2d(&M.out[t.pt], otile_u32 + hh * kOHalf + k * kOStoreRows * 128,
                                 fb * 128 + hh * 64, static_cast<int>(t.p0) + k * kOStoreRows);
                }
                bulk_commit();
                const size_t stride = MODE == kGateUp ? pc.I : H;
                uint16_t* base = MODE == kGateUp ? (t.pt ? a.h_sh : a.h) : (t.pt ? a.y_sh : a.y);
                uint16_t* dst = base + static_cast<size_t>(t.p0) * stride + fb * 128;
                for (int i = n32 * kOStoreRows * 16 + et; i < t.n * 16; i += 128) {
                    const int rr = i >> 4, hh = (i >> 3) & 1, c8 = i & 7;
                    *reinterpret_cast<uint4*>(dst + rr * stride + hh * 64 + c8 * 8) =
                        *reinterpret_cast<const uint4*>(otile + hh * kOHalf + rr * 128 + ((c8 ^ (rr & 7)) << 4));
                }
            }
        };
        if (MODE == kGateUp) {
            // Thread lt copies 16-byte chunk ch of rows r0 + 24k, keeping those
            // rows' token indices in registers for the whole tile; the 128-byte
            // swizzle of those rows is the same for every k.
            const int lt = threadIdx.x - kWarpTok * 32;  // 0..191
            const int r0 = lt >> 3, ch = lt & 7;
            const uint32_t cch = static_cast<uint32_t>((ch ^ (r0 & 7)) << 4);
            constexpr int kRowsPerThread = (kNMax + kGatherThreads / 8 - 1) / (kGatherThreads / 8);
            uint32_t tok[kRowsPerThread];
            long g = 0;
            Tile prev{};
            bool have_prev = false;
            for (int item = blockIdx.x; item < total; item += gridDim.x) {
                const Tile t = tile_of<MODE>(a, pre, item);
                const PartCfg pc = part_cfg<MODE>(a, t.pt);
                named_barrier_sync(2, kGatherThreads);
                bool bad = false;
                for (int r = lt; r < t.n; r += kGatherThreads) {
                    int tk = 0;
                    const long p = t.p0 + r;
                    if (t.pt) {
                        tk = static_cast<int>(p);
                    } else {
                        const int rt = a.sorted_route[p];
                        if (rt >= 0 && rt < R)
                            tk = rt / a.K;
                        else
                            bad = true;
                    }
                    row_tok[r] = tk;
                }
                if (bad) report_status(a.status, MOE_STATUS_BAD_MAP);
                named_barrier_sync(2, kGatherThreads);
#pragma unroll
                for (int k = 0; k < kRowsPerThread; ++k)
                    tok[k] = r0 + 24 * k < t.n ? row_tok[r0 + 24 * k] : 0u;
                for (int kb = 0; kb < pc.KB; ++kb, ++g) {
                    const int s = static_cast<int>(g % kSB);
                    if (g >= kSB) wait_bar(&B->b_done[s], static_cast<uint32_t>((g / kSB - 1) & 1), B, a.status);
                    const uint32_t bdst = smem_u32(b_ring + s * kBStage) + r0 * 128 + cch;
                    const uint16_t* xs = a.x16 + kb * 64 + ch * 8;
#pragma unroll
                    for (int k = 0; k < kRowsPerThread; ++k)
                        if (r0 + 24 * k < t.n)
                            cp_async16(bdst + k * 24 * 128, xs + static_cast<size_t>(tok[k]) * H, 16u);
                    cp_async_arrive_noinc(&B->b_full[s]);
                    // The previous item's MMAs are done once the ring has turned
                    // over: run its epilogue while these loads are in flight.
                    if (epi_warp && have_prev && kb == min(kSB, pc.KB) - 1) {
                        epilogue(prev);
                        have_prev = false;
                    }
                }
                prev = t;
                have_prev = true;
            }
            if (epi_warp && have_prev) epilogue(prev);
            cp_async_wait<0>();
        } else if (!epi_warp) {
            const int lt = threadIdx.x - kWarpTok * 32;  // 0..63
            grid_dependency_wait();  // h comes from the gate/up grid
            if (lt == 0)
                for (int pt = 0; pt < (has_sh ? 2 : 1); ++pt) tma_prefetch_desc(&M.act[pt]);
            long g = 0;
            for (int item = blockIdx.x; item < total; item += gridDim.x) {
                const Tile t = tile_of<MODE>(a, pre, item);
                const PartCfg pc = part_cfg<MODE>(a, t.pt);
                for (int kb = 0; kb < pc.KB; ++kb, ++g) {
                    const int s = static_cast<int>(g % kSB);
                    if (g >= kSB) wait_bar(&B->b_done[s], static_cast<uint32_t>((g / kSB - 1) & 1), B, a.status);
                    if (lt == 0) {
                        mbar_arrive_expect_tx(&B->b_full[s], kBStage);
                        tma_load_2d(b_ring + s * kBStage, &M.act[t.pt], &B->b_full[s], kb * 64,
                                    static_cast<int>(t.p0));
                    }
                }
            }
        } else {
            for (int item = blockIdx.x; item < total; item += gridDim.x) epilogue(tile_of<MODE>(a, pre, item));
        }
        if (epi_warp) bulk_wait0();
    } else if (warp >= kWarpXform) {
        // ------------------------------------------------ transform: FP8 -> bf16 -> TMEM (A)
        // gate/up: warp (q, mt) owns lane quarter q of M-tile mt and all 64 codes
        // of a step; down: warp (q, hf) owns lane quarter q and half of the codes.
        const int q = warp & 3, hi = (warp - kWarpXform) >> 2;
        const int xt = threadIdx.x - kWarpXform * 32;           // 0..255
        const int row = 32 * q + lane;  // TMEM lane = weight row of the M-tile
        constexpr int NW = MODE == kGateUp ? 32 : 16;           // words (bf16 pairs) per thread per step
        long g = 0;                                             // MMA steps (64 columns)
        for (int item = blockIdx.x; item < total; item += gridDim.x) {
            const Tile t = tile_of<MODE>(a, pre, item);
            const PartCfg pc = part_cfg<MODE>(a, t.pt);
            const ExpertsView& ev = t.pt ? a.sh : a.ex;
            const int KB = pc.KB, KB128 = pc.KB128;
            // Block scales of the item, staged once: gate/up -> [gate, up][KB128],
            // down -> [output block][KB128].
            named_barrier_sync(3, kXformWarps * 32);
            if (MODE == kGateUp) {
                const size_t off = (static_cast<size_t>(t.e) * (pc.I / 128) + t.fb0) * KB128;
                for (int i = xt; i < 2 * KB128; i += kXformWarps * 32)
                    sc_sm[i] = __ldg((i < KB128 ? ev.s_gate : ev.s_up) + off + (i % KB128));
            } else {
                for (int i = xt; i < t.nfb * KB128; i += kXformWarps * 32) {
                    const int f = i / KB128, k = i - f * KB128;
                    sc_sm[i] = __ldg(ev.s_down + (static_cast<size_t>(t.e) * (H / 128) + (t.fb0 + f)) * KB128 + k);
                }
            }
            named_barrier_sync(3, kXformWarps * 32);
            // Source row in the weight stage.  gate/up: in the lane quarter of
            // warp q, lanes 0-15 hold the gate rows and lanes 16-31 the up rows
            // of features 16q .. 16q+15 of the M-tile (so the eight lanes of a
            // shared-memory phase read eight different rows).
            const bool up_row = MODE == kGateUp && (lane & 16);
            const int srow = MODE == kGateUp ? hi * 64 + 16 * q + (lane & 15) : row;
            const int sub = up_row ? kWStage / 2 : 0;
            const int c0 = MODE == kGateUp ? 0 : 2 * hi;  // first 16-byte chunk of this thread in a step
            // gate/up: the f16 operands of this row are e4m3 * s * 2^ka, with ka
            // from the largest block scale of the row's block row (gate or up).
            float pa = 1.f;
            if (MODE == kGateUp) {
                const float* sr = sc_sm + (up_row ? KB128 : 0);
                float m = 0.f;
                for (int i = 0; i < KB128; ++i) m = fmaxf(m, sr[i]);
                pa = exp2_int(f16_row_exponent(m));
            }
            for (int f = 0; f < t.nfb; ++f) {
                const float* scr = sc_sm + (MODE == kGateUp ? (up_row ? KB128 : 0) : f * KB128);
                for (int kb = 0; kb < KB; ++kb, ++g) {
                    constexpr int kSPS = C::kWCols / 64;  // MMA steps per weight stage
                    const long gw = g / kSPS;  // weight stage holding this step
                    const long u = MODE == kGateUp ? 2 * g + hi : g;  // A unit of this warp's work
                    const int sw = static_cast<int>(gw % kSW), sa = static_cast<int>(u % kSA);
                    const bool ok1 = wait_bar(&B->w_full[sw], static_cast<uint32_t>((gw / kSW) & 1), B, a.status);
                    uint32_t v[NW];
                    if (ok1) {
                        const float sc = scr[kb >> 1];
                        __half2 s2h = __float2half2_rn(sc * pa);
                        const uint32_t s2 = *reinterpret_cast<uint32_t*>(&s2h);
                        const uint8_t* base = w_ring + sw * kWStage + sub + srow * C::kWCols;
#pragma unroll
                        for (int c = 0; c < NW / 8; ++c) {
                            // 16-byte chunk of this thread's row in the stage, placed by
                            // the TMA swizzle of the stage's row width (128 or 64 bytes).
                            const int chunk = static_cast<int>(g % kSPS) * 4 + c0 + c;
                            const int phys = C::kWCols == 128 ? (chunk ^ (srow & 7)) : (chunk ^ ((srow >> 1) & 3));
                            const uint4 w = *reinterpret_cast<const uint4*>(base + (phys << 4));
                            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (MODE == kGateUp) {
                                    v[c * 8 + 2 * k] = decode_scaled_f16(static_cast<uint16_t>(ws[k] & 0xFFFFu), s2);
                                    v[c * 8 + 2 * k + 1] = decode_scaled_f16(static_cast<uint16_t>(ws[k] >> 16), s2);
                                } else {
                                    v[c * 8 + 2 * k] = decode_scaled(static_cast<uint16_t>(ws[k] & 0xFFFFu), sc);
                                    v[c * 8 + 2 * k + 1] = decode_scaled(static_cast<uint16_t>(ws[k] >> 16), sc);
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < NW; ++k) v[k] = 0;
                    }
                    if (g % kSPS == kSPS - 1) release_stage(&B->w_empty[sw], lane);
                    else __syncwarp();
                    // The A slot is free once the MMAs that last read it have
                    // completed; the decode above overlapped that wait.
                    const int ss = static_cast<int>(g % C::kSS);  // step slot of this step
                    if (g >= C::kSS) wait_bar(&B->a_done[ss], static_cast<uint32_t>((g / C::kSS - 1) & 1), B, a.status);
                    tc_fence_after();
                    const uint32_t acol = kACol + sa * 32 + (MODE == kGateUp ? 0 : hi * 16);
                    if constexpr (MODE == kGateUp)
                        tmem_st32(tmem + (static_cast<uint32_t>(32 * q) << 16) + acol, v);
                    else
                        tmem_st16(tmem + (static_cast<uint32_t>(32 * q) << 16) + acol, v);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B->a_full[ss]);
                }
            }
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------ MMA issuer
        // The whole warp runs the loop with warp-uniform operands; one elected
        // lane issues each tcgen05 instruction.  Operands are bases computed
        // once plus per-slot offsets.
        const uint64_t bdesc0 = umma_desc_sw128(smem_u32(b_ring));
        const uint32_t a_base = tmem + kACol;
        // gate/up: the operands of every ring position, computed once.
        uint64_t bq[kSB][4];   // B descriptor of token stage s, K=16 step k
        uint32_t aq[kSAMax][4];  // A column of unit u, K=16 step k
#pragma unroll
        for (int s2 = 0; s2 < kSB; ++s2)
#pragma unroll
            for (int k = 0; k < 4; ++k) bq[s2][k] = bdesc0 + static_cast<uint64_t>((s2 * kBStage) >> 4) + 2 * k;
#pragma unroll
        for (int u = 0; u < kSAMax; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) aq[u][k] = a_base + u * 32 + 8 * k;
        long ga = 0, gb = 0;
        int uses[2] = {0, 0};
        int tc = 0;
        for (int item = blockIdx.x; item < total; item += gridDim.x) {
            const Tile t = tile_of<MODE>(a, pre, item);
            const PartCfg pc = part_cfg<MODE>(a, t.pt);
            const int KB = pc.KB;
            const bool resident = pc.resident;
            const int N = (t.n + 15) & ~15;
            // gate/up: f16 operands (decoded weights and the f16 copy of x); down: bf16.
            const uint32_t idesc = MODE == kGateUp ? umma_idesc_f16(128, N) : umma_idesc_bf16(128, N);
            for (int f = 0; f < t.nfb; ++f, ++tc) {
                // Accumulator regions of this output block: both (gate/up) or one (down).
                const int r0 = MODE == kGateUp ? 0 : (tc & 1);
                for (int mt = 0; mt < MT; ++mt) {
                    const int r = r0 + mt;
                    if (uses[r] >= 1)
                        wait_bar(&B->d_empty[r], static_cast<uint32_t>((uses[r] - 1) & 1), B, a.status);
                    ++uses[r];
                }
                tc_fence_after();
                const bool last = f == t.nfb - 1;
                const uint32_t d_base = tmem + r0 * kDRegion;
                bool grouped = false;
                constexpr bool kGroupable = MODE == kGateUp && kSB == 4 && C::kSS == 2 && kSA == 4;
                if constexpr (kGroupable) grouped = KB % kSB == 0 && (ga % kSB) == 0;
                if constexpr (kGroupable) if (grouped) {
                    // gate/up in groups of kSB steps aligned with the token ring
                    // (so also with the two A step slots): every ring index and
                    // barrier parity of a group is a compile-time function of
                    // one value, and each step is two waits, two fences and one
                    // issue of eight MMAs with two commits.
                    for (int kb = 0; kb < KB; kb += kSB, ga += kSB, gb += kSB) {
                        const uint32_t pb = static_cast<uint32_t>((ga / kSB) & 1);
                        const uint32_t pa = static_cast<uint32_t>((ga / C::kSS) & 1);
#pragma unroll
                        for (int j = 0; j < kSB; ++j) {
                            const int ss = j & 1;
                            const bool okb = wait_bar(&B->b_full[j], pb, B, a.status);
                            const bool oka = wait_bar(&B->a_full[ss], pa ^ static_cast<uint32_t>(j >> 1), B, a.status);
                            tc_fence_after();
                            // Token rows written by cp.async (generic proxy) are read by the MMA
                            // (async proxy).
                            fence_proxy_async_smem();
                            if (okb && oka) {
                                umma_ts_step2_commit2_elect(d_base, d_base + kDRegion, aq[2 * ss], aq[2 * ss + 1],
                                                            bq[j], idesc, (kb | j) ? 1u : 0u, &B->a_done[ss],
                                                            &B->b_done[j]);
                            } else {
                                umma_commit_elect(&B->a_done[ss]);
                                umma_commit_elect(&B->b_done[j]);
                            }
                        }
                    }
                }
                if (!grouped)
                for (int kb = 0; kb < KB; ++kb, ++ga) {
                    const long g_b = resident ? gb + kb : gb;  // token stage of this step
                    const int sb = static_cast<int>(g_b % kSB);
                    const bool okb = wait_bar(&B->b_full[sb], static_cast<uint32_t>((g_b / kSB) & 1), B, a.status);
                    const uint64_t bdesc = bdesc0 + static_cast<uint64_t>((sb * kBStage) >> 4);
                    // The step's A units (one per M-tile) arrive together.
                    const int ss = static_cast<int>(ga % C::kSS);
                    const bool oka = wait_bar(&B->a_full[ss], static_cast<uint32_t>((ga / C::kSS) & 1), B, a.status);
                    tc_fence_after();
                    // Token rows written by cp.async (generic proxy) are read by the MMA
                    // (async proxy).
                    if (MODE == kGateUp) fence_proxy_async_smem();
                    if (okb && oka) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const int sa = static_cast<int>((ga * MT + mt) % kSA);  // TMEM slot of the unit
                            if (mt == MT - 1)
                                umma_ts_f16_x4_commit_elect(d_base + mt * kDRegion, a_base + sa * 32, bdesc, idesc,
                                                            kb > 0 ? 1u : 0u, &B->a_done[ss]);
                            else
                                umma_ts_f16_x4_elect(d_base + mt * kDRegion, a_base + sa * 32, bdesc, idesc,
                                                     kb > 0 ? 1u : 0u);
                        }
                    } else {
                        umma_commit_elect(&B->a_done[ss]);
                    }
                    if (!resident) {
                        umma_commit_elect(&B->b_done[sb]);
                        ++gb;
                    } else if (last) {
                        umma_commit_elect(&B->b_done[sb]);
                    }
                }
                for (int mt = 0; mt < MT; ++mt) umma_commit_elect(&B->d_full[r0 + mt]);
            }
            if (resident) gb += KB;
        }
        // Every MMA has completed once this barrier flips.
        umma_commit_elect(&B->final_bar);
        mbar_wait(&B->final_bar, 0, a.status);
        __syncwarp();
    }
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    // When launched as a programmatic dependent of the weight-streaming down
    // kernel on the same stream (launch_ffn_prefill's gateup_after_decode),
    // gate/up overlaps that grid's tail without reading anything it writes;
    // waiting for it here, at the end, makes this grid's completion -- which
    // the down GEMM and later launches wait for -- imply that grid's.  A no-op
    // for a normal launch (the hybrid form now runs the two forms on two
    // streams instead).
    if (MODE == kGateUp && threadIdx.x == 0) grid_dependency_wait();
}

__global__ void __launch_bounds__(256) acc_to_bf16_kernel(const float* __restrict__ acc, long n8,
                                                          uint16_t* __restrict__ out) {
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n8;
         i += static_cast<long>(gridDim.x) * blockDim.x) {
        const float4 a0 = reinterpret_cast<const float4*>(acc)[2 * i];
        const float4 a1 = reinterpret_cast<const float4*>(acc)[2 * i + 1];
        uint4 r;
        r.x = pack_bf16x2(a0.x, a0.y);
        r.y = pack_bf16x2(a0.z, a0.w);
        r.z = pack_bf16x2(a1.x, a1.y);
        r.w = pack_bf16x2(a1.z, a1.w);
        reinterpret_cast<uint4*>(out)[i] = r;
    }
}

size_t prefill_smem(int E) {
    return 1024 + kWRing + kSB * kBStage + 2 * kOHalf + sizeof(Barriers) + 2 * kNMax * 4 + kScales * 4 +
           (E + 2) * 4 + 64;
}

int num_sms() {
    static int sms = 0;
    if (!sms) {
        int dev = 0;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (sms <= 0) sms = 148;
    }
    return sms;
}

}  // namespace

cudaError_t launch_acc_to_bf16(const float* acc, long n, uint16_t* out, cudaStream_t stream) {
    const long n8 = n / 8;
    long blocks = (n8 + 255) / 256;
    if (blocks > 148L * 32) blocks = 148L * 32;
    if (blocks < 1) return cudaSuccess;
    acc_to_bf16_kernel<<<static_cast<int>(blocks), 256, 0, stream>>>(acc, n8, out);
    return cudaGetLastError();
}

bool ffn_prefill_supported(int H, int I) { return H % 128 == 0 && I % 128 == 0 && prefill_smem(MOE_MAX_E) <= 227 * 1024; }

cudaError_t launch_ffn_prefill(const FfnArgs& a, cudaStream_t stream, bool x16_done, bool gateup_after_decode) {
    if (a.identity || !a.x16 || !a.xinv) return cudaErrorInvalidValue;
    const uint64_t E = static_cast<uint64_t>(a.ex.n), I = a.ex.inter, H = a.H;
    const uint64_t R = static_cast<uint64_t>(a.T) * a.K, T = static_cast<uint64_t>(a.T);
    PrefillMaps mg, md;  // gate/up and down launches
    memset(&mg, 0, sizeof(mg));
    memset(&md, 0, sizeof(md));
    cudaError_t err = make_tmap_u8_2d(&mg.w0[0], a.ex.w_gate, E * I, H, Cfg<0>::kWCols, 128, Cfg<0>::kWCols);
    if (err == cudaSuccess) err = make_tmap_u8_2d(&mg.w1[0], a.ex.w_up, E * I, H, Cfg<0>::kWCols, 128, Cfg<0>::kWCols);
    if (err == cudaSuccess) err = make_tmap_bf16_2d(&mg.out[0], a.h, R, I, 64, kOStoreRows);
    if (err == cudaSuccess) err = make_tmap_u8_2d(&md.w0[0], a.ex.w_down, E * H, I, 128, 128);
    if (err == cudaSuccess) err = make_tmap_bf16_2d(&md.act[0], a.h, R, I, 64, kNMax);
    if (err == cudaSuccess && !a.out_acc) err = make_tmap_bf16_2d(&md.out[0], a.y, R, H, 64, kOStoreRows);
    if (a.sh.n) {
        const uint64_t Is = a.sh.inter;
        if (err == cudaSuccess) err = make_tmap_u8_2d(&mg.w0[1], a.sh.w_gate, Is, H, Cfg<0>::kWCols, 128, Cfg<0>::kWCols);
        if (err == cudaSuccess) err = make_tmap_u8_2d(&mg.w1[1], a.sh.w_up, Is, H, Cfg<0>::kWCols, 128, Cfg<0>::kWCols);
        if (err == cudaSuccess) err = make_tmap_bf16_2d(&mg.out[1], a.h_sh, T, Is, 64, kOStoreRows);
        if (err == cudaSuccess) err = make_tmap_u8_2d(&md.w0[1], a.sh.w_down, H, Is, 128, 128);
        if (err == cudaSuccess) err = make_tmap_bf16_2d(&md.act[1], a.h_sh, T, Is, 64, kNMax);
        if (err == cudaSuccess && !a.out_acc) err = make_tmap_bf16_2d(&md.out[1], a.y_sh, T, H, 64, kOStoreRows);
    }
    if (err != cudaSuccess) return err;
    const size_t smem = prefill_smem(a.ex.n);
    err = cudaFuncSetAttribute(prefill_kernel<kGateUp>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(prefill_kernel<kDown>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    const int grid = a.sm_limit > 0 ? std::min(a.sm_limit, num_sms()) : num_sms();
    if (!x16_done) {
        err = launch_x16(a, stream);
        if (err != cudaSuccess) return err;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // gate/up: a programmatic dependent of the preceding kernel only when the
    // caller asks for it (the preceding kernel being the weight-streaming down
    // GEMM of the same call).
    cfg.numAttrs = gateup_after_decode ? 1 : 0;
    err = cudaLaunchKernelEx(&cfg, prefill_kernel<kGateUp>, mg, a);
    if (err != cudaSuccess) return err;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_kernel<kDown>, md, a);
}

cudaError_t launch_x16(const FfnArgs& a, cudaStream_t stream) {
    x16_kernel<<<static_cast<unsigned>((static_cast<long>(a.T) * 32 + 255) / 256), 256, 0, stream>>>(a.x, a.T, a.H,
                                                                                                   a.x16, a.xinv);
    return cudaGetLastError();
}

}  // namespace moe
