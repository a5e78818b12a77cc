// rows.cu -- rows sorted by expert and back (moe_permute, moe_unpermute) and
// the gradients (moe_unpermute_bwd), for bf16, f16 and f32 rows.
//
// Everything here is indexed by token: inv_route gives the sorted position of
// each of a token's K routes, so a token's row is read once for its K copies
// (permute), its K sorted rows are summed in slot order by one thread per
// 16-byte column (unpermute, a fixed order), and no two tokens write the same
// row.  A position outside [0, T*K) is skipped: -1 silently, anything else
// with MOE_STATUS_BAD_MAP.  All of it is bound by memory: a few operations for
// every element read or written.
//
// Each kernel has two forms: rows whose bytes are a multiple of 16 are moved by
// aligned 16-byte vectors, other rows by 4-byte words, by elements or by shifted
// blocks of 16 bytes (rows.cuh), whichever was fastest there.
#include <type_traits>

#include "launch_after.cuh"
#include "rows.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // slots of a token whose rows are in flight together

// The sorted position of a route, or -1; flags corrupt entries.
__device__ __forceinline__ int32_t position(const int32_t* __restrict__ inv, long r, long R, bool* bad) {
    const int32_t p = __ldg(inv + r);
    if (p >= 0 && p < R) return p;
    if (p != -1) *bad = true;
    return -1;
}

// Zeros in the sorted rows [*n_rows, R) (grid-stride over the whole grid).
__device__ __forceinline__ void zero_tail(const int32_t* __restrict__ n_rows, long R, long row_bytes, void* rows) {
    if (!n_rows) return;
    long n = __ldg(n_rows);
    if (n >= R) return;
    n = n < 0 ? 0 : n;
    char* o = static_cast<char*>(rows);
    const long begin = n * row_bytes, end = R * row_bytes;  // multiples of 2
    for (long b = (begin & ~15L) + (static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x) * 16; b < end;
         b += static_cast<long>(gridDim.x) * blockDim.x * 16) {
        if (b >= begin && b + 16 <= end) {
            *reinterpret_cast<uint4*>(o + b) = make_uint4(0, 0, 0, 0);
        } else {
            for (long i = b; i < b + 16; i += 2)
                if (i >= begin && i < end) *reinterpret_cast<uint16_t*>(o + i) = 0;
        }
    }
}

// x_sorted[inv[t, j]] = x[t].  One thread per 16-byte column of a token: one
// load, K stores.  Bound by the writes: 8192 bf16 rows of 4096, top-10, in 121
// us, 6.1 TB/s of the 738 MB it cannot do without.
__global__ void __launch_bounds__(kThreads) permute_kernel(const char* __restrict__ x,
                                                           const int32_t* __restrict__ inv,
                                                           const int32_t* __restrict__ n_rows, int T, int K,
                                                           long row_bytes, const FastDiv vecs,
                                                           char* __restrict__ x_sorted, int32_t* __restrict__ status) {
    const long R = static_cast<long>(T) * K, total = static_cast<long>(T) * vecs.d;
    bool bad = false;
    grid_dependency_wait();
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long>(gridDim.x) * blockDim.x) {
        const long t = vecs.div(i), c = i - t * vecs.d;
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(x) + i);
#pragma unroll 4
        for (int j = 0; j < K; ++j) {
            const int32_t p = position(inv, t * K + j, R, &bad);
            if (p >= 0) reinterpret_cast<uint4*>(x_sorted + p * row_bytes)[c] = v;
        }
    }
    zero_tail(n_rows, R, row_bytes, x_sorted);
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

// The same for rows that are no multiple of 16 bytes, by 4-byte words on the
// alignment of the rows written (RowWords).  A thread has W words of a token,
// a warp's width apart; where rows may start within a word (HALF) it keeps
// them as they are and shifted by half a word, for either start.
template <bool HALF, int W>
__global__ void __launch_bounds__(kThreads) permute_words_kernel(const char* __restrict__ x,
                                                                 const int32_t* __restrict__ inv,
                                                                 const int32_t* __restrict__ n_rows, int T, int K,
                                                                 long row_bytes, const FastDiv tiles,
                                                                 char* __restrict__ x_sorted,
                                                                 int32_t* __restrict__ status) {
    const long R = static_cast<long>(T) * K, total = static_cast<long>(T) * tiles.d * (W > 1 ? 32 : 1);
    bool bad = false;
    grid_dependency_wait();
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long>(gridDim.x) * blockDim.x) {
        const long tile = W > 1 ? i >> 5 : i, t = tiles.div(tile);
        const int k0 = static_cast<int>(tile - t * tiles.d) * (W > 1 ? 32 * W : 1) + (W > 1 ? threadIdx.x & 31 : 0);
        const RowWords<HALF> src(x, t, row_bytes, T * row_bytes);
        uint32_t same[W], other[W];
#pragma unroll
        for (int u = 0; u < W; ++u) {
            same[u] = src.word(k0 + 32 * u);
            if (HALF) other[u] = src.beside(k0 + 32 * u);
        }
        if (HALF) {
#pragma unroll
            for (int u = 0; u < W; ++u) other[u] = src.shifted(same[u], other[u]);
        }
#pragma unroll 2
        for (int j = 0; j < K; ++j) {
            const int32_t p = position(inv, t * K + j, R, &bad);
            if (p < 0) continue;
            const long at = p * row_bytes;
            const bool alike = !HALF || (at & 2) == src.lead;
#pragma unroll
            for (int u = 0; u < W; ++u) store_word<HALF>(x_sorted, at, row_bytes, k0 + 32 * u, alike ? same[u] : other[u]);
        }
    }
    zero_tail(n_rows, R, row_bytes, x_sorted);
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}


// The positions and weights of slots j0 .. j0 + n of a token, -1 for those that
// add nothing.
template <int B>
__device__ __forceinline__ void slot_batch(const int32_t* __restrict__ inv, const float* __restrict__ w, long r, long R,
                                           int n, int32_t (&p)[B], float (&wj)[B], bool* bad) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
        p[b] = -1;
        wj[b] = 1.f;
        if (b < n) {
            p[b] = position(inv, r + b, R, bad);
            if (w) wj[b] = __ldg(w + r + b);
            if (wj[b] == 0.f) p[b] = -1;
        }
    }
}

// out[t] = sum_j w[t, j] y[inv[t, j]] (+ y_shared[t]).  One thread per 16-byte
// column of a token; slots in batches: all positions, then all rows, then the
// sums in slot order, so that the loads of a batch (of at most B) are in flight
// together.  8192 bf16 rows of 4096, top-10: 135 us, which the ring below takes
// to 111 us; here are the calls that are too small for it, bound by latency.
template <class E, int B>
__global__ void __launch_bounds__(kThreads) unpermute_kernel(const char* __restrict__ y_sorted,
                                                             const int32_t* __restrict__ inv,
                                                             const float* __restrict__ w,
                                                             const char* __restrict__ y_shared, int T, int K,
                                                             int batch, long row_bytes, const FastDiv vecs,
                                                             char* __restrict__ out, int32_t* __restrict__ status) {
    constexpr int N = kVec<E>;
    const long R = static_cast<long>(T) * K, total = static_cast<long>(T) * vecs.d;
    bool bad = false;
    grid_dependency_wait();
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long>(gridDim.x) * blockDim.x) {
        const long t = vecs.div(i), c = i - t * vecs.d;
        float acc[N];
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = 0.f;
        for (int j0 = 0; j0 < K; j0 += batch) {
            int32_t p[B];
            float wj[B];
            slot_batch(inv, w, t * K + j0, R, K - j0 < batch ? K - j0 : batch, p, wj, &bad);
            uint4 v[B];
#pragma unroll
            for (int b = 0; b < B; ++b)
                if (p[b] >= 0) v[b] = __ldg(reinterpret_cast<const uint4*>(y_sorted + p[b] * row_bytes) + c);
#pragma unroll
            for (int b = 0; b < B; ++b)
                if (p[b] >= 0) add_weighted<E>(acc, v[b], wj[b]);
        }
        if (y_shared) {
            float f[N];
            unpack<E>(__ldg(reinterpret_cast<const uint4*>(y_shared) + i), f);
#pragma unroll
            for (int n = 0; n < N; ++n) acc[n] += f[n];
        }
        reinterpret_cast<uint4*>(out)[i] = pack<E>(acc);
    }
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

// The same for rows that are no multiple of 16 bytes, by 4-byte words where they
// are a multiple of 4 and by elements (2 bytes) otherwise; a thread has W of
// them, a warp's width apart.
template <class E, class Word, int W>
__global__ void __launch_bounds__(kThreads) unpermute_words_kernel(const char* __restrict__ y_sorted,
                                                                   const int32_t* __restrict__ inv,
                                                                   const float* __restrict__ w,
                                                                   const char* __restrict__ y_shared, int T, int K,
                                                                   int batch, long row_bytes, const FastDiv tiles,
                                                                   char* __restrict__ out,
                                                                   int32_t* __restrict__ status) {
    constexpr int B = kBatch;
    const long R = static_cast<long>(T) * K, total = static_cast<long>(T) * tiles.d * (W > 1 ? 32 : 1);
    constexpr int N = sizeof(Word) / sizeof(E);
    const int words = static_cast<int>(row_bytes / sizeof(Word));
    bool bad = false;
    grid_dependency_wait();
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long>(gridDim.x) * blockDim.x) {
        const long tile = W > 1 ? i >> 5 : i, t = tiles.div(tile);
        const int k0 = static_cast<int>(tile - t * tiles.d) * (W > 1 ? 32 * W : 1) + (W > 1 ? threadIdx.x & 31 : 0);
        auto load = [&](const char* row, Word (&v)[W]) {
#pragma unroll
            for (int u = 0; u < W; ++u)
                v[u] = k0 + 32 * u < words ? __ldg(reinterpret_cast<const Word*>(row) + k0 + 32 * u) : Word(0);
        };
        float acc[W][N];
#pragma unroll
        for (int u = 0; u < W; ++u)
#pragma unroll
            for (int n = 0; n < N; ++n) acc[u][n] = 0.f;
        auto add = [&](const Word (&v)[W], float by) {
#pragma unroll
            for (int u = 0; u < W; ++u) {
                E e[N];
                memcpy(e, &v[u], sizeof(Word));
#pragma unroll
                for (int n = 0; n < N; ++n) acc[u][n] = fmaf(by, elem_to_float(e[n]), acc[u][n]);
            }
        };
        for (int j0 = 0; j0 < K; j0 += batch) {
            int32_t p[B];
            float wj[B];
            slot_batch(inv, w, t * K + j0, R, K - j0 < batch ? K - j0 : batch, p, wj, &bad);
            Word v[B][W];
#pragma unroll
            for (int b = 0; b < B; ++b)
                if (p[b] >= 0) load(y_sorted + p[b] * row_bytes, v[b]);
#pragma unroll
            for (int b = 0; b < B; ++b)
                if (p[b] >= 0) add(v[b], wj[b]);
        }
        if (y_shared) {
            Word v[W];
            load(y_shared + t * row_bytes, v);
            add(v, 1.f);
        }
#pragma unroll
        for (int u = 0; u < W; ++u) {
            E e[N];
#pragma unroll
            for (int n = 0; n < N; ++n) e[n] = elem_from_float<E>(acc[u][n]);
            Word o;
            memcpy(&o, e, sizeof(Word));
            if (k0 + 32 * u < words) reinterpret_cast<Word*>(out + t * row_bytes)[k0 + 32 * u] = o;
        }
    }
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

// ---------------------------------------------------------------- unpermute through shared memory
//
// The same sums for long rows and many tokens.  The loads of unpermute_kernel
// keep a thread's registers busy until they arrive; here one block per SM keeps
// up to 200 KB of row pieces in flight by bulk copies into rings of stages in
// shared memory, and kTeams teams of eight warps, each with a ring of its own,
// sum them from there, one 16-byte column a thread.  A stage is a piece of
// 512 * m bytes of up to kGroup rows of each of 8 / m tokens, where m warps
// take a token (m = 8 for rows of a multiple of 4 KB); tokens with more rows take
// several stages.  A team's kProducers warps issue its stages in turn, each a
// stage's positions ahead.
//
// Waiting on a barrier's phase by its parity needs the phase before it to be
// over.  A team's consumers take the stages in order, so they have seen that
// one themselves.  A producer that fills a stage the n-th time has filled,
// kProducers steps before, one that had to be consumed after this stage's
// (n-2)-th filling, because there are at least kProducers stages.
//
// A copy moves whole 16-byte blocks: the piece of a row, rounded out to them.
// Rows that are no multiple of 16 bytes start anywhere in their slots: there a
// thread takes every 32nd 4-byte word of its warp's 512 bytes, which needs no
// shift unless the row starts within a word, and no bank twice.
//
// 8192 bf16 rows of 4096, top-10: 111 us, 6.6 TB/s of 739 MB, with 73 % of the
// issue slots in use (two teams 118 us, one 155 us: the sums of 16-bit rows
// need the warps); of 4095: 120 us, bound by instructions.

constexpr int kConsumers = 8;  // warps of a team
constexpr int kTeams = 3;
constexpr int kProducers = 2;  // warps of a team
constexpr int kRingThreads = kTeams * (kConsumers + kProducers) * 32;
constexpr int kMaxStages = 12;
constexpr int kGroup = 4;
constexpr int kRingBytes = 212 * 1024 / kTeams / 128 * 128;  // of a team
// Room before and after a piece for the blocks that shifted columns reach into.
constexpr int kShiftPad = 64;
static_assert(kConsumers * kGroup <= 32, "a lane for every row of a stage");
static_assert(kRingBytes / (kConsumers * kGroup * (512 + kShiftPad)) >= kProducers, "the ring has too few stages");
// Taken for rows of at least kRingMinRow bytes and sorted rows of so many bytes
// in all, where it overtakes the plain kernel, which starts faster.  Plain kernel
// against ring, us, the same call again and again (up to about 100 MB from L2):
//   bf16 x 4096, top-1:   32 MB 17.6 / 17.0   64 MB 43.8 / 32.3   160 MB 97 / 75
//                top-10:  48 MB  9.3 /  9.6   64 MB 11.6 / 11.9    96 MB 23.8 / 19.0
//                top-16:  48 MB  8.8 /  9.2   64 MB 10.2 / 12.4    96 MB 19.9 / 17.0
//   f32 x 4096,  top-1:   32 MB 15.5 / 15.6   64 MB 40.2 / 29.5   160 MB 90 / 68
//                top-10:  48 MB  7.3 /  7.9   64 MB  9.0 /  9.7    96 MB 22.1 / 17.4
//   bf16 x 4095, top-1:   16 MB 17.4 / 12.9   32 MB 30.2 / 22.8   160 MB 166 / 102
//                top-10:  16 MB  6.8 /  5.8   32 MB 11.7 /  8.9   160 MB 63 / 35
//                top-16:  32 MB 10.3 / 11.1   48 MB 15.0 / 11.4   160 MB 54 / 31
// With one or two rows a token it pays earlier than the rule says.  Rows of 2 KB
// that do not start on 16 bytes are better off without it for most K, which the
// rule does not look at (bf16 x 1030: top-4 64 MB 20.2 / 22.4, 96 MB 33.8 / 33.4;
// top-10 32 MB 8.3 / 13.8, 160 MB 45.7 / 49.4; f32 x 1031, top-10 96 MB 24.7 /
// 27.3), and rows of 512 bytes always (134 MB 31.6 / 33.2).
constexpr long kRingMinRow = 1024;
constexpr long kRingMinBytes = 64L << 20, kRingMinBytesShift = 24L << 20;

struct RingMeta {
    float w;
    int at;  // byte of the slot where the piece's first row byte is, or -1: no row
};

struct RingHead {
    uint64_t full[kMaxStages], empty[kMaxStages];
    RingMeta meta[kMaxStages][32];  // a producer's lane for every row
};
constexpr int kRingHead = (sizeof(RingHead) * kTeams + 16 + 127) / 128 * 128;

struct RingArgs {
    const char* y;
    const int32_t* inv;
    const float* w;
    const char* shared;  // or NULL
    char* out;
    int32_t* status;
    int T, K;
    int rows, groups, group;  // rows = K (+ 1 for y_shared), in `groups` groups of at most `group`
    int m, tokens;            // warps of a token, tokens of a stage (8 / m)
    int slot, stages;         // bytes of a row piece's slot, stages of a ring
    long R, row_bytes, items;
    FastDiv pieces;           // pieces of a token
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// A piece of a token's output row: its first byte (SHIFT: on a 4-byte boundary
// of the output, so up to 2 bytes before the row) and the row's bytes in it.
struct Piece {
    long begin, from, to;
    template <bool SHIFT>
    static __device__ __forceinline__ Piece of(const RingArgs& a, long t, long q) {
        const long size = a.m * 512L;
        const long begin = q * size - (SHIFT ? (t * a.row_bytes) & 3 : 0);
        return {begin, begin > 0 ? begin : 0, begin + size < a.row_bytes ? begin + size : a.row_bytes};
    }
};

// The row that a producer's lane copies for one stage.
struct RingRow {
    long t;
    int q, j;   // piece; slot of the token (-1: none)
    int32_t p;  // as loaded, not looked at before it is needed
    float w;
};

__device__ __forceinline__ RingRow ring_row(const RingArgs& a, long item, int group, int lane) {
    RingRow r;
    const long tb = a.pieces.div(item);
    const int sub = lane / a.group, j = group * a.group + lane % a.group;
    r.t = tb * a.tokens + sub;
    r.q = static_cast<int>(item - tb * a.pieces.d);
    r.j = item < a.items && sub < a.tokens && r.t < a.T && j < a.rows ? j : -1;
    r.p = -1;
    r.w = 1.f;
    if (r.j >= 0 && j < a.K) {
        r.p = __ldg(a.inv + r.t * a.K + j);
        if (a.w) r.w = __ldg(a.w + r.t * a.K + j);
    }
    return r;
}

template <bool SHIFT>
__device__ __forceinline__ void ring_issue(const RingArgs& a, const RingRow& r, RingHead* head, char* slots, int stage,
                                           int lane, bool* bad) {
    uint32_t bytes = 0;
    const char* src = nullptr;
    char* dst = nullptr;
    RingMeta m{r.w, -1};
    const Piece piece = Piece::of<SHIFT>(a, r.t, r.q);
    if (r.j >= 0 && piece.from < piece.to) {
        const bool shared = r.j == a.K, inside = r.p >= 0 && r.p < a.R;
        if (!shared && !inside && r.p != -1) *bad = true;
        if (shared || (inside && r.w != 0.f)) {
            const char* base = shared ? a.shared : a.y;
            const long total = (shared ? a.T : a.R) * a.row_bytes;
            const long row = (shared ? r.t : r.p) * a.row_bytes;
            const long first = row + piece.from, past = row + piece.to, lo = first & ~15L;
            long hi = (past + 15) & ~15L;
            dst = slots + (stage * (a.tokens * a.group) + lane) * a.slot + (SHIFT ? 16 : 0);
            if (SHIFT && hi > total) {  // the tensor's last bytes are no whole block
                hi = total & ~15L;
                for (long b = hi; b < past; b += 2)
                    *reinterpret_cast<uint16_t*>(dst + (b - lo)) = __ldg(reinterpret_cast<const uint16_t*>(base + b));
            }
            src = base + lo;
            bytes = static_cast<uint32_t>(hi - lo);
            m.at = static_cast<int>(first - lo) + (SHIFT ? 16 : 0);
        }
    }
    head->meta[stage][lane] = m;
    const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(&head->full[stage], all);
    __syncwarp();
    if (bytes) bulk_load(dst, src, bytes, &head->full[stage]);
}

template <class E, bool SHIFT>
__global__ void __launch_bounds__(kRingThreads, 1) unpermute_ring_kernel(const RingArgs a) {
    extern __shared__ __align__(128) char smem[];
    constexpr int N = kVec<E>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool producer = warp >= kTeams * kConsumers;
    const int team = producer ? (warp - kTeams * kConsumers) / kProducers : warp / kConsumers;
    RingHead* head = reinterpret_cast<RingHead*>(smem) + team;
    volatile int* abort_flag = reinterpret_cast<int*>(reinterpret_cast<RingHead*>(smem) + kTeams);
    char* slots = smem + kRingHead + team * kRingBytes;
    if (!producer && warp % kConsumers == 0 && lane == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&head->full[i], 1);
            mbar_init(&head->empty[i], kConsumers);
        }
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    grid_dependency_wait();
    // The items of this team: every step-th from the first.
    const long first_item = static_cast<long>(blockIdx.x) * kTeams + team;
    const long step = static_cast<long>(gridDim.x) * kTeams;
    const long mine = first_item < a.items ? (a.items - first_item + step - 1) / step : 0;
    const long steps = mine * a.groups;

    if (producer) {
        // Step s fills stage s % stages; this warp takes every kProducers-th.
        const int first = warp % kProducers;
        bool bad = false;
        long item = first_item + static_cast<long>(first / a.groups) * step;
        int group = first % a.groups, stage = first;
        long turn = 0;
        RingRow r = ring_row(a, item, group, lane);
        for (long s = first; s < steps; s += kProducers) {
            group += kProducers;
            while (group >= a.groups) {
                group -= a.groups;
                item += step;
            }
            const RingRow next = ring_row(a, item, group, lane);
            const bool ok = turn == 0 || mbar_wait_or_abort(&head->empty[stage], static_cast<uint32_t>((turn - 1) & 1),
                                                            abort_flag, a.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            ring_issue<SHIFT>(a, r, head, slots, stage, lane, &bad);
            r = next;
            for (stage += kProducers; stage >= a.stages; stage -= a.stages) ++turn;
        }
        if (bad) report_status(a.status, MOE_STATUS_BAD_MAP);
    } else {
        // A thread's columns: 16 bytes of its warp's 512, or with SHIFT every 32nd 4-byte word of them.
        const int own = warp % kConsumers, sub = own / a.m, col = (own % a.m) * 512 + lane * (SHIFT ? 4 : 16);
        int stage = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (long item = first_item; ok && item < a.items; item += step) {
            const long tb = a.pieces.div(item), t = tb * a.tokens + sub;
            const Piece piece = Piece::of<SHIFT>(a, t, item - tb * a.pieces.d);
            const long rel = piece.begin + col;  // this thread's first column of the output row
            const bool here = t < a.T && rel < a.row_bytes;
            const int at = SHIFT ? static_cast<int>(piece.begin - piece.from) + col : col;
            float acc[N];
#pragma unroll
            for (int n = 0; n < N; ++n) acc[n] = 0.f;
            for (int group = 0; group < a.groups; ++group) {
                ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&head->full[stage], parity, abort_flag, a.status));
                if (!ok) break;
                if (here) {
                    const RingMeta* meta = head->meta[stage] + sub * a.group;
                    const char* slot = slots + (stage * a.tokens + sub) * (a.group * a.slot);
                    RingMeta mt[kGroup];
                    uint4 v[kGroup];
#pragma unroll
                    for (int g = 0; g < kGroup; ++g) {
                        mt[g].at = -1;
                        if (g < a.group) mt[g] = meta[g];
                        const char* row = slot + g * a.slot;
                        if (mt[g].at >= 0)
                            v[g] = SHIFT ? load_shared_words(row, mt[g].at + at)
                                         : *reinterpret_cast<const uint4*>(row + at);
                    }
#pragma unroll
                    for (int g = 0; g < kGroup; ++g)
                        if (mt[g].at >= 0) add_weighted<E>(acc, v[g], mt[g].w);
                }
                release_stage(&head->empty[stage], lane);
                if (++stage == a.stages) {
                    stage = 0;
                    parity ^= 1;
                }
            }
            if (ok && here) {
                char* o = a.out + t * a.row_bytes + rel;
                if (SHIFT) store_words<E>(o, pack<E>(acc), rel, a.row_bytes);
                else *reinterpret_cast<uint4*>(o) = pack<E>(acc);
            }
        }
    }
    __syncthreads();
    // A wait expired: every copy that was issued lands before the block ends (each wait has its limit).
    if (*abort_flag && !producer && warp % kConsumers == 0 && lane < a.stages)
        for (uint32_t parity = 0; parity < 2; ++parity) mbar_wait(&head->full[lane], parity, a.status);
}

// The sum of dot over the G lanes of a route: a butterfly and, for G > 32, over the warps in order.
template <int G>
__device__ __forceinline__ float lanes_sum(float dot, float* sh) {
#pragma unroll
    for (int off = (G < 32 ? G : 32) / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (G > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = dot;
        __syncthreads();
        dot = 0.f;
        const int first = threadIdx.x / G * (G / 32);
#pragma unroll
        for (int i = 0; i < G / 32; ++i) dot += sh[first + i];
    }
    return dot;
}

// dy[p] = w dout[t], dw = <dout[t], y[p]> for p = inv[t, j].  G threads per
// route and RU routes at a time, each thread with every G-th 16-byte vector,
// U of them at a time.  8192 bf16 rows of 4096, top-10: 215 us, 6.6 TB/s of
// 1.41 GB (dout's row comes from L1 and L2 for all but the first of its K
// routes).  Short rows are bound by what a route costs, about 9 ns an SM.
template <class E, int G, int RU, int U>
__global__ void __launch_bounds__(kThreads) unpermute_bwd_kernel(
    const char* __restrict__ dout, const char* __restrict__ y_sorted, const int32_t* __restrict__ inv,
    const float* __restrict__ w, const int32_t* __restrict__ n_rows, int T, const FastDiv K, long row_bytes,
    char* __restrict__ dy_sorted, float* __restrict__ dw, int32_t* __restrict__ status) {
    constexpr int N = kVec<E>;
    constexpr int PER = kThreads / G;  // routes of a block side by side
    __shared__ float sh[kThreads / 32];
    const long R = static_cast<long>(T) * K.d;
    const int lane = threadIdx.x % G, vecs = static_cast<int>(row_bytes >> 4);
    bool bad = false;
    grid_dependency_wait();
    for (long r0 = static_cast<long>(blockIdx.x) * (PER * RU); r0 < R; r0 += static_cast<long>(gridDim.x) * (PER * RU)) {
        int32_t p[RU];
        float wr[RU], dot[RU];
        const uint4 *d[RU], *y[RU];
#pragma unroll
        for (int i = 0; i < RU; ++i) {
            const long r = r0 + i * PER + threadIdx.x / G;
            p[i] = r < R ? position(inv, r, R, &bad) : -1;
            wr[i] = w && r < R ? __ldg(w + r) : 1.f;
            dot[i] = 0.f;
            d[i] = reinterpret_cast<const uint4*>(dout + K.div(r) * row_bytes);
            y[i] = reinterpret_cast<const uint4*>(y_sorted + p[i] * row_bytes);
        }
        for (int c0 = lane; c0 < vecs; c0 += G * U) {
            uint4 vd[RU][U], vy[RU][U];
#pragma unroll
            for (int i = 0; i < RU; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * G;
                    if (p[i] < 0 || c >= vecs) continue;
                    vd[i][u] = __ldg(d[i] + c);
                    if (dw) vy[i][u] = __ldg(y[i] + c);
                }
#pragma unroll
            for (int i = 0; i < RU; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * G;
                    if (p[i] < 0 || c >= vecs) continue;
                    float fd[N];
                    unpack<E>(vd[i][u], fd);
                    if (dw) {
                        float fy[N];
                        unpack<E>(vy[i][u], fy);
#pragma unroll
                        for (int n = 0; n < N; ++n) dot[i] = fmaf(fd[n], fy[n], dot[i]);
                    }
                    if (dy_sorted) {
#pragma unroll
                        for (int n = 0; n < N; ++n) fd[n] = wr[i] == 0.f ? 0.f : wr[i] * fd[n];
                        reinterpret_cast<uint4*>(dy_sorted + p[i] * row_bytes)[c] = pack<E>(fd);
                    }
                }
        }
        if (dw) {
#pragma unroll
            for (int i = 0; i < RU; ++i) {
                const float sum = lanes_sum<G>(dot[i], sh);
                const long r = r0 + i * PER + threadIdx.x / G;
                if (lane == 0 && r < R) dw[r] = sum;
            }
        }
    }
    if (dy_sorted) zero_tail(n_rows, R, row_bytes, dy_sorted);
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

// The same for rows that are no multiple of 16 bytes: by the 16-byte blocks of
// memory that the sorted row touches, dout's bytes shifted to them (by the same
// distance for all of a route).  Blocks at least one away from the row's ends
// need no check of bounds; the first and the last two are taken with care.
// 8192 bf16 rows of 4095, top-10: 279 us, bound by instructions and latency
// (four vectors at a time cost more warps than they gain: 334 us).
template <class E, int G>
__global__ void __launch_bounds__(kThreads) unpermute_bwd_shift_kernel(
    const char* __restrict__ dout, const char* __restrict__ y_sorted, const int32_t* __restrict__ inv,
    const float* __restrict__ w, const int32_t* __restrict__ n_rows, int T, const FastDiv K, long row_bytes,
    char* __restrict__ dy_sorted, float* __restrict__ dw, int32_t* __restrict__ status) {
    constexpr int N = kVec<E>;
    constexpr int U = 2;
    constexpr int PER = kThreads / G;
    constexpr int S = sizeof(E);
    __shared__ float sh[kThreads / 32];
    const long R = static_cast<long>(T) * K.d;
    const int lane = threadIdx.x % G, bytes = static_cast<int>(row_bytes);
    bool bad = false;
    grid_dependency_wait();
    for (long r0 = static_cast<long>(blockIdx.x) * PER; r0 < R; r0 += static_cast<long>(gridDim.x) * PER) {
        const long r = r0 + threadIdx.x / G;
        const int32_t p = r < R ? position(inv, r, R, &bad) : -1;
        float dot = 0.f;
        if (p >= 0) {
            const float wr = w ? __ldg(w + r) : 1.f;
            const long row = p * row_bytes, drow = K.div(r) * row_bytes;
            const int lead = static_cast<int>(row & 15), blocks = (lead + bytes + 15) >> 4;
            const int by = static_cast<int>((drow - lead) & 15);  // dout's shift
            const uint4* py = reinterpret_cast<const uint4*>(y_sorted + (row - lead));
            const uint4* pd = reinterpret_cast<const uint4*>(dout + (drow - lead - by));
            uint4* po = reinterpret_cast<uint4*>(dy_sorted + (row - lead));
            auto scaled = [&](float (&f)[N]) {
#pragma unroll
                for (int n = 0; n < N; ++n) f[n] = wr == 0.f ? 0.f : wr * f[n];
                return pack<E>(f);
            };
            for (int c0 = 1 + lane; c0 < blocks - 2; c0 += G * U) {
                uint4 vd[U], vn[U], vy[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * G;
                    if (c >= blocks - 2) continue;
                    vd[u] = __ldg(pd + c);
                    if (by) vn[u] = __ldg(pd + c + 1);
                    if (dw) vy[u] = __ldg(py + c);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * G;
                    if (c >= blocks - 2) continue;
                    float fd[N];
                    unpack<E>(by ? shift_blocks(vd[u], vn[u], by) : vd[u], fd);
                    if (dw) {
                        float fy[N];
                        unpack<E>(vy[u], fy);
#pragma unroll
                        for (int n = 0; n < N; ++n) dot = fmaf(fd[n], fy[n], dot);
                    }
                    if (dy_sorted) po[c] = scaled(fd);
                }
            }
            if (lane < 3 && (lane == 0 || blocks > lane)) {
                const int c = lane == 0 ? 0 : blocks - lane;
                const int rel = 16 * c - lead;
                const int from = rel < 0 ? -rel / S : 0, to = bytes - rel < 16 ? (bytes - rel) / S : N;
                float fd[N];
                unpack<E>(load_window(dout, drow + rel, T * row_bytes), fd);
                if (dw) {
                    float fy[N];
                    unpack<E>(load_block(y_sorted, row + rel, R * row_bytes), fy);
#pragma unroll
                    for (int n = 0; n < N; ++n)
                        if (n >= from && n < to) dot = fmaf(fd[n], fy[n], dot);
                }
                if (dy_sorted) store_part<E>(dy_sorted + row + rel, scaled(fd), from, to);
            }
        }
        if (dw) {
            dot = lanes_sum<G>(dot, sh);
            if (lane == 0 && r < R) dw[r] = dot;
        }
    }
    if (dy_sorted) zero_tail(n_rows, R, row_bytes, dy_sorted);
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

int grid_for(long threads) {
    const long blocks = (threads + kThreads - 1) / kThreads;
    return static_cast<int>(blocks < 1 ? 1 : blocks > 148L * 64 ? 148L * 64 : blocks);
}

long row_bytes_of(const RowsArgs& a) { return static_cast<long>(a.H) * dtype_bytes(a.dtype); }

// A row's words in tiles of one, or of W to each lane of a warp.
struct WordTiles {
    FastDiv div;  // tiles of a row
    int grid;
    WordTiles(const RowsArgs& a, long words, int W) : div(static_cast<unsigned>(W > 1 ? (words + 32 * W - 1) / (32 * W) : words)) {
        grid = grid_for(static_cast<long>(a.T) * div.d * (W > 1 ? 32 : 1));
    }
};

template <int V>
using Int = std::integral_constant<int, V>;

// Calls f with the words that a thread takes of a row: as many as leave no more
// than half of a warp's without work (20000 tokens of 97 elements, top-8: 16.6 us
// with 4, 22.1 us with 2, 29.2 us with 1; 65536 of 61: 35.2 us with 2, 55.4 us
// with 1).
template <class F>
auto with_words(long words, F f) {
    return words > 96 ? f(Int<4>{}) : words > 32 ? f(Int<2>{}) : f(Int<1>{});
}

// Calls f(E, SHIFT) for the row type and alignment.
template <class F>
void dispatch(const RowsArgs& a, F f) {
    const bool shift = row_bytes_of(a) % 16 != 0;
    switch (a.dtype) {
        case MOE_DTYPE_BF16: shift ? f(__nv_bfloat16{}, std::true_type{}) : f(__nv_bfloat16{}, std::false_type{}); break;
        case MOE_DTYPE_F16: shift ? f(__half{}, std::true_type{}) : f(__half{}, std::false_type{}); break;
        default: shift ? f(float{}, std::true_type{}) : f(float{}, std::false_type{}); break;
    }
}

}  // namespace

cudaError_t launch_permute(const RowsArgs& a, const void* x, void* x_sorted, cudaStream_t stream) {
    const long row = row_bytes_of(a);
    const char* in = static_cast<const char*>(x);
    char* out = static_cast<char*>(x_sorted);
    if (row % 16 == 0) {
        const FastDiv vecs(static_cast<unsigned>(row / 16));
        return launch_after(permute_kernel, grid_for(static_cast<long>(a.T) * vecs.d), kThreads, 0, stream, in, a.inv, a.n_rows, a.T, a.K,
                            row, vecs, out, a.status);
    }
    const long words = (row + (row % 4 ? 2 : 0) + 3) / 4;  // at either start
    auto launch = [&](auto half, auto W) {
        const WordTiles tiles(a, words, decltype(W)::value);
        return launch_after(permute_words_kernel<decltype(half)::value, decltype(W)::value>, tiles.grid, kThreads, 0,
                            stream, in, a.inv, a.n_rows, a.T, a.K, row, tiles.div, out, a.status);
    };
    return with_words(words, [&](auto W) { return row % 4 ? launch(std::true_type{}, W) : launch(std::false_type{}, W); });
}

namespace {

cudaError_t launch_unpermute_ring(const RowsArgs& a, const void* y_sorted, const float* w, const void* y_shared,
                                  void* out, cudaStream_t stream) {
    const long row = row_bytes_of(a), R = static_cast<long>(a.T) * a.K;
    const bool shift = row % 16 != 0;
    RingArgs g{static_cast<const char*>(y_sorted), a.inv, w, static_cast<const char*>(y_shared),
               static_cast<char*>(out), a.status, a.T, a.K, a.K + (y_shared ? 1 : 0), 0, 0, 8, 1, 0, 0, R, row, 0,
               FastDiv(1)};
    // Warps of a token: the most whose pieces are filled to 8/9 on average, or as
    // well as those of any fewer.  (A shifted row's words may begin 2 bytes before it.)
    const long span = row + (a.dtype != MOE_DTYPE_F32 && row % 4 ? 2 : 0);
    auto padded = [&](long m) { return (span + 512 * m - 1) / (512 * m) * (512 * m); };
    for (int m = 8; m > 0 && padded(g.m) * 8 > span * 9; m /= 2)
        if (padded(m) < padded(g.m)) g.m = m;
    g.tokens = kConsumers / g.m;
    g.groups = (g.rows + kGroup - 1) / kGroup;
    g.group = (g.rows + g.groups - 1) / g.groups;
    const long size = g.m * 512;
    g.pieces = FastDiv(static_cast<unsigned>(padded(g.m) / size));
    g.items = (static_cast<long>(a.T) + g.tokens - 1) / g.tokens * g.pieces.d;
    g.slot = static_cast<int>(size) + (shift ? kShiftPad : 0);
    const int fit = kRingBytes / (g.tokens * g.group * g.slot);
    g.stages = fit < kMaxStages ? fit : kMaxStages;
    const long blocks = (g.items + kTeams - 1) / kTeams;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaError_t e = cudaSuccess;
    dispatch(a, [&](auto el, auto sh) {
        auto* kernel = unpermute_ring_kernel<decltype(el), decltype(sh)::value>;
        constexpr int smem = kRingHead + kTeams * kRingBytes;
        static_assert(smem <= 227 * 1024, "the rings exceed an SM's shared memory");
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return;
        e = launch_after(kernel, static_cast<int>(blocks < sms ? blocks : sms), kRingThreads, smem, stream, g);
    });
    return e;
}

}  // namespace

cudaError_t launch_unpermute(const RowsArgs& a, const void* y_sorted, const float* w, const void* y_shared, void* out,
                             cudaStream_t stream) {
    const long row = row_bytes_of(a);
    if (row >= kRingMinRow && a.T * a.K * row >= (row % 16 ? kRingMinBytesShift : kRingMinBytes))
        return launch_unpermute_ring(a, y_sorted, w, y_shared, out, stream);
    const char *y = static_cast<const char*>(y_sorted), *sh = static_cast<const char*>(y_shared);
    char* to = static_cast<char*>(out);
    cudaError_t err = cudaSuccess;
    auto even = [&](int most) { return (a.K + (a.K + most - 1) / most - 1) / ((a.K + most - 1) / most); };
    dispatch(a, [&](auto e, auto shift) {
        using E = decltype(e);
        if constexpr (!decltype(shift)::value) {
            const FastDiv vecs(static_cast<unsigned>(row / 16));
            const int grid = grid_for(static_cast<long>(a.T) * vecs.d);
            auto vectors = [&](auto most) {
                constexpr int B = decltype(most)::value;
                err = launch_after(unpermute_kernel<E, B>, grid, kThreads, 0, stream, y, a.inv, w, sh, a.T, a.K, even(B),
                                   row, vecs, to, a.status);
            };
            // One wave of blocks: one batch of all slots is one wait less (64 tokens of width 2048,
            // top-8: 2.6 us against 2.8 us).  More: the registers of larger batches cost more warps
            // than the wait.
            if (a.K > 4 && grid <= 148 * 3) vectors(Int<8>{});
            else vectors(Int<kBatch>{});
        } else {
            auto words = [&](auto word, auto W) {
                using Word = decltype(word);
                const WordTiles tiles(a, row / static_cast<long>(sizeof(Word)), decltype(W)::value);
                err = launch_after(unpermute_words_kernel<E, Word, decltype(W)::value>, tiles.grid, kThreads, 0, stream,
                                   y, a.inv, w, sh, a.T, a.K, even(kBatch), row, tiles.div, to, a.status);
            };
            if constexpr (sizeof(E) == 2) {
                if (row % 4) return with_words(a.H, [&](auto W) { words(uint16_t{}, W); });
            }
            with_words(row / 4, [&](auto W) { words(uint32_t{}, W); });
        }
    });
    return err;
}

cudaError_t launch_unpermute_bwd(const RowsArgs& a, const void* dout, const void* y_sorted, const float* w,
                                 void* dy_sorted, float* dw, cudaStream_t stream) {
    const long row = row_bytes_of(a), R = static_cast<long>(a.T) * a.K, vecs = (row + 15) / 16;
    const FastDiv K(static_cast<unsigned>(a.K));
    // Threads per route: so few that each has four vectors, down to 8 (32768
    // tokens of width 256: 58 us with 8, 114 us with 32 threads), but a whole
    // block while the routes are too few to fill the GPU with warps (64 tokens
    // of width 7168: 4.1 us against 10.0 us).
    const int g = vecs > 64 && R < 148 * 16 ? 256 : vecs <= 32 ? 8 : vecs <= 64 ? 16 : 32;
    const char *d = static_cast<const char*>(dout), *y = static_cast<const char*>(y_sorted);
    char* dy = static_cast<char*>(dy_sorted);
    cudaError_t err = cudaSuccess;
    dispatch(a, [&](auto e, auto shift) {
        using E = decltype(e);
        if constexpr (!decltype(shift)::value) {
            auto launch = [&](auto G, auto RU, auto U) {
                constexpr int kG = decltype(G)::value, kRU = decltype(RU)::value;
                err = launch_after(unpermute_bwd_kernel<E, kG, kRU, decltype(U)::value>,
                                   grid_for((R + kRU - 1) / kRU * kG), kThreads, 0, stream, d, y, a.inv, w, a.n_rows,
                                   a.T, K, row, dy, dw, a.status);
            };
            if (vecs <= 8) launch(Int<8>{}, Int<2>{}, Int<1>{});
            else if (g == 8) launch(Int<8>{}, Int<1>{}, Int<4>{});
            else if (g == 16) launch(Int<16>{}, Int<1>{}, Int<4>{});
            else if (g == 32) launch(Int<32>{}, Int<1>{}, Int<4>{});
            else launch(Int<256>{}, Int<1>{}, Int<4>{});
        } else {
            auto launch = [&](auto G) {
                constexpr int kG = decltype(G)::value;
                err = launch_after(unpermute_bwd_shift_kernel<E, kG>, grid_for(R * kG), kThreads, 0, stream, d, y,
                                   a.inv, w, a.n_rows, a.T, K, row, dy, dw, a.status);
            };
            if (g == 8) launch(Int<8>{});
            else if (g == 16) launch(Int<16>{});
            else if (g == 32) launch(Int<32>{});
            else launch(Int<256>{});
        }
    });
    return err;
}

}  // namespace moe
