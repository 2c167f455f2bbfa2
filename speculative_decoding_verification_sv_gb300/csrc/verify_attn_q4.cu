// verify_attn_q4.cu -- attention of the k+1 verify rows over a 4-bit paged KV
// cache (format: kv_q4.cuh) and the block's own bf16 K/V.
//
// out = softmax(scale q K^T) V over the cached positions and the block rows
// that the row may see.  The cache is 0.28 of the bf16 cache's bytes, so what
// bounds verify_attn.cu (HBM) bounds this kernel less than the work on the SM:
// unpacking the codes, the exponentials, and shared memory.
//
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T, with the cache
// as the A operand in tensor memory (tcgen05.mma, M = 128 keys or dims, N = 64
// rows).  A thread then unpacks one key's K, or one dim's V, straight from the
// packed bytes into its own TMEM lane: the 16-bit forms of K and V never pass
// through shared memory (written there and read back by the MMA they would cost
// 1024 of its cycles a step, against 656 for everything that is left), and the
// MMAs fill all 128 rows of the tensor core where a block of 63 query rows
// would fill half.
//   S^T: lane = key, column = query row.  B = Q, K-major in shared memory.
//   P:   exp2(s - m), bf16, written by the key's thread as one line of
//        [keys][64 rows] in shared memory, the MN-major B of the second product.
//        (The MMA takes V and P of one type, and only bf16 holds V's scales exactly and
//        a P above 65504.  Rounding moves a weight by at most 2^-8 of it, up or down; the
//        row's sum is taken of P before it.  With the output's own rounding that is 0.0024 of the
//        result, 0.0017 where P is fp32.)
//   O^T: lane = dim, column = row.
// A row's maximum runs across lanes here, so it is not formed: P is taken against
// a reference, the row's score with the run's first key.  bf16 and fp32 have the
// same range, so nothing is lost by a P far above 1 as long as no sum reaches
// kMostSum; a run where one does (some score 60 powers of two above the first
// key's) is done again with the reference moved to the maximum every step.  So is
// one where a row's sum stays below kLeastSum: its reference is a key that it does
// not see, or 0 for a score that is not finite, and its P may all be 0.
//
// Work.  A unit is one (sequence, KV head, tile of 64 query rows).  Where there are
// few of them over a short table each has a cluster of CTAs that leave their partial
// rows (m, l, O) in shared memory and join them over it.  Otherwise the units' pages,
// and the block as one more, are laid end to end over all units, and each CTA (one an
// SM) takes an equal run of them, whatever the sequences' lengths; a unit that lies in
// several CTAs' runs leaves partials in the workspace -- at most two a CTA -- and a
// second small kernel joins them.
//
// Warps: 8 softmax (TMEM quadrant w % 4, half of the tile's rows each), 4 unpack
// K, 4 unpack V, one issues the copies (two pages of K and V, 18 KB, a ring
// stage: each (page, head) is one 4608-byte bulk copy), one the MMAs, one brings
// the query rows of the next run while the present one is worked on.
//
// Measured.  16 x 9 rows of 28 heads over 4, 8192 positions: 36.7 us, 461 TFLOP/s and
// 2.1 TB/s of the cache's 76 MB.  A step of 128 keys is about 4660 warp instructions
// (16384 codes of K and 16384 of V unpacked, 8192 exponentials) and takes 0.7 to 1 us.  No
// unit is full: 54% of the issue slots, the ALU 36%, the tensor pipe 24%, FMA 23%, LSU 21%,
// special functions 13%; what holds a step up is that the roles wait for one another
// and for tensor memory (of the cycles between two of a warp's instructions a third is
// spent on such waits and barriers, an eighth each waiting for its turn to issue and for
// the next instruction to be fetched).  With one row a sequence the same cache takes 31.4 us.
// One sequence of 5 rows, 12 heads over 2, 4096 positions: 10.3 us, a chain of latencies:
// 2 us until the first page is there, 3 us for five steps, 1.5 us for the last sums and O,
// 3 us for the cluster's join and end.
#include <cooperative_groups.h>
#include <math.h>

#include <mutex>
#include <type_traits>

#include "kv_q4.cuh"
#include "sv_internal.h"

namespace cg = cooperative_groups;

namespace sv {
namespace {

constexpr int kRows = 64;                 // query rows of a tile
constexpr int kStepKeys = 128;            // two pages
constexpr int kStages = 6;
constexpr int kStageBytes = 4 * kQ4Bytes; // K of two pages, V of two pages
constexpr int kMaxR = 128;
constexpr int kSoftWarps = 8, kKWarp = 8, kVWarp = 12, kTmaWarp = 16, kMmaWarp = 17, kQWarp = 18, kThreads = 32 * 19;
constexpr int kGrain = 4;                 // pages a CTA takes at least (where there are as many)
constexpr float kMostSum = 0x1p64f;       // of a row's P, for the result to stand,
constexpr float kLeastSum = 0.5f;         // and at least (a reference that the row sees gives 1)
constexpr int kRecFloats = kRows * (kQ4D + 2);   // a partial: O [64][128], then (m, l) [64]
constexpr int kCombineThreads = 256;
constexpr int kMaxCluster = 8;

// TMEM columns: two K operands, two V operands (64 columns: 128 bf16 each), two
// S^T, one O^T
constexpr uint32_t kColK = 0, kColV = 128, kColS = 256, kColO = 384, kTmemCols = 512;

constexpr int kOffQ = 0;                                  // 2 x [2 halves of 64 dims][64 rows][128 B], swizzled
constexpr int kQBytes = kRows * kQ4D * 2;
constexpr int kOffP = kOffQ + 2 * kQBytes;                // kPBufs x [128 keys][128 B], swizzled
constexpr int kPBufs = 4;
constexpr int kPBytes = kStepKeys * kRows * 2;
constexpr int kOffRing = kOffP + kPBufs * kPBytes;
constexpr int kOffBar = kOffRing + kStages * kStageBytes;
constexpr int kOffNm = kOffBar + 272;                     // [64] -m, m the rows' references
constexpr int kOffMove = kOffNm + kRows * 4;              // [64] what O and l of the row are multiplied by
constexpr int kOffRed = kOffMove + kRows * 4;             // [4 quadrants][64]
constexpr int kOffBad = kOffRed + 4 * kRows * 4;          // [kStages] pages of the stage outside the pool
constexpr int kOffFail = kOffBad + 32;                    // a sum left its range; then where the runs start
constexpr int kOffPar = kOffFail + 32;                     // [128] parents
constexpr int kOffAnc = kOffPar + kMaxR * 4;              // [128][2] 64-bit path masks
constexpr int kOffRow = kOffAnc + kMaxR * 16;             // [64] (sequence, block row, head) of a tile row, -1 past the last
constexpr int kOffScale = kOffRow + kRows * 4;            // [4 V warps][s of 64 key pairs, then -136 s]
constexpr int kSmemBytes = kOffScale + 4 * 512;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
static_assert(kStages * 4 <= 32, "bad-page words");

struct Work {
    int U;         // units of a sequence: Hkv * row tiles
    int row_tiles;
    int tile_rows; // rows of a tile but the last
    int cluster;   // CTAs of a unit where each unit has a cluster, 0 where the pages are split evenly
    int inv_g;     // ceil(2^16 / G): r * inv_g >> 16 is r / G for every row r < 2048 of G <= 16
};

// Pages of sequence b (its length clamped into the table), the block not counted.
__device__ __forceinline__ int ctx_len(const AttnQ4Args& a, int b) {
    const int t = a.len[b];
    return t < 0 ? 0 : min(t, a.max_pages * kQ4Page);
}
__device__ __forceinline__ int ctx_pages(int t) { return (t + kQ4Page - 1) / kQ4Page; }

// Work of all sequences (sum of pages + 1), and of those before sequence
// `before`; one warp, every lane gets both.
__device__ __forceinline__ int2 work_sums(const AttnQ4Args& a, int before) {
    int all = 0, head = 0;
    for (int b = threadIdx.x & 31; b < a.B; b += 32) {
        const int w = ctx_pages(ctx_len(a, b)) + 1;
        all += w;
        if (b < before) head += w;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, off);
        head += __shfl_xor_sync(0xffffffffu, head, off);
    }
    return make_int2(all, head);
}

// CTAs that share W pages, and the first page of CTA i among them.
__device__ __forceinline__ int active_ctas(int W, int grid) { return max(1, min(grid, W / kGrain)); }
__device__ __forceinline__ int cta_first(int W, int i, int n) {
    return static_cast<int>(static_cast<int64_t>(W) * i / n);
}
// The CTA whose run holds page x: the largest i with floor(W i / n) <= x, that is
// W i < (x + 1) n.
__device__ __forceinline__ int cta_of(int W, int x, int n) {
    const int64_t most = (static_cast<int64_t>(x) + 1) * n - 1;
    return most < (int64_t(1) << 32) ? static_cast<int>(static_cast<uint32_t>(most) / static_cast<uint32_t>(W))
                                     : static_cast<int>(most / W);
}

// The runs of this CTA, unit by unit; every warp walks them by itself.
struct Walk {
    int pos, end;          // what is left of the CTA's run
    int b, unit, off;      // where pos lies: sequence, unit of it, page of the unit
    int t, np;             // length and pages of sequence b
    // the current run
    int p0, p1;            // its pages
    bool block, whole;     // the block is in it; it is all of the unit

    __device__ __forceinline__ void start(const AttnQ4Args& a, const Work& w, int cta, int grid) {
        const int lane = threadIdx.x & 31;
        // (the first 32 lengths stay in registers: a round trip less for most batches)
        const int t0 = lane < a.B ? ctx_len(a, lane) : 0;
        const int w0 = lane < a.B ? (ctx_pages(t0) + 1) * w.U : 0;
        int W = w0;
        for (int i = 32 + lane; i < a.B; i += 32) W += (ctx_pages(ctx_len(a, i)) + 1) * w.U;
        W = __reduce_add_sync(0xffffffffu, W);
        const int n = active_ctas(W, grid);
        pos = end = 0;
        b = -1;
        if (cta >= n) return;
        pos = cta_first(W, cta, n);
        end = cta_first(W, cta + 1, n);
        // the sequence that pos lies in
        int base = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int tb = b0 == 0 ? t0 : b0 + lane < a.B ? ctx_len(a, b0 + lane) : 0;
            const int wt = b0 == 0 ? w0 : b0 + lane < a.B ? (ctx_pages(tb) + 1) * w.U : 0;
            int sum = wt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += x;
            }
            const uint32_t m = __ballot_sync(0xffffffffu, base + sum > pos);
            if (m != 0u) {
                const int k = __ffs(m) - 1;
                b = b0 + k;
                base += __shfl_sync(0xffffffffu, sum - wt, k);
                t = __shfl_sync(0xffffffffu, tb, k);
                break;
            }
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
        np = ctx_pages(t);
        unit = (pos - base) / (np + 1);
        off = (pos - base) % (np + 1);
    }
    // Unit u's pages for CTA `rank` of the cluster that has the unit.
    __device__ __forceinline__ void start_unit(const AttnQ4Args& a, const Work& w, int u, int rank) {
        b = u / w.U;
        unit = u - b * w.U;
        t = ctx_len(a, b);
        np = ctx_pages(t);
        pos = off = static_cast<int>(static_cast<int64_t>(np + 1) * rank / w.cluster);
        end = static_cast<int>(static_cast<int64_t>(np + 1) * (rank + 1) / w.cluster);
    }
    __device__ __forceinline__ bool next(const AttnQ4Args& a, const Work& w) {
        if (pos >= end) return false;
        const int n = min(end - pos, np + 1 - off);
        p0 = off;
        p1 = min(off + n, np);
        block = off + n == np + 1;
        whole = n == np + 1;
        pos += n;
        cur_b = b;
        cur_unit = unit;
        cur_t = t;
        off = 0;
        if (block && ++unit == w.U) {
            unit = 0;
            if (++b < a.B) {
                t = ctx_len(a, b);
                np = ctx_pages(t);
            }
        }
        return true;
    }
    int cur_b, cur_unit, cur_t;
    __device__ __forceinline__ void save(volatile int* to) const {
        to[0] = pos, to[1] = end, to[2] = b, to[3] = unit, to[4] = off;
    }
    __device__ __forceinline__ void load(const AttnQ4Args& a, const volatile int* from) {
        pos = from[0], end = from[1], b = from[2], unit = from[3], off = from[4];
        t = ctx_len(a, b);
        np = ctx_pages(t);
    }
    __device__ __forceinline__ int ctx_steps() const { return (p1 - p0 + 1) / 2; }
};

// --- packed arithmetic ---------------------------------------------------------

__device__ __forceinline__ uint32_t bfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// bf16 pair 128 + c of elements 2k, 2k + 1 of a word: one shift, one three-input
// logical operation on registers (as immediates the two constants would take two)
struct CodeMask {
    uint32_t nibbles, exps;
    __device__ __forceinline__ CodeMask() {
        asm volatile("mov.u32 %0, 0x000F000F;\n\tmov.u32 %1, 0x43004300;" : "=r"(nibbles), "=r"(exps));
    }
    __device__ __forceinline__ uint32_t pair(uint32_t w, int k) const {
        uint32_t r;
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * k)), "r"(nibbles), "r"(exps));
        return r;
    }
};
constexpr uint32_t kM136 = 0xC308C308u;   // bf16 pair of -136

// One lane of the (converged) warp, always the same one.  A branch on it is
// known to be taken by one thread, and the MMAs' operands then stay in uniform
// registers: 25 cycles an MMA issued in place of 45 under lane == 0 (M = 128, N
// = 64, whose own time is 35).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r));
    return r != 0u;
}


__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Sums of kN values over the lanes: half of the values are handed to the lane
// whose number differs in the bit kN / 2, and so on; v[0] of lane e ends as value
// e's sum over the lanes that agree with e below kN.
template <int kN, int kLen>
__device__ __forceinline__ void fold_sums_step(float (&v)[kLen]) {
    const bool upper = (threadIdx.x & (kN / 2)) != 0;
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
        const float give = upper ? v[i] : v[i + kN / 2];
        const float keep = upper ? v[i + kN / 2] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, kN / 2);
    }
    if constexpr (kN > 2) fold_sums_step<kN / 2>(v);
}
template <int kN>
__device__ __forceinline__ void fold_sums(float (&v)[kN]) {
    fold_sums_step<kN>(v);
}

// Joins n partials of a row, eight in flight; get(i, ml, o) loads the i-th's
// (m, l) and the lane's four dims of its O.
template <typename Get>
__device__ __forceinline__ void join_row(int n, Get&& get, uint16_t* dst) {
    const int lane = threadIdx.x & 31;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < n; c0 += 8) {
        float2 ml[8];
        float4 o[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            ml[u] = make_float2(-INFINITY, 0.f);
            o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c0 + u < n) get(c0 + u, ml[u], o[u]);
        }
        float mn = M;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (ml[u].y != 0.f) mn = fmaxf(mn, ml[u].x);
        const float c = M == -INFINITY ? 0.f : exp2f(M - mn);
        acc.x *= c, acc.y *= c, acc.z *= c, acc.w *= c, L *= c;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (ml[u].y == 0.f) continue;   // all of the row's scores there are -inf
            const float w = exp2f(ml[u].x - mn);
            L += w * ml[u].y;
            acc.x += w * o[u].x;
            acc.y += w * o[u].y;
            acc.z += w * o[u].z;
            acc.w += w * o[u].w;
        }
        M = mn;
    }
    const float inv = L != 0.f ? 1.0f / L : 0.f;
    *reinterpret_cast<uint2*>(dst + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// kRT: rows a softmax thread takes; the tile's rows past 2 kRT do not exist (their
// columns of P stay zero)
template <int kRT, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1) attn_q4_kernel(AttnQ4Args a, Work wk, float* __restrict__ ws) {
    constexpr int kLive = 2 * kRT;
    // (aligned by its declaration: addresses are then constants, not registers)
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* ring_full = bars;                   // [kStages]
    uint64_t* ring_empty = ring_full + kStages;   // [kStages]
    uint64_t* k_full = ring_empty + kStages;      // [2] K operand unpacked
    uint64_t* v_full = k_full + 2;                // [2]
    uint64_t* s_full = v_full + 2;                // [2] S^T formed (and the K operand read)
    uint64_t* s_empty = s_full + 2;               // [2] scores read
    uint64_t* p_full = s_empty + 2;               // [kPBufs] P written (and O rescaled): one each, as a warp may
                                                  // be two steps ahead of another
    uint64_t* pv_done = p_full + kPBufs;               // [2] O^T has the step (P and the V operand read)
    uint64_t* q_ready = pv_done + 2;              // [2] query rows there
    uint64_t* q_free = q_ready + 2;               // [2] the run's S^T are formed
    uint64_t* o_free = q_free + 2;                // O^T read by the epilogue
    uint64_t* o_done = o_free + 1;                // O^T has the run's last step (pv_done is no help there: two
                                                  // of its phases may be missing, and a wait passes at once)
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(o_done + 1);
    static_assert((2 * kStages + 16 + kPBufs) * 8 + 4 <= 272, "barrier area");
    float* nm_s = reinterpret_cast<float*>(smem + kOffNm);
    float* move_s = reinterpret_cast<float*>(smem + kOffMove);
    float* red_s = reinterpret_cast<float*>(smem + kOffRed);
    volatile uint32_t* bad_s = reinterpret_cast<volatile uint32_t*>(smem + kOffBad);
    int32_t* par_s = reinterpret_cast<int32_t*>(smem + kOffPar);
    uint64_t* anc_s = reinterpret_cast<uint64_t*>(smem + kOffAnc);
    int* row_s = reinterpret_cast<int*>(smem + kOffRow);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *reinterpret_cast<volatile int*>(smem + kOffFail) = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&v_full[i], 4);
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kSoftWarps);
            mbar_init(&pv_done[i], 1);
            mbar_init(&q_ready[i], 1);
            mbar_init(&q_free[i], 1);
        }
        for (int i = 0; i < kPBufs; ++i) mbar_init(&p_full[i], kSoftWarps);
        mbar_init(o_free, kSoftWarps);
        mbar_init(o_done, 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_s, kTmemCols);
    if (kLive < kRows) {   // the columns of P past the live rows stay zero
        for (int x = threadIdx.x; x < kPBufs * kPBytes / 16; x += kThreads)
            reinterpret_cast<uint4*>(smem + kOffP)[x] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    const int q4 = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    auto tK = [tmem](int i) { return tmem + kColK + static_cast<uint32_t>(i) * 64u; };
    auto tV = [tmem](int i) { return tmem + kColV + static_cast<uint32_t>(i) * 64u; };
    auto tS = [tmem](int i) { return tmem + kColS + static_cast<uint32_t>(i) * 64u; };
    const uint32_t tO = tmem + kColO;

    // With cache_ready the lengths, the page table and the committed pages were
    // final before the preceding kernel ran: the walk and the page copies start
    // under it, and whoever touches anything else waits first.
    const bool early = a.cache_ready;
    if (!early) pdl_wait();
    Walk walk;
    const int rank = kCluster ? blockIdx.x % wk.cluster : 0;
    if constexpr (kCluster) walk.start_unit(a, wk, blockIdx.x / wk.cluster, rank);
    else walk.start(a, wk, blockIdx.x, gridDim.x);
    volatile int* fail_s = reinterpret_cast<volatile int*>(smem + kOffFail);
    if (threadIdx.x == 0) walk.save(fail_s + 1);
    // Each role runs the CTA's runs once, and once more with `safe` where a sum
    // left its range (the softmax warps' verdict, after all have finished).
    bool safe = false;
    // a warp's wait; its lanes go on together (what follows is warp-collective)
    auto wait = [&](uint64_t* bar, int parity) {
        mbar_wait(bar, static_cast<uint32_t>(parity), a.err);
        __syncwarp();
    };
    auto again = [&]() {
        if (safe) return false;
        __syncwarp();
        named_barrier(2, kThreads);
        safe = true;
        if (*fail_s == 0) return false;
        walk.load(a, fail_s + 1);
        return true;
    };

    if (warp == kTmaWarp) {
        // ---------------- page copies ----------------
        int c = 0;   // context steps so far
        do {
            while (walk.next(a, wk)) {
                const int g = walk.cur_unit / wk.row_tiles;
                const int32_t* tab = a.pages + static_cast<size_t>(walk.cur_b) * a.max_pages;
                const int np = walk.p1 - walk.p0;
                for (int i0 = 0; i0 < np; i0 += 32) {
                    // 32 table entries at once: lane l holds page p0 + i0 + l
                    int pg = i0 + lane < np ? __ldg(tab + walk.p0 + i0 + lane) : 0;
                    const bool bad = pg < 0 || pg >= a.num_pages;
                    if (bad) {
                        raise_error(a.err, SV_DEVERR_PAGE);
                        pg = -1;
                    }
                    for (int i = 0; i < 32 && i0 + i < np; i += 2, ++c) {
                        const int pa = __shfl_sync(0xffffffffu, pg, i), pb = __shfl_sync(0xffffffffu, pg, i + 1);
                        const bool two = i0 + i + 1 < np;
                        if (lane == 0) {
                            const int s = c % kStages;
                            mbar_wait(&ring_empty[s], ((c / kStages) & 1) ^ 1, a.err);
                            uint8_t* st = smem + kOffRing + s * kStageBytes;
                            const bool la = pa >= 0, lb = two && pb >= 0;
                            bad_s[s] = (la ? 0u : 1u) | (two && pb < 0 ? 2u : 0u);
                            mbar_arrive_expect_tx(&ring_full[s], (la ? 2 * kQ4Bytes : 0) + (lb ? 2 * kQ4Bytes : 0));
                            const size_t oa = (static_cast<size_t>(pa) * a.Hkv + g) * kQ4Bytes;
                            const size_t ob = (static_cast<size_t>(pb) * a.Hkv + g) * kQ4Bytes;
                            if (la) bulk_g2s(st, a.k_pool + oa, kQ4Bytes, &ring_full[s]);
                            if (lb) bulk_g2s(st + kQ4Bytes, a.k_pool + ob, kQ4Bytes, &ring_full[s]);
                            if (la) bulk_g2s(st + 2 * kQ4Bytes, a.v_pool + oa, kQ4Bytes, &ring_full[s]);
                            if (lb) bulk_g2s(st + 3 * kQ4Bytes, a.v_pool + ob, kQ4Bytes, &ring_full[s]);
                        }
                        __syncwarp();
                    }
                }
            }
        } while (again());
    } else if (warp == kMmaWarp) {
        // ---------------- MMA issuer ----------------
        constexpr uint32_t id_s = idesc_bf16_f32(128, kLive, false, false);
        constexpr uint32_t id_o = idesc_bf16_f32(128, kRows, false, true);
        int it = 0, seg = 0;
        do {
            while (walk.next(a, wk)) {
                const int n = walk.ctx_steps() + (walk.block ? 1 : 0);
                if (elect_one()) {
                    const uint64_t qd = smem_desc_sw128(smem_u32(smem + kOffQ + (seg & 1) * kQBytes), 16, 1024);
                    // S of step i + 2 goes ahead of P V of step i: it only waits for the
                    // scores of step i to be read, not for their P
                    auto scores = [&](int i) {
                        const int x = i & 1;
                        mbar_wait(&k_full[x], (i >> 1) & 1, a.err);
                        mbar_wait(&s_empty[x], ((i >> 1) & 1) ^ 1, a.err);
                        tc_fence_after();
#pragma unroll
                        for (int kc = 0; kc < kQ4D / 16; ++kc)
                            tc_mma_ts(tS(x), tK(x) + kc * 8, qd + (((kc >> 2) * kRows * 128 + (kc & 3) * 32) >> 4), id_s,
                                      kc > 0 ? 1u : 0u);
                        tc_commit(&s_full[x]);
                        if (i == it + n - 1) tc_commit(&q_free[seg & 1]);
                    };
                    mbar_wait(&q_ready[seg & 1], (seg >> 1) & 1, a.err);
#pragma unroll 1
                    for (int st = -2; st < n; ++st) {
                        if (st + 2 < n) scores(it + st + 2);
                        if (st < 0) continue;
                        const int i = it + st, x = i & 1;
                        if (st == 0) mbar_wait(o_free, (seg & 1) ^ 1, a.err);
                        mbar_wait(&v_full[x], (i >> 1) & 1, a.err);
                        mbar_wait(&p_full[i % kPBufs], (i / kPBufs) & 1, a.err);
                        tc_fence_after();
                        const uint64_t pd = smem_desc_sw128(smem_u32(smem + kOffP + i % kPBufs * kPBytes), 16, 1024);
#pragma unroll
                        for (int kc = 0; kc < kStepKeys / 16; ++kc)
                            tc_mma_ts(tO, tV(x) + kc * 8, pd + kc * (2048 >> 4), id_o, (kc > 0 || st > 0) ? 1u : 0u);
                        tc_commit(&pv_done[x]);
                        if (st == n - 1) tc_commit(o_done);
                    }
                }
                __syncwarp();
                it += n;
                ++seg;
            }
        } while (again());
    } else if (warp == kQWarp) {
        // ---------------- query rows ----------------
        if (early) pdl_wait();
        int seg = 0;
        do {
            while (walk.next(a, wk)) {
                const int g = walk.cur_unit / wk.row_tiles, row0 = walk.cur_unit % wk.row_tiles * wk.tile_rows;
                const int nrows = min(wk.tile_rows, a.R * a.G - row0);
                // where each row lies (two a lane), -1 past the last
                int at[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 32 * h + lane, gr = row0 + r, j = gr * wk.inv_g >> 16;
                    at[h] = r < nrows ? (walk.cur_b * a.R + j) * a.Hq + g * a.G + gr - j * a.G : -1;
                }
                wait(&q_free[seg & 1], ((seg >> 1) & 1) ^ 1);
                uint8_t* q_s = smem + kOffQ + (seg & 1) * kQBytes;
                // K-major, 128-byte swizzle, zeros past the last row: half a warp a row
                const int ch = lane & 15;
#pragma unroll
                for (int h = 0; h < kLive / 32; ++h) {
#pragma unroll 8
                    for (int i = 0; i < 32; i += 2) {
                        const int r = 32 * h + i + (lane >> 4), row = __shfl_sync(0xffffffffu, at[h], r & 31);
                        uint8_t* dst = q_s + (ch >> 3) * (kRows * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
                        if (row >= 0) cp_async16(dst, reinterpret_cast<const uint4*>(a.q + static_cast<size_t>(row) * kQ4D) + ch);
                        else *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                cp_async_wait_all();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_ready[seg & 1]);
                ++seg;
            }
        } while (again());
    } else if (warp >= kKWarp) {
        // ---------------- unpacking: a key's K, a dim's V ----------------
        const bool is_v = warp >= kVWarp;
        const int l = q4 * 32 + lane;   // TMEM lane: key of the step, or dim
        uint64_t* full = is_v ? v_full : k_full;
        uint64_t* freed = is_v ? pv_done : s_full;
        int it = 0, c = 0;
        bool waited = !early;
        const CodeMask cm;
        auto put = [&](int col, const uint32_t(&w)[16]) {
            tmem_st16((is_v ? tV(it & 1) : tK(it & 1)) + lane_off + col, w);
        };
        auto done = [&]() {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[it & 1]);
        };
        do {
            while (walk.next(a, wk)) {
                // the block's rows, read at the end of the run by loads that wait for one
                // another, are brought near meanwhile (256 bytes a row; a thread a line or two)
                const size_t blk0 = (static_cast<size_t>(walk.cur_b) * a.Hkv + walk.cur_unit / wk.row_tiles) * a.R * kQ4D;
                if (walk.block && waited) {
                    const uint16_t* near = (is_v ? a.v_blk : a.k_blk) + blk0;
                    for (int x = l; x < 2 * a.R; x += 128) asm volatile("prefetch.global.L1 [%0];" ::"l"(near + 64 * x));
                }
                for (int st = 0; st < walk.ctx_steps(); ++st, ++it, ++c) {
                    const int s = c % kStages;
                    const uint8_t* stage = smem + kOffRing + s * kStageBytes;
                    wait(&ring_full[s], (c / kStages) & 1);
                    const uint32_t bad = bad_s[s];
                    wait(&freed[it & 1], ((it >> 1) & 1) ^ 1);
                    tc_fence_after();
                    if (!is_v) {
                        const uint8_t* blk = stage + (l >> 6) * kQ4Bytes;
                        const int pos = l & 63;
                        uint2 sc = *reinterpret_cast<const uint2*>(blk + q4_k_scale_off(0, pos));
                        if (bad >> (l >> 6) & 1u) sc = make_uint2(0u, 0u);
                        uint4 cw = *reinterpret_cast<const uint4*>(blk + q4_k_code_off(0, pos));
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const uint32_t s2 = __byte_perm(sc.x, 0u, 0x1010);
                            sc.x = g == 1 ? sc.y : sc.x >> 16;
                            const uint32_t o2 = bmul2(s2, kM136);
                            const uint32_t ww[4] = {cw.x, cw.y, cw.z, cw.w};
                            if (g < 3) cw = *reinterpret_cast<const uint4*>(blk + q4_k_code_off(g + 1, pos));
                            uint32_t r[16];
#pragma unroll
                            for (int w = 0; w < 4; ++w)
#pragma unroll
                                for (int k = 0; k < 4; ++k) r[4 * w + k] = bfma2(cm.pair(ww[w], k), s2, o2);
                            put(16 * g, r);
                        }
                    } else {
                        // keys of the step that exist: the others, and pages outside
                        // the pool, are zeros (0 * a non-finite V would be NaN)
                        const int have = min(walk.cur_t - (walk.p0 + 2 * st) * kQ4Page, (walk.p1 - walk.p0 - 2 * st) * kQ4Page);
                        // the warp's 32 dims are one group: the step's 64 pairs of scales and
                        // -136 times them, formed once by its lanes
                        uint32_t* sc_s = reinterpret_cast<uint32_t*>(smem + kOffScale + q4 * 512);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t s2 = *reinterpret_cast<const uint32_t*>(stage + (2 + h) * kQ4Bytes +
                                                                             q4_v_scale_off(q4, 2 * lane));
                            if (have < kStepKeys || bad != 0u) {
                                const int n = (bad >> h & 1u) ? 0 : have - kQ4Page * h - 2 * lane;
                                s2 &= n > 1 ? ~0u : n > 0 ? 0xFFFFu : 0u;
                            }
                            sc_s[32 * h + lane] = s2;
                            sc_s[64 + 32 * h + lane] = bmul2(s2, kM136);
                        }
                        __syncwarp();
#pragma unroll
                        for (int h = 0; h < 4; ++h) {   // 32 keys: half a page
                            const uint8_t* blk = stage + (2 + (h >> 1)) * kQ4Bytes;
                            uint32_t r[16];
#pragma unroll
                            for (int o = 0; o < 4; ++o) {
                                const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + q4_v_code_off((h & 1) * 4 + o, l));
                                const uint4 sv = reinterpret_cast<const uint4*>(sc_s)[4 * h + o];
                                const uint4 ov = reinterpret_cast<const uint4*>(sc_s)[16 + 4 * h + o];
                                r[4 * o] = bfma2(cm.pair(w, 0), sv.x, ov.x);
                                r[4 * o + 1] = bfma2(cm.pair(w, 1), sv.y, ov.y);
                                r[4 * o + 2] = bfma2(cm.pair(w, 2), sv.z, ov.z);
                                r[4 * o + 3] = bfma2(cm.pair(w, 3), sv.w, ov.w);
                            }
                            put(16 * h, r);
                        }
                    }
                    done();
                    if (lane == 0) mbar_arrive(&ring_empty[s]);
                }
                if (walk.block) {
                    if (!waited) pdl_wait();
                    waited = true;
                    wait(&freed[it & 1], ((it >> 1) & 1) ^ 1);
                    tc_fence_after();
                    if (!is_v) {
                        const uint4* src = reinterpret_cast<const uint4*>(a.k_blk + blk0 + l * kQ4D);
#pragma unroll 1
                        for (int x = 0; x < 4; ++x) {
                            uint32_t r[16];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                                if (l < a.R) v = __ldg(src + 4 * x + y);
                                r[4 * y] = v.x, r[4 * y + 1] = v.y, r[4 * y + 2] = v.z, r[4 * y + 3] = v.w;
                            }
                            put(16 * x, r);
                        }
                    } else {
                        const uint16_t* src = a.v_blk + blk0 + l;
#pragma unroll 1
                        for (int h = 0; h < 4; ++h) {
                            uint32_t r[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const int key = 32 * h + 2 * k;
                                const uint32_t lo = key < a.R ? __ldg(src + key * kQ4D) : 0u;
                                const uint32_t hi = key + 1 < a.R ? __ldg(src + (key + 1) * kQ4D) : 0u;
                                r[k] = lo | hi << 16;
                            }
                            put(16 * h, r);
                        }
                    }
                    done();
                    ++it;
                }
            }
        } while (again());
        if (!waited) pdl_wait();
    } else {
        // ---------------- softmax, epilogue ----------------
        // (the barrier counts whole warps: they arrive converged)
        auto soft_sync = []() {
            __syncwarp();
            named_barrier(1, 32 * kSoftWarps);
        };
        if (early) pdl_wait();
        // A cluster's successor may start now.  (Not before the wait: the successor may
        // read a cache that only this kernel's predecessor must not be writing.)
        if constexpr (kCluster) pdl_launch_dependents();
        const int hh = warp >> 2;              // rows hh * kRT .. of the tile
        const int l = q4 * 32 + lane;          // key of the step; dim in the epilogue
        const int tid = threadIdx.x;
        const float sc = a.scale_log2;
        const int rows = a.R * a.G;
        int it = 0, seg = 0;
        do {
            int part = 0;
            while (walk.next(a, wk)) {
                const int b = walk.cur_b, g = walk.cur_unit / wk.row_tiles, rt = walk.cur_unit % wk.row_tiles;
                const int row0 = rt * wk.tile_rows, nrows = min(wk.tile_rows, rows - row0);
                if (tid == 0) {
                    const int t = a.len[b];
                    if (t < 0 || t > a.max_pages * kQ4Page) raise_error(a.err, SV_DEVERR_LENGTH);
                }
                if (tid < kRows) {
                    const int gr = row0 + tid, j = gr * wk.inv_g >> 16;
                    row_s[tid] = tid < nrows ? (b * a.R + j) * a.Hq + g * a.G + gr - j * a.G : -1;
                    nm_s[tid] = 0.f;
                }
                const bool tree = walk.block && a.parent != nullptr;
                if (tree && tid < a.R) par_s[tid] = __ldg(a.parent + static_cast<size_t>(b) * a.R + tid);
                soft_sync();   // row_s, nm_s, par_s
                if (tree) {
                    if (tid < a.R) {
                        uint64_t m0 = 0, m1 = 0;
                        int i = tid;
                        bool bad = false;
                        for (int n = 0; n <= a.R && i >= 0; ++n) {
                            if (i < 64) m0 |= 1ull << i;
                            else m1 |= 1ull << (i - 64);
                            const int p = par_s[i];
                            if ((i == 0 && p != -1) || (i > 0 && (p < 0 || p >= i))) {
                                bad = true;
                                break;
                            }
                            i = p;
                        }
                        if (bad) {
                            raise_error(a.err, SV_DEVERR_TREE);
                            m0 = tid < 64 ? 1ull << tid : 0ull;
                            m1 = tid >= 64 ? 1ull << (tid - 64) : 0ull;
                        }
                        anc_s[2 * tid] = m0;
                        anc_s[2 * tid + 1] = m1;
                    }
                    soft_sync();
                }
                float sums[kRT];
#pragma unroll
                for (int i = 0; i < kRT; ++i) sums[i] = 0.f;
                bool found = false;   // (safe) row tid has a reference
                const int nctx = walk.ctx_steps(), n = nctx + (walk.block ? 1 : 0);
                auto step = [&](int st, auto general_c) {
                    constexpr bool kGeneral = decltype(general_c)::value;
                    const int x = it & 1;
                    wait(&s_full[x], (it >> 1) & 1);
                    tc_fence_after();
                    // the rows that see this thread's key (bit e: row hh * kRT + e), in the
                    // steps where some do not: of the context, keys before the length (the
                    // second page of a step may be missing); block row l is seen from query
                    // rows l G on, or by the tree rows on whose path it lies
                    uint32_t seen = ~0u;
                    if constexpr (kGeneral) {
                        if (st < nctx) {
                            if ((walk.p0 + 2 * st) * kQ4Page + l >= min(walk.cur_t, walk.p1 * kQ4Page)) seen = 0u;
                        } else if (!tree) {
                            const int lo = l < a.R ? l * a.G - row0 - hh * kRT : kRT;
                            seen = lo >= kRT ? 0u : lo > 0 ? ~0u << lo : ~0u;
                        } else {
                            // block row by block row: its G query rows see the same keys
                            seen = 0u;
                            const int r0 = row0 + hh * kRT, r1 = min(r0 + kRT, rows);
                            int j = r0 * wk.inv_g >> 16;
                            for (int r = j * a.G - r0; l < a.R && r + r0 < r1; ++j, r += a.G) {
                                if ((anc_s[2 * j + (l >> 6)] >> (l & 63) & 1ull) == 0ull) continue;
                                const uint32_t run = (1u << a.G) - 1u;   // (G <= 16)
                                seen |= r >= 0 ? run << r : run >> -r;
                            }
                        }
                    }
                    // exponents of rows c0 .. of the thread's against their references
                    auto exponents = [&](int c0, float(&e)[16]) {
                        uint32_t s[16];
                        tmem_ld16_sync(tS(x) + lane_off + hh * kRT + c0, s);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 nm = reinterpret_cast<const float4*>(nm_s + hh * kRT + c0)[i];
                            e[4 * i] = fmaf(__uint_as_float(s[4 * i]), sc, nm.x);
                            e[4 * i + 1] = fmaf(__uint_as_float(s[4 * i + 1]), sc, nm.y);
                            e[4 * i + 2] = fmaf(__uint_as_float(s[4 * i + 2]), sc, nm.z);
                            e[4 * i + 3] = fmaf(__uint_as_float(s[4 * i + 3]), sc, nm.w);
                        }
                        if constexpr (kGeneral) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (!(seen >> (c0 + i) & 1u)) e[i] = -INFINITY;
                        }
                    };
                    // the references (until now 0): the first key's scores where they are finite,
                    // or, with `safe`, the running maxima.  (A row that does not see that key, or
                    // whose score with it is not finite, may find its sum below kLeastSum.)
                    if constexpr (kGeneral) {
                        if (st == 0 && !safe) {
                            if (q4 == 0) {
#pragma unroll 1
                                for (int c0 = 0; c0 < kRT; c0 += 16) {
                                    uint32_t s[16];
                                    tmem_ld16_sync(tS(x) + lane_off + hh * kRT + c0, s);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        const float e = __uint_as_float(s[i]) * -sc;
                                        s[i] = fabsf(e) < INFINITY ? __float_as_uint(e) : 0u;
                                    }
                                    if (lane == 0) {
#pragma unroll
                                        for (int i = 0; i < 16; i += 4)
                                            *reinterpret_cast<uint4*>(nm_s + hh * kRT + c0 + i) =
                                                make_uint4(s[i], s[i + 1], s[i + 2], s[i + 3]);
                                    }
                                    __syncwarp();
                                }
                            }
                            soft_sync();
                        }
                        if (safe) {
#pragma unroll 1
                            for (int c0 = 0; c0 < kRT; c0 += 16) {
                                float e[16];
                                exponents(c0, e);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    e[i] = warp_max(e[i]);
                                    if (lane == 0) red_s[q4 * kRows + hh * kRT + c0 + i] = e[i];
                                }
                            }
                            soft_sync();
                            if (tid < kLive) {
                                // up, or where no score was finite so far (P, the sum and O are
                                // 0 then) to wherever the maximum is
                                float d = fmaxf(fmaxf(red_s[tid], red_s[kRows + tid]),
                                                fmaxf(red_s[2 * kRows + tid], red_s[3 * kRows + tid]));
                                const bool none = d == -INFINITY;
                                if (none || (found && d < 0.f)) d = 0.f;
                                nm_s[tid] -= d;
                                move_s[tid] = found ? fast_exp2(-d) : 1.0f;
                                found = found || !none;
                            }
                            soft_sync();
                            if (st > 0) {
#pragma unroll
                                for (int i = 0; i < kRT; ++i) sums[i] *= move_s[hh * kRT + i];
                                // O^T (lane = dim) once the step before is in it
                                wait(&pv_done[x ^ 1], ((it - 1) >> 1) & 1);
                                tc_fence_after();
#pragma unroll 1
                                for (int c0 = 0; c0 < kRT; c0 += 16) {
                                    const uint32_t ta = tO + lane_off + hh * kRT + c0;
                                    uint32_t o[16];
                                    tmem_ld16_sync(ta, o);
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        o[e] = __float_as_uint(__uint_as_float(o[e]) * move_s[hh * kRT + c0 + e]);
                                    tmem_st16(ta, o);
                                }
                                tmem_st_wait();
                            }
                        }
                    }
                    // a key's line of P takes eight rows in 16 bytes.  (The buffer is free: S of
                    // this step was issued behind P V of three steps before.)
                    uint8_t* prow = smem + kOffP + it % kPBufs * kPBytes + l * 128;
#pragma unroll
                    for (int c0 = 0; c0 < kRT; c0 += 16) {
                        float e[16];
                        exponents(c0, e);
                        if (c0 + 16 == kRT) {   // the scores are read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&s_empty[x]);
                        }
#pragma unroll
                        for (int ch = 0; ch < 2; ++ch) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float p = fast_exp2(e[8 * ch + 2 * i]), q = fast_exp2(e[8 * ch + 2 * i + 1]);
                                sums[c0 + 8 * ch + 2 * i] += p;
                                sums[c0 + 8 * ch + 2 * i + 1] += q;
                                w[i] = pack_bf16x2(p, q);
                            }
                            *reinterpret_cast<uint4*>(prow + (((hh * (kRT / 8) + c0 / 8 + ch) ^ (l & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[it % kPBufs]);
                    ++it;
                };
                // the plain steps -- whole context steps but the run's first -- apart, so
                // that they carry neither masks nor references
                const bool ragged = nctx > 0 && ((walk.p1 - walk.p0) & 1 || walk.p1 * kQ4Page > walk.cur_t);
                const int nwhole = safe ? 0 : nctx - (ragged ? 1 : 0);
#pragma unroll 1
                for (int st = 0; st < n; ++st) {
                    if (st > 0 && st < nwhole) step(st, std::false_type{});
                    else step(st, std::true_type{});
                }
                // the rows' sums over the keys: lane e of a warp ends with its row e's
                // (halving the rows and the lanes that differ, step by step)
                fold_sums(sums);
                if (kRT == 16) sums[0] += __shfl_xor_sync(0xffffffffu, sums[0], 16);
                if (lane < kRT) red_s[q4 * kRows + hh * kRT + lane] = sums[0];
                // (a cluster's partials stay on chip: the copies into the ring have all been read)
                float* rec = kCluster ? reinterpret_cast<float*>(smem + kOffRing)
                             : walk.whole ? nullptr : ws + (static_cast<size_t>(blockIdx.x) * 2 + part) * kRecFloats;
                soft_sync();
                bool bad = false;
                float lsum = 0.f;
                if (tid < kLive) {
                    lsum = (red_s[tid] + red_s[kRows + tid]) + (red_s[2 * kRows + tid] + red_s[3 * kRows + tid]);
                    bad = !(lsum < kMostSum) || (lsum < kLeastSum && tid < nrows);
                    move_s[tid] = lsum != 0.f ? 1.0f / lsum : 0.f;
                }
                wait(o_done, seg & 1);
                // (a cluster's partial overwrites the ring: only now have all pages been read)
                if (rec && tid < kLive)
                    *reinterpret_cast<float2*>(rec + kRows * kQ4D + 2 * tid) = make_float2(-nm_s[tid], lsum);
                tc_fence_after();
                soft_sync();
#pragma unroll
                for (int c0 = 0; c0 < kRT; c0 += 16) {
                    uint32_t o[16];
                    tmem_ld16_sync(tO + lane_off + hh * kRT + c0, o);
                    if (rec) {   // (rows past the tile's last are written too, and never read)
                        float* dst = rec + (hh * kRT + c0) * kQ4D + l;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if constexpr (kCluster) dst[e * kQ4D] = __uint_as_float(o[e]);
                            else __stcg(dst + e * kQ4D, __uint_as_float(o[e]));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int row = row_s[hh * kRT + c0 + e];
                            const uint16_t v = f32_bf16_bits(__uint_as_float(o[e]) * move_s[hh * kRT + c0 + e]);
                            if (row >= 0) a.out[static_cast<size_t>(row) * kQ4D + l] = v;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) bad |= !(fabsf(__uint_as_float(o[e])) < INFINITY);
                }
                if constexpr (kCluster) fence_proxy_async_smem();   // (copies may be made there again)
                if (bad) *fail_s = 1;
                part = 1;   // a partial run that is not the CTA's first is its last
                tc_fence_before();
                soft_sync();   // red_s and nm_s read by everyone before the next run writes them
                if (lane == 0) mbar_arrive(o_free);
                ++seg;
            }
        } while (again());
        if constexpr (kCluster) {   // no page of the unit fell to this CTA
            if (seg == 0 && tid < kRows)
                *reinterpret_cast<float2*>(smem + kOffRing + (kRows * kQ4D + 2 * tid) * 4) = make_float2(-INFINITY, 0.f);
        }
    }
    __syncwarp();
    if constexpr (kCluster) {
        cluster_sync_warp();   // every CTA's partial is there
        cg::cluster_group cluster = cg::this_cluster();
        const int u = blockIdx.x / wk.cluster, b = u / wk.U, ub = u - b * wk.U, g = ub / wk.row_tiles;
        const int row0 = (ub - g * wk.row_tiles) * wk.tile_rows, nrows = min(wk.tile_rows, a.R * a.G - row0);
        for (int r = rank + wk.cluster * warp; r < nrows; r += wk.cluster * (kThreads / 32)) {
            const int gr = row0 + r, j = gr * wk.inv_g >> 16;
            auto get = [&](int i, float2& ml, float4& o) {
                const float* rec = reinterpret_cast<const float*>(cluster.map_shared_rank(smem + kOffRing, i));
                ml = *reinterpret_cast<const float2*>(rec + kRows * kQ4D + 2 * r);
                o = *(reinterpret_cast<const float4*>(rec + r * kQ4D) + lane);
            };
            join_row(wk.cluster, get, a.out + (static_cast<size_t>(b * a.R + j) * a.Hq + g * a.G + gr - j * a.G) * kQ4D);
        }
        __syncwarp();
        cluster_sync_warp();   // this CTA's partial has been read
    }
    if constexpr (!kCluster) pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the partial rows of the units that lie in several CTAs' runs, a warp a row.
__global__ void __launch_bounds__(kCombineThreads)
    combine_q4_kernel(AttnQ4Args a, Work wk, const float* __restrict__ ws, int grid) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int gr = blockIdx.x * (kCombineThreads / 32) + (threadIdx.x >> 5);
    if (gr >= a.R * a.G) return;
    const int b = blockIdx.y / a.Hkv, g = blockIdx.y % a.Hkv;
    const int rt = gr / wk.tile_rows, r = gr % wk.tile_rows;
    const int2 sums = work_sums(a, b);
    const int W = sums.x * wk.U, n = active_ctas(W, grid);
    const int np = ctx_pages(ctx_len(a, b));
    const int w0 = sums.y * wk.U + (g * wk.row_tiles + rt) * (np + 1), w1 = w0 + np + 1;
    const int i0 = cta_of(W, w0, n), i1 = cta_of(W, w1 - 1, n);
    const bool later = static_cast<int64_t>(w0) * n > static_cast<int64_t>(W) * i0;   // w0 is past CTA i0's first page
    if (i0 == i1) return;   // one CTA had the whole unit and wrote its rows
    auto get = [&](int i, float2& ml, float4& o) {
        // a unit that starts inside CTA i0's run is its second partial
        const float* rec = ws + (static_cast<size_t>(i0 + i) * 2 + (i == 0 && later ? 1 : 0)) * kRecFloats;
        ml = __ldcg(reinterpret_cast<const float2*>(rec + kRows * kQ4D + 2 * r));
        o = __ldcg(reinterpret_cast<const float4*>(rec + r * kQ4D) + lane);
    };
    join_row(i1 - i0 + 1, get,
             a.out + ((static_cast<size_t>(b) * a.R + gr / a.G) * a.Hq + g * a.G + gr % a.G) * kQ4D);
}

Work work_of(int R, int G, int Hkv) {
    Work w{};
    const int rows = R * G;
    w.row_tiles = (rows + kRows - 1) / kRows;
    w.tile_rows = (rows + w.row_tiles - 1) / w.row_tiles;
    w.U = Hkv * w.row_tiles;
    w.inv_g = (65536 + G - 1) / G;
    return w;
}

template <int kRT, bool kCluster>
cudaError_t prepare() {
    static PerDeviceOnce once;
    return once.run([]() {
        return cudaFuncSetAttribute(attn_q4_kernel<kRT, kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
}

// Clusters of c CTAs (one an SM) that can be resident at once; 0 where that cannot be asked.
int resident_clusters(int c) {
    static std::mutex mu;
    static int cache[64][kMaxCluster + 1] = {};   // + 1
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 0;
    }
    std::lock_guard<std::mutex> lk(mu);
    if (cache[dev][c]) return cache[dev][c] - 1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (prepare<32, true>() != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, attn_q4_kernel<32, true>, &cfg) != cudaSuccess)
        n = 0;
    cudaGetLastError();
    cache[dev][c] = n + 1;
    return n;
}

// How the work is split, in pages that the busiest CTA takes: evenly over the SMs
// and joined by a second kernel, or a cluster of 2, 4 or 8 CTAs for each unit, joined
// on chip, whose barriers and remote reads cost about two pages.  The second kernel and
// the partials' way through L2 cost about ten, and three for each ten partials of a unit.
// Measured, cluster against even split: 5 x 12 heads over 2 of 4096 positions 10.4 and
// 11.8 us, of 16384 (the rule splits there) 18.1 and 19.2; 9 x 28 over 4, 4096: 11.5 and
// 14.6, 12288: 17.4 and 17.4, 16384: 20.3 and 17.4; 65 x 28 over 4, 4096: 17.0 and 19.7,
// 8192: 22.9 and 24.6.  The table's capacity decides, as the lengths are on the device: 5
// x 12 heads over 4096 positions take 12.3 us with a table for 131072.
void plan(Work& w, int B, int max_pages, int& grid) {
    const int64_t units = static_cast<int64_t>(B) * w.U, pages = units * (static_cast<int64_t>(max_pages) + 1);
    const int sms = device_sm_count();
    const int64_t most = pages / kGrain;
    grid = static_cast<int>(most < 1 ? 1 : most < sms ? most : sms);
    w.cluster = 0;
    int64_t best = (pages + grid - 1) / grid + (grid > 1 ? 10 + 3 * (grid / units) / 10 : 0);
    for (int c = kMaxCluster; c >= 2; c /= 2) {
        const int64_t cost = (max_pages + c) / c + 2;
        if (cost >= best || units > resident_clusters(c)) continue;
        best = cost;
        w.cluster = c;
    }
    if (w.cluster) grid = static_cast<int>(units) * w.cluster;
}

template <int kRT>
cudaError_t launch_rt(const AttnQ4Args& a, const Work& w, int grid, float* ws, cudaStream_t st) {
    if (w.cluster == 0) {
        const cudaError_t e = prepare<kRT, false>();
        if (e != cudaSuccess) return e;
        return launch_pdl(attn_q4_kernel<kRT, false>, dim3(grid), dim3(kThreads), kSmemBytes, st, a, w, ws);
    }
    const cudaError_t e = prepare<kRT, true>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = w.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, attn_q4_kernel<kRT, true>, a, w, ws);
}

}  // namespace

size_t attn_q4_workspace(const sv_attn_shape& s) {
    Work w = work_of(s.R, s.Hq / s.Hkv, s.Hkv);
    int grid;
    plan(w, s.B, (s.T_cap + kQ4Page - 1) / kQ4Page, grid);
    return grid > 1 && w.cluster == 0 ? static_cast<size_t>(grid) * 2 * kRecFloats * sizeof(float) : 0;
}

cudaError_t launch_verify_attn_q4(const AttnQ4Args& a, void* ws, cudaStream_t st) {
    Work w = work_of(a.R, a.G, a.Hkv);
    int grid;
    plan(w, a.B, a.max_pages, grid);
    float* part = static_cast<float*>(ws);
    const cudaError_t e = w.tile_rows <= 32 ? launch_rt<16>(a, w, grid, part, st) : launch_rt<32>(a, w, grid, part, st);
    if (e != cudaSuccess || grid == 1 || w.cluster != 0) return e;
    return launch_pdl(combine_q4_kernel, dim3((a.R * a.G + 7) / 8, a.B * a.Hkv), dim3(kCombineThreads), 0, st, a, w, part, grid);
}

}  // namespace sv
