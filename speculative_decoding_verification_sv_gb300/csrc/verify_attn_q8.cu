// verify_attn_q8.cu -- attention of the k+1 verify rows over an 8-bit paged KV
// cache (format: kv_q8.cuh) and the block's own bf16 K/V.
//
// out = softmax(scale q K^T) V over the cached positions and the block rows that the
// row may see.  The cache is half of the bf16 cache's bytes, and what bounds the kernel
// is to be reading them.
//
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T (M = 128 keys or dims,
// N = 64 query rows), so that a block of few rows still fills the tensor core.
//   S^T: lane = key, column = query row.  K's codes are e4m3 and lie in memory as the
//        swizzled tile that the MMA reads: they go from memory to shared memory to the
//        product (kind::f8f6f4) without passing a register.  Q has to be e4m3 then, and
//        is, without loss: a bf16 has 8 significant bits, and the nearest e4m3 to a
//        value and the e4m3 of what that leaves hold 4 + 4 (the remainder of a
//        rounding to 4 bits is at most half a step, 8 halves of which are 4 bits).  So
//        K Q^T is K Q1^T + K Q2^T into one accumulator.  A row of Q is in units of a
//        power of two that takes its largest element to (224, 448], and what is lost
//        lies below 2^-10 of such a unit: 2^-17.8 of the row's largest element.
//        Scales of Q's rows and of K's runs, powers of two, multiply the scores.
//   P:   exp2(s - m), bf16, written by the key's thread as one line of
//        [keys][64 rows] in shared memory, the MN-major B of the second product.
//   O^T: lane = dim, column = row.  P far above or below 1 has to be held to 8 bits,
//        which only bf16 does: V's codes are made bf16 by the warps that hold a dim each
//        (a permute, a shift, a mask and a product for two codes) and are the A operand
//        in tensor memory.
// The block's K rows are held as Q's are, two e4m3 in units of the row's own (four
// products); its V rows are bf16 as they are.
// A row's maximum runs across lanes here, so it is not formed: P is taken against
// a reference, the row's score with the run's first key.  bf16 and fp32 have the
// same range, so nothing is lost by a P far above 1 as long as no sum reaches
// kMostSum; a run where one does (some score 60 powers of two above the first
// key's) is done again with the reference moved to the maximum every step.  So is
// one where a row's sum stays below kLeastSum: its reference is a key that it does
// not see, or 0 for a score that is not finite, and its P may all be 0.
//
// Work: units and runs as in attn_cache.cuh.  A unit that lies in several CTAs' runs
// leaves partials in the workspace -- at most two a CTA -- and a second small kernel
// joins them; a cluster's partials stay in shared memory and are joined over it.
//
// Warps: 8 softmax (TMEM quadrant w % 4, half of the tile's rows each), 4 that split
// rows of bf16 into e4m3 pairs (Q of the next run, K of the block), 4 that unpack V, one
// that issues the copies (two pages of K and V, 32 KB, a ring stage), one the MMAs.
#include <cooperative_groups.h>
#include <math.h>

#include <mutex>
#include <type_traits>

#include "attn_cache.cuh"
#include "kv_q8.cuh"
#include "sv_internal.h"

namespace cg = cooperative_groups;

namespace sv {
namespace {

constexpr int kStepKeys = 128;            // two pages
constexpr int kStages = 4;
constexpr int kTileBytes = kStepKeys * kQ8D;     // codes of a step's K, or V
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kMaxR = 128;
constexpr int kSoftWarps = 8, kSplitWarp = 8, kVWarp = 12, kTmaWarp = 16, kMmaWarp = 17, kThreads = 32 * 18;
constexpr float kMostSum = 0x1p64f;       // of a row's P, for the result to stand,
constexpr float kLeastSum = 0.5f;         // and at least (a reference that the row sees gives 1)
constexpr int kRecFloats = kRows * (kQ8D + 2);   // a partial: O [64][128], then (m, l) [64]
constexpr int kCombineThreads = 256;
constexpr int kMaxCluster = 8;

// TMEM columns: two V operands (64 columns: 128 bf16 each), two S^T, one O^T
constexpr uint32_t kColV = 0, kColS = 128, kColO = 256, kTmemCols = 512;

constexpr int kOffQ = 0;                                  // 2 x [2 parts][64 rows][128 B], swizzled
constexpr int kQBytes = 2 * kRows * kQ8D;
constexpr int kOffP = kOffQ + 2 * kQBytes;                // kPBufs x [128 keys][128 B], swizzled
constexpr int kPBufs = 3;
constexpr int kPBytes = kStepKeys * kRows * 2;
constexpr int kOffRing = kOffP + kPBufs * kPBytes;        // kStages x [K 128 keys][V 2 pages]
// Scales of a step: of a context step K's two pages [2][4], V's [2][4]; of a block
// [128 rows].  More slots than ring stages: a stage is free when its codes have been
// read, which the scores' readers are up to two steps behind.
constexpr int kOffScl = kOffRing + kStages * kStageBytes;
constexpr int kSclSlots = 8, kSclBytes = 512;
constexpr int kOffBar = kOffScl + kSclSlots * kSclBytes;
constexpr int kOffNm = kOffBar + 320;                     // [64] -m, m the rows' references
constexpr int kOffMove = kOffNm + kRows * 4;              // [64] what O and l of the row are multiplied by
constexpr int kOffRed = kOffMove + kRows * 4;             // [4 quadrants][64]
constexpr int kOffFail = kOffRed + 4 * kRows * 4;         // a sum left its range; then where the runs start
constexpr int kOffPar = kOffFail + 32;                    // [128] parents
constexpr int kOffAnc = kOffPar + kMaxR * 4;              // [128][2] 64-bit path masks
constexpr int kOffRow = kOffAnc + kMaxR * 16;             // [64] (sequence, block row, head) of a tile row, -1 past the last
constexpr int kOffUnit = kOffRow + kRows * 4;             // [2][64] units of the query rows
// [3 runs][128 dims][2] block rows whose V is not finite there.  Three, as V is unpacked up to
// two steps ahead of O^T, which can be two runs, and the epilogue behind that reads this.
constexpr int kOffInf = kOffUnit + 2 * kRows * 4;
constexpr int kSmemBytes = kOffInf + 3 * kQ8D * 16;
static_assert(kOffInf % 16 == 0, "16-byte masks");
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
static_assert(kOffRing % 1024 == 0, "swizzled tiles");
static_assert(kRecFloats * 4 <= kStages * kStageBytes, "a cluster's partial in the ring");
// a slot is written again kSclSlots steps on, by when the scores of the step kStages + 2
// before that one have been read
static_assert(kSclSlots >= kStages + 2, "scale slots");

// Instruction descriptor of tcgen05.mma kind::f8f6f4: e4m3 A and B (K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem], 32 bytes of K, issued by one thread.
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint16_t f32_bf16_bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// One row of bf16, 8 dims in each lane of a half-warp (dims 8 (lane & 15) ..), into row r
// of two swizzled tiles of e4m3 (`second` bytes apart) and its unit.
__device__ __forceinline__ void split_row(uint4 x, int r, uint8_t* tile, int second, float* unit) {
    const int ch = threadIdx.x & 15;
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m2 = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, w[i] & 0x7fff7fffu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    const uint32_t m = max(m2 >> 16, m2 & 0xffffu);
    const bool bad = m >= 0x7f80u;   // NaN or infinity: the row's scores are NaN
    const int e = bad ? 0 : q8_exponent(__uint_as_float(m << 16));
    const float rs = q8_pow2(-e);
    uint32_t c1[2], c2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v[4] = {__uint_as_float(w[2 * h] << 16) * rs, __uint_as_float(w[2 * h] & 0xffff0000u) * rs,
                      __uint_as_float(w[2 * h + 1] << 16) * rs, __uint_as_float(w[2 * h + 1] & 0xffff0000u) * rs};
        c1[h] = q8_codes4(v[0], v[1], v[2], v[3]);
        float y[4];
        q8_values4(c1[h], y);
        c2[h] = q8_codes4(v[0] - y[0], v[1] - y[1], v[2] - y[2], v[3] - y[3]);
        if (bad) c1[h] = c2[h] = 0x7f7f7f7fu;
    }
    uint8_t* at = tile + r * 128 + (((ch >> 1) ^ (r & 7)) << 4) + (ch & 1) * 8;
    *reinterpret_cast<uint2*>(at) = make_uint2(c1[0], c1[1]);
    *reinterpret_cast<uint2*>(at + second) = make_uint2(c2[0], c2[1]);
    if (ch == 0) *unit = q8_pow2(e);
}

// kRT: rows a softmax thread takes; the tile's rows past 2 kRT do not exist (their
// columns of P stay zero)
template <int kRT, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1) attn_q8_kernel(CacheAttnArgs a, Work wk, float* __restrict__ ws) {
    constexpr int kLive = 2 * kRT;
    // (aligned by its declaration: addresses are then constants, not registers)
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* ring_full = bars;                   // [kStages]
    uint64_t* ring_empty = ring_full + kStages;   // [kStages] V unpacked (4 warps) and S^T formed
    uint64_t* ring_go = ring_empty + kStages;     // [kStages] free for a block's K
    uint64_t* v_full = ring_go + kStages;         // [2] V operand unpacked
    uint64_t* s_full = v_full + 2;                // [2] S^T formed
    uint64_t* s_empty = s_full + 2;               // [2] scores read
    uint64_t* p_full = s_empty + 2;               // [kPBufs] P written (and O rescaled): one each, as a warp may
                                                  // be two steps ahead of another
    uint64_t* pv_done = p_full + kPBufs;          // [2] O^T has the step (P and the V operand read)
    uint64_t* q_ready = pv_done + 2;              // [2] query rows there
    uint64_t* q_free = q_ready + 2;               // [2] the run's S^T are formed, and its units no longer wanted
    uint64_t* o_free = q_free + 2;                // O^T read by the epilogue
    uint64_t* o_done = o_free + 1;                // O^T has the run's last step (pv_done is no help there: two
                                                  // of its phases may be missing, and a wait passes at once)
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(o_done + 1);
    static_assert((3 * kStages + 14 + kPBufs) * 8 + 4 <= 320, "barrier area");
    float* nm_s = reinterpret_cast<float*>(smem + kOffNm);
    float* move_s = reinterpret_cast<float*>(smem + kOffMove);
    float* red_s = reinterpret_cast<float*>(smem + kOffRed);
    int32_t* par_s = reinterpret_cast<int32_t*>(smem + kOffPar);
    uint64_t* anc_s = reinterpret_cast<uint64_t*>(smem + kOffAnc);
    int* row_s = reinterpret_cast<int*>(smem + kOffRow);
    uint64_t* inf_s = reinterpret_cast<uint64_t*>(smem + kOffInf);
    auto scales = [](int it) { return reinterpret_cast<float*>(smem + kOffScl + it % kSclSlots * kSclBytes); };
    auto stage = [](int it) { return smem + kOffRing + it % kStages * kStageBytes; };

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *reinterpret_cast<volatile int*>(smem + kOffFail) = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], 5);
            mbar_init(&ring_go[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&v_full[i], 4);
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kSoftWarps);
            mbar_init(&pv_done[i], 1);
            mbar_init(&q_ready[i], 4);
            mbar_init(&q_free[i], 1 + kSoftWarps);
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

    // Every step, of the context or a block, has a ring stage: step `it` stage it %
    // kStages in its it / kStages-th use.
    if (warp == kTmaWarp) {
        // ---------------- page copies ----------------
        int it = 0;
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
                    for (int i = 0; i < 32 && i0 + i < np; i += 2, ++it) {
                        const int pa = __shfl_sync(0xffffffffu, pg, i), pb = __shfl_sync(0xffffffffu, pg, i + 1);
                        const bool two = i0 + i + 1 < np, la = pa >= 0, lb = two && pb >= 0;
                        const int s = it % kStages;
                        uint8_t* st = stage(it);
                        float* sc = scales(it);
                        wait(&ring_empty[s], ((it / kStages) & 1) ^ 1);
                        if (!la || (two && !lb)) {   // a page outside the pool reads as zeros
                            for (int p = 0; p < 2; ++p) {
                                if (p == 0 ? la : lb || !two) continue;
                                for (int x = lane; x < kQ8Codes / 16; x += 32) {
                                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                                    reinterpret_cast<uint4*>(st + p * kQ8Codes)[x] = z;
                                    reinterpret_cast<uint4*>(st + kTileBytes + p * kQ8Codes)[x] = z;
                                }
                                if (lane < 4) sc[4 * p + lane] = sc[8 + 4 * p + lane] = q8_pow2(kQ8MinExp);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&ring_full[s], ((la ? 2u : 0u) + (lb ? 2u : 0u)) * (kQ8Codes + 16u));
                            auto copy = [&](int p, int page) {
                                const size_t at = (static_cast<size_t>(page) * a.Hkv + g) * kQ8Bytes;
                                bulk_g2s(st + p * kQ8Codes, a.k_pool + at, kQ8Codes, &ring_full[s]);
                                bulk_g2s(sc + 4 * p, a.k_pool + at + kQ8Codes, 16, &ring_full[s]);
                                bulk_g2s(st + kTileBytes + p * kQ8Codes, a.v_pool + at, kQ8Codes, &ring_full[s]);
                                bulk_g2s(sc + 8 + 4 * p, a.v_pool + at + kQ8Codes, 16, &ring_full[s]);
                            };
                            if (la) copy(0, pa);
                            if (lb) copy(1, pb);
                        }
                        __syncwarp();
                    }
                }
                if (walk.block) {   // the stage of the block's K, whose writers do not follow the others' use of it
                    wait(&ring_empty[it % kStages], ((it / kStages) & 1) ^ 1);
                    if (lane == 0) mbar_arrive(&ring_go[it % kStages]);
                    __syncwarp();
                    ++it;
                }
            }
        } while (again());
    } else if (warp == kMmaWarp) {
        // ---------------- MMA issuer ----------------
        constexpr uint32_t id_s = idesc_e4m3_f32(128, kLive);
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
                        const int x = i & 1, s = i % kStages;
                        mbar_wait(&ring_full[s], (i / kStages) & 1, a.err);
                        mbar_wait(&s_empty[x], ((i >> 1) & 1) ^ 1, a.err);
                        tc_fence_after();
                        const uint64_t kd = smem_desc_sw128(smem_u32(stage(i)), 16, 1024);
                        const bool last = i == it + n - 1;
#pragma unroll
                        for (int kc = 0; kc < kQ8D / 32; ++kc)
                            tc_mma_e4m3(tS(x), kd + kc * 2, qd + kc * 2, id_s, kc > 0 ? 1u : 0u);
#pragma unroll
                        for (int kc = 0; kc < kQ8D / 32; ++kc)
                            tc_mma_e4m3(tS(x), kd + kc * 2, qd + (kQBytes / 2 >> 4) + kc * 2, id_s, 1u);
                        if (last && walk.block) {   // the remainders of the block's K
#pragma unroll
                            for (int kc = 0; kc < kQ8D / 32; ++kc)
                                tc_mma_e4m3(tS(x), kd + (kTileBytes >> 4) + kc * 2, qd + kc * 2, id_s, 1u);
#pragma unroll
                            for (int kc = 0; kc < kQ8D / 32; ++kc)
                                tc_mma_e4m3(tS(x), kd + (kTileBytes >> 4) + kc * 2, qd + (kQBytes / 2 >> 4) + kc * 2, id_s, 1u);
                        }
                        tc_commit(&s_full[x]);
                        tc_commit(&ring_empty[s]);
                        if (last) tc_commit(&q_free[seg & 1]);
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
    } else if (warp >= kVWarp) {
        // ---------------- V: a dim's codes to bf16 ----------------
        const int l = q4 * 32 + lane;   // TMEM lane: the dim
        int it = 0, seg = -1;
        bool waited = !early;
        do {
            while (walk.next(a, wk)) {
                ++seg;
                const size_t blk0 = (static_cast<size_t>(walk.cur_b) * a.Hkv + walk.cur_unit / wk.row_tiles) * a.R * kQ8D;
                // the block's rows, read at the end of the run by loads that wait for one
                // another, are brought near meanwhile (256 bytes a row; a thread a line or two)
                if (walk.block && waited)
                    for (int x = l; x < 2 * a.R; x += 128)
                        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.v_blk + blk0 + 64 * x));
                for (int st = 0; st < walk.ctx_steps(); ++st, ++it) {
                    const uint8_t* v = stage(it) + kTileBytes;
                    wait(&ring_full[it % kStages], (it / kStages) & 1);
                    // keys of the step that exist: what the others' codes hold is not looked
                    // at (0 * a V that is not finite would be NaN)
                    const int have = min(walk.cur_t - (walk.p0 + 2 * st) * kQ8Page, (walk.p1 - walk.p0 - 2 * st) * kQ8Page);
                    const uint4 f0 = reinterpret_cast<const uint4*>(scales(it))[2], f1 = reinterpret_cast<const uint4*>(scales(it))[3];
                    const uint32_t f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
                    // NaN rows: all dims' codes are then NaN, so a lane looks at four positions of one
                    // dim; and scales above 2^7, whose product with 2^120 bf16 cannot hold
                    uint32_t odd = q8_nan_bytes(*reinterpret_cast<const uint32_t*>(v + q8_v_off(lane >> 1, q4 * 32) + 4 * (lane & 1)));
#pragma unroll
                    for (int r = 0; r < 8; ++r) odd |= f[r] > 0x43000000u ? 1u : 0u;
                    const bool general = __any_sync(0xffffffffu, odd != 0u) || have < kStepKeys;
                    wait(&pv_done[it & 1], ((it >> 1) & 1) ^ 1);
                    tc_fence_after();
                    auto unpack = [&](auto general_c) {
                        constexpr bool kGeneral = decltype(general_c)::value;
#pragma unroll
                        for (int h = 0; h < 4; ++h) {   // 32 keys: two runs
                            uint32_t r[16];
#pragma unroll
                            for (int o = 0; o < 4; ++o) {
                                uint2 w = *reinterpret_cast<const uint2*>(v + q8_v_off(4 * h + o, l));
                                const uint32_t fs = f[2 * h + (o >> 1)];
                                // 2^120 times the scale, as a bf16 pair
                                uint32_t m = ((fs >> 23) + 120u) * 0x00800080u;
                                if constexpr (kGeneral) {
                                    const int left = have - 32 * h - 8 * o;   // keys of the octet that exist
                                    if (left < 8) {
                                        const uint64_t keep = left <= 0 ? 0ull : (1ull << 8 * left) - 1ull;
                                        w.x &= static_cast<uint32_t>(keep);
                                        w.y &= static_cast<uint32_t>(keep >> 32);
                                        if (left <= 0) m = 0u;
                                    }
                                    if (fs > 0x43000000u) m = q8_pow2_pair(127);
                                }
                                uint32_t p[4] = {q8_pair<0, 1>(w.x, 0u), q8_pair<2, 3>(w.x, 0u), q8_pair<0, 1>(w.y, 0u),
                                                 q8_pair<2, 3>(w.y, 0u)};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    uint32_t y = q8_mul2(p[k], m);
                                    if constexpr (kGeneral) {
                                        if (fs > 0x43000000u && have > 32 * h + 8 * o)
                                            y = q8_mul2(y, ((fs >> 23) - 7u) * 0x00800080u);
                                        y = q8_nan_pair(p[k], y);
                                    }
                                    r[4 * o + k] = y;
                                }
                            }
                            tmem_st16(tV(it & 1) + lane_off + 16 * h, r);
                        }
                    };
                    if (general) unpack(std::true_type{});
                    else unpack(std::false_type{});
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&v_full[it & 1]);
                        mbar_arrive(&ring_empty[it % kStages]);
                    }
                }
                if (walk.block) {
                    if (!waited) pdl_wait();
                    waited = true;
                    wait(&pv_done[it & 1], ((it >> 1) & 1) ^ 1);
                    tc_fence_after();
                    const uint16_t* src = a.v_blk + blk0 + l;
                    uint32_t most = 0u;   // the largest magnitude's bits (in either half)
                    uint64_t inf[2] = {0ull, 0ull};
                    auto unpack = [&](auto fix_c) {
#pragma unroll 1
                        for (int h = 0; h < 4; ++h) {
                            uint32_t r[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const int key = 32 * h + 2 * k;
                                uint32_t lo = key < a.R ? __ldg(src + key * kQ8D) : 0u;
                                uint32_t hi = key + 1 < a.R ? __ldg(src + (key + 1) * kQ8D) : 0u;
                                if constexpr (decltype(fix_c)::value) {
                                    if ((lo & 0x7f80u) == 0x7f80u) inf[h >> 1] |= 1ull << (key & 63), lo = 0u;
                                    if ((hi & 0x7f80u) == 0x7f80u) inf[h >> 1] |= 2ull << (key & 63), hi = 0u;
                                } else {
                                    most = max(most, max(lo & 0x7fffu, hi & 0x7fffu));
                                }
                                r[k] = lo | hi << 16;
                            }
                            tmem_st16(tV(it & 1) + lane_off + 16 * h, r);
                        }
                    };
                    unpack(std::false_type{});
                    // V that is not finite would reach the rows that do not see it (0 times it is NaN):
                    // it stays out of the product, and the epilogue adds it where it is seen
                    if (__any_sync(0xffffffffu, most >= 0x7f80u)) unpack(std::true_type{});
                    inf_s[(seg % 3 * kQ8D + l) * 2] = inf[0];
                    inf_s[(seg % 3 * kQ8D + l) * 2 + 1] = inf[1];
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_full[it & 1]);
                    // (an arrival before the block's K is there would count for the stage's use before)
                    wait(&ring_full[it % kStages], (it / kStages) & 1);
                    if (lane == 0) mbar_arrive(&ring_empty[it % kStages]);
                    ++it;
                }
            }
        } while (again());
        if (!waited) pdl_wait();
    } else if (warp >= kSplitWarp) {
        // ---------------- rows of bf16 to e4m3 pairs: Q, and the block's K ----------------
        if (early) pdl_wait();
        constexpr int kAhead = 8;   // rows a half-warp has in flight
        const int sub = 2 * (warp - kSplitWarp) + (lane >> 4), ch = lane & 15;   // half-warps take rows sub, sub + 8, ..
        int it = 0, seg = 0;
        uint32_t gone = 0;          // (bit s) parity of the next block in stage s
        do {
            while (walk.next(a, wk)) {
                const int g = walk.cur_unit / wk.row_tiles, row0 = walk.cur_unit % wk.row_tiles * wk.tile_rows;
                const int nrows = min(wk.tile_rows, a.R * a.G - row0);
                uint4 x[kAhead];
#pragma unroll
                for (int i = 0; i < kLive / 8; ++i) {
                    const int r = sub + 8 * i, gr = row0 + r, j = gr * wk.inv_g >> 16;
                    x[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < nrows)
                        x[i] = __ldg(reinterpret_cast<const uint4*>(
                                         a.q + (static_cast<size_t>(walk.cur_b * a.R + j) * a.Hq + g * a.G + gr - j * a.G) * kQ8D) + ch);
                }
                wait(&q_free[seg & 1], ((seg >> 1) & 1) ^ 1);
#pragma unroll
                for (int i = 0; i < kLive / 8; ++i)
                    split_row(x[i], sub + 8 * i, smem + kOffQ + (seg & 1) * kQBytes, kQBytes / 2,
                              reinterpret_cast<float*>(smem + kOffUnit) + (seg & 1) * kRows + sub + 8 * i);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_ready[seg & 1]);
                ++seg;
                it += walk.ctx_steps();
                if (walk.block) {
                    const int s = it % kStages;
                    const uint4* src = reinterpret_cast<const uint4*>(a.k_blk + (static_cast<size_t>(walk.cur_b) * a.Hkv + g) * a.R * kQ8D) + ch;
                    bool go = false;
#pragma unroll 1
                    for (int r0 = 0; r0 < a.R; r0 += 8 * kAhead) {
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            const int r = r0 + sub + 8 * i;
                            x[i] = make_uint4(0u, 0u, 0u, 0u);
                            if (r < a.R) x[i] = __ldg(src + r * (kQ8D / 8));
                        }
                        if (!go) {
                            wait(&ring_go[s], gone >> s & 1u);
                            gone ^= 1u << s;
                            go = true;
                        }
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            if (r0 + 8 * i < a.R)
                                split_row(x[i], r0 + sub + 8 * i, stage(it), kTileBytes, scales(it) + r0 + sub + 8 * i);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    named_barrier(3, 128);
                    if (warp == kSplitWarp && lane == 0) mbar_arrive(&ring_full[s]);
                    __syncwarp();
                    ++it;
                }
            }
        } while (again());
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
                    if (t < 0 || t > a.max_pages * kQ8Page) raise_error(a.err, SV_DEVERR_LENGTH);
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
                // (the rows' units; everything else that the split warps write comes by way of S^T)
                const float* unit_s = reinterpret_cast<const float*>(smem + kOffUnit) + (seg & 1) * kRows;
                wait(&q_ready[seg & 1], (seg >> 1) & 1);
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
                    // the key's scale: of its run, or of the block's row
                    const float* scl = scales(it);
                    const float ks = sc * (kGeneral && st >= nctx ? scl[l] : scl[l >> 4]);
                    // the rows that see this thread's key (bit e: row hh * kRT + e), in the
                    // steps where some do not: of the context, keys before the length (the
                    // second page of a step may be missing); block row l is seen from query
                    // rows l G on, or by the tree rows on whose path it lies
                    uint32_t seen = ~0u;
                    if constexpr (kGeneral) {
                        if (st < nctx) {
                            if ((walk.p0 + 2 * st) * kQ8Page + l >= min(walk.cur_t, walk.p1 * kQ8Page)) seen = 0u;
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
                            const float4 un = reinterpret_cast<const float4*>(unit_s + hh * kRT + c0)[i];
                            // (the scales first: codes times one of them can pass fp32's largest; and in the
                            // steps that may be `safe` the score is rounded before its reference is taken
                            // off, so that the largest gives 0 however large it is)
                            auto at = [&](uint32_t x, float u, float m) {
                                if constexpr (kGeneral) return __fadd_rn(__fmul_rn(__uint_as_float(x), u * ks), m);
                                else return fmaf(__uint_as_float(x), u * ks, m);
                            };
                            e[4 * i] = at(s[4 * i], un.x, nm.x);
                            e[4 * i + 1] = at(s[4 * i + 1], un.y, nm.y);
                            e[4 * i + 2] = at(s[4 * i + 2], un.z, nm.z);
                            e[4 * i + 3] = at(s[4 * i + 3], un.w, nm.w);
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
                                        const float e = __uint_as_float(s[i]) * (unit_s[hh * kRT + c0 + i] * -ks);
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
                                uint32_t s[16];
                                tmem_ld16_sync(tS(x) + lane_off + hh * kRT + c0, s);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float z = __fmul_rn(__uint_as_float(s[i]), unit_s[hh * kRT + c0 + i] * ks);
                                    const float m = warp_max(seen >> (c0 + i) & 1u ? z : -INFINITY);
                                    if (lane == 0) red_s[q4 * kRows + hh * kRT + c0 + i] = m;
                                }
                            }
                            soft_sync();
                            if (tid < kLive) {
                                // up, or where no score was finite so far (P, the sum and O are
                                // 0 then) to wherever the maximum is
                                const float m = fmaxf(fmaxf(red_s[tid], red_s[kRows + tid]),
                                                      fmaxf(red_s[2 * kRows + tid], red_s[3 * kRows + tid]));
                                const float was = -nm_s[tid];
                                float move = 1.0f;
                                if (m > -INFINITY && (!found || m > was)) {
                                    if (found) move = fast_exp2(was - m);
                                    nm_s[tid] = -m;
                                    found = true;
                                }
                                move_s[tid] = move;
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
                const bool ragged = nctx > 0 && ((walk.p1 - walk.p0) & 1 || walk.p1 * kQ8Page > walk.cur_t);
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
                    *reinterpret_cast<float2*>(rec + kRows * kQ8D + 2 * tid) = make_float2(-nm_s[tid], lsum);
                tc_fence_after();
                soft_sync();
                const uint64_t inf0 = inf_s[(seg % 3 * kQ8D + l) * 2], inf1 = inf_s[(seg % 3 * kQ8D + l) * 2 + 1];
#pragma unroll
                for (int c0 = 0; c0 < kRT; c0 += 16) {
                    uint32_t o[16];
                    tmem_ld16_sync(tO + lane_off + hh * kRT + c0, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) bad |= !(fabsf(__uint_as_float(o[e])) < INFINITY);
                    if (walk.block && (inf0 | inf1) != 0ull) {   // (rare) V that is not finite and that the row sees
#pragma unroll 1
                        for (int e = 0; e < 16; ++e) {
                            const int j = (row0 + hh * kRT + c0 + e) * wk.inv_g >> 16;   // (any row past the tile's last)
                            if (j >= a.R) continue;
                            uint64_t m0 = inf0, m1 = inf1;
                            if (tree) m0 &= anc_s[2 * j], m1 &= anc_s[2 * j + 1];
                            else m0 &= ~0ull >> (63 - min(j, 63)), m1 &= j < 64 ? 0ull : ~0ull >> (127 - j);
                            float add = 0.f;
                            for (; m0 | m1; (m0 ? m0 : m1) &= (m0 ? m0 : m1) - 1ull) {
                                const int key = m0 ? __ffsll(m0) - 1 : 63 + __ffsll(m1);
                                add += __uint_as_float(static_cast<uint32_t>(__ldg(
                                    a.v_blk + ((static_cast<size_t>(b) * a.Hkv + g) * a.R + key) * kQ8D + l)) << 16);
                            }
                            if (add != 0.f) {   // (NaN too)
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    if (i == e) o[i] = __float_as_uint(__uint_as_float(o[i]) + add);
                            }
                        }
                    }
                    if (rec) {   // (rows past the tile's last are written too, and never read)
                        float* dst = rec + (hh * kRT + c0) * kQ8D + l;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if constexpr (kCluster) dst[e * kQ8D] = __uint_as_float(o[e]);
                            else __stcg(dst + e * kQ8D, __uint_as_float(o[e]));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int row = row_s[hh * kRT + c0 + e];
                            const uint16_t v = f32_bf16_bits(__uint_as_float(o[e]) * move_s[hh * kRT + c0 + e]);
                            if (row >= 0) a.out[static_cast<size_t>(row) * kQ8D + l] = v;
                        }
                    }
                }
                if constexpr (kCluster) fence_proxy_async_smem();   // (copies may be made there again)
                if (bad) *fail_s = 1;
                part = 1;   // a partial run that is not the CTA's first is its last
                tc_fence_before();
                soft_sync();   // red_s and nm_s read by everyone before the next run writes them
                if (lane == 0) {
                    mbar_arrive(o_free);
                    mbar_arrive(&q_free[seg & 1]);
                }
                ++seg;
            }
        } while (again());
        if constexpr (kCluster) {   // no page of the unit fell to this CTA
            if (seg == 0 && tid < kRows)
                *reinterpret_cast<float2*>(smem + kOffRing + (kRows * kQ8D + 2 * tid) * 4) = make_float2(-INFINITY, 0.f);
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
                ml = *reinterpret_cast<const float2*>(rec + kRows * kQ8D + 2 * r);
                o = *(reinterpret_cast<const float4*>(rec + r * kQ8D) + lane);
            };
            join_row(wk.cluster, get, a.out + (static_cast<size_t>(b * a.R + j) * a.Hq + g * a.G + gr - j * a.G) * kQ8D);
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
    combine_q8_kernel(CacheAttnArgs a, Work wk, const float* __restrict__ ws, int grid) {
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
        ml = __ldcg(reinterpret_cast<const float2*>(rec + kRows * kQ8D + 2 * r));
        o = __ldcg(reinterpret_cast<const float4*>(rec + r * kQ8D) + lane);
    };
    join_row(i1 - i0 + 1, get,
             a.out + ((static_cast<size_t>(b) * a.R + gr / a.G) * a.Hq + g * a.G + gr % a.G) * kQ8D);
}

template <int kRT, bool kCluster>
cudaError_t prepare() {
    static PerDeviceOnce once;
    return once.run([]() {
        return cudaFuncSetAttribute(attn_q8_kernel<kRT, kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
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
    if (prepare<32, true>() != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, attn_q8_kernel<32, true>, &cfg) != cudaSuccess)
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
cudaError_t launch_rt(const CacheAttnArgs& a, const Work& w, int grid, float* ws, cudaStream_t st) {
    if (w.cluster == 0) {
        const cudaError_t e = prepare<kRT, false>();
        if (e != cudaSuccess) return e;
        return launch_pdl(attn_q8_kernel<kRT, false>, dim3(grid), dim3(kThreads), kSmemBytes, st, a, w, ws);
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
    return cudaLaunchKernelEx(&cfg, attn_q8_kernel<kRT, true>, a, w, ws);
}

}  // namespace

size_t attn_q8_workspace(const sv_attn_shape& s) {
    Work w = work_of(s.R, s.Hq / s.Hkv, s.Hkv);
    int grid;
    plan(w, s.B, (s.T_cap + kQ8Page - 1) / kQ8Page, grid);
    return grid > 1 && w.cluster == 0 ? static_cast<size_t>(grid) * 2 * kRecFloats * sizeof(float) : 0;
}

cudaError_t launch_verify_attn_q8(const CacheAttnArgs& a, void* ws, cudaStream_t st) {
    Work w = work_of(a.R, a.G, a.Hkv);
    int grid;
    plan(w, a.B, a.max_pages, grid);
    float* part = static_cast<float*>(ws);
    const cudaError_t e = w.tile_rows <= 32 ? launch_rt<16>(a, w, grid, part, st) : launch_rt<32>(a, w, grid, part, st);
    if (e != cudaSuccess || grid == 1 || w.cluster != 0) return e;
    return launch_pdl(combine_q8_kernel, dim3((a.R * a.G + 7) / 8, a.B * a.Hkv), dim3(kCombineThreads), 0, st, a, w, part, grid);
}

}  // namespace sv
