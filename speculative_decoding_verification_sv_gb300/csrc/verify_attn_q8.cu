// verify_attn_q8.cu -- attention of the k+1 verify rows over an 8-bit paged KV
// cache (format: kv_q8.cuh) and the block's own bf16 K/V.
//
// out = softmax(scale q K^T) V over the cached positions and the block rows that the
// row may see.  Both products run transposed, S^T = K Q^T and O^T = V^T P^T (M = 128 keys or
// dims, N = the tile's query rows, 32 or 64), so that a block of few rows still fills the
// tensor core.
//   S^T: lane = key, column = query row.  K's codes are e4m3 and lie in memory as the
//        swizzled tile that the MMA reads: they go from memory to shared memory to the
//        product (kind::f8f6f4) without passing a register.  Q has to be e4m3 then, and
//        is, without loss: a bf16 has 8 significant bits, and the nearest e4m3 to a
//        value and the e4m3 of what that leaves hold 4 + 4 (the remainder of a
//        rounding to 4 bits is at most half a step, 8 halves of which are 4 bits).  So
//        K Q^T is K Q1^T + K Q2^T.  A row of Q is in units of a
//        power of two that takes its largest element to (224, 448], and what is lost
//        lies below 2^-10 of such a unit: 2^-17.8 of the row's largest element.
//        Scales of Q's rows and of K's runs, powers of two, multiply the scores.
//   P:   exp2(s - m), f16, written by the key's thread as one line of
//        [keys][64 rows] in shared memory, the MN-major B of the second product.
//   O^T: lane = dim, column = row.  V's codes are made f16 by the warps that hold a dim
//        each (one conversion and one product by the run's scale for two codes) and are
//        the A operand in tensor memory; f16, because it holds P to 11 bits, an eighth of
//        bf16's rounding (0.0017 of the result against 0.0023), and every e4m3.  What it
//        lacks is range.  V is therefore in units of the largest scale of the run's first two
//        pages, 2^kVUp of it (a value is exact where its own scale is no less than 2^-11
//        of that, which is looked at; one too large for f16 makes O infinite), and P is 2^kUp
//        at a reference, below.
// The block's K rows are held as Q's are, two e4m3 in units of the row's own (four
// products).  Its V rows may be of any size, whether seen or not, and stay bf16 in V's units; its P is
// in two bf16 parts then (16 bits).  (A V too large in those units is infinite there, and O not finite:
// the run is done again, in the end without units; so is one whose units are so large that V could be
// lost.)  What of them is not finite is kept out of the product and added to the rows that see it at
// the end.
// A row's maximum runs across lanes here, so it is formed once, over the first 32 keys
// of the run (of the block, where the run has it: the row's own key and those next to
// it), and is the row's reference m for the whole run.  P is 2^-5 at the reference: a
// score 21 powers of two above it makes P infinite, and a P below 2^-25, a weight 2^-20
// of the reference's, is lost.  A run whose O is not finite, or where a row's sum is so
// small that what was lost could matter (kLost), is done again with references that the sums
// give, P then summing to 2^15.  Where they give none (the reference was a key that the row does
// not see, or none was finite), where V's scales lie further apart than f16 holds, and where that
// fails too, the run is done without f16: V in bf16 in units of 1, as the read-back gives it, P in two
// bf16 parts as the block's is, references from the sums (then 1) or rising with the maximum.
// (64 single tokens x 28 heads, where each token scores the first position 30 nats above itself:
// 67 us for 44, where one of the 64 does 51; 16 sequences 58 for 35.  Without f16: 92, 66 and 87.)
//
// What bounds it, in us of graph replays over inputs larger than L2 (heads and positions as
// named).  16 sequences x 9 rows, 28 heads over 4, 8192 positions: 34.5, for 137 MB, which take
// 20.1 at copy rate; 64 single tokens of up to 4097: 44.0 (175 MB, 25.7).  CTAs that stream reach
// 5.5 to 5.9 TB/s; the rest is the start and the end of a run, chains of steps that each run
// once, most of whose instructions come from L2 then: from the launch to the end of the
// block's step 13,000 cycles with tiles of more than 32 rows (Q's rows made e4m3 2000, the
// block's K 2300, its scores 1500, references 2500, P 2400: the last three take half of that
// once their code is there), 7000 with others; the sums, O and their join 4000.  A CTA that goes on
// to another unit pays 6000 of these again.  A step of two pages takes 1100 and 1300 cycles:
// 112 and 128 KB pass shared memory at 128 bytes a cycle.  5 rows x 12 heads over 2, 4096: 9.8, and
// 100001 positions 18.9 (floor 7.5), both latency: few pages a CTA.  A tree of 65 rows: 24.6; eight
// tiles of rows a head stream the same pages, 17 steps each.
// Tried: P in bf16; an MMA warp for both products, and one copier (a step waits for the
// other's); 16 softmax warps of 16 rows (tensor memory reads and references double); two
// groups of softmax warps in turn (16 sequences 42 -> 51.8: spills); the block as a run's second
// step, so that references are of 32 keys of the cache (64 single tokens 43.4 -> 49.3: the first
// pages come late); the next 32 pages' table and scales fetched ahead (43.4 -> 45.4); V's scales looked
// at by the warps that convert (44.4 -> 50.1), zeros told from what f16 loses by reading their codes
// again (587 where half of V is zeros); one code for all passes (44.0 -> 48 to 54).
//
// Work: units and runs as in attn_cache.cuh.  A unit that lies in several CTAs' runs
// leaves partials in the workspace -- at most two a CTA -- and a second small kernel
// joins them; a cluster's partials stay in shared memory and are joined over it.  A run
// takes its block first: those rows are there before the first page.
//
// Warps: 8 softmax (TMEM quadrant w % 4, half of the tile's rows each), 4 that convert
// (Q and the block's K to e4m3 pairs, then V, a quadrant of the dims each), one each that
// copies K and V (two pages of both, 32 KB, are a ring stage; a copy takes 230 cycles to
// issue, so that one warp for both held a step up), and one for the MMAs of either product.
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
constexpr int kSoftWarps = 8, kConvWarp = 8, kConvWarps = 4, kTmaWarp = 12, kQkWarp = 14, kPvWarp = 15,
              kThreads = 32 * 16;
constexpr int kVUp = 4;                   // V is in units of 2^kVUp of its first scales
// f16 holds a run exactly whose scale is 2^-15 of the unit or more (its steps end at 2^-24, e4m3's
// at 2^-9), 2^-kVDown of the largest scale there.  One below that is left to the last pass, but
// for those of the least scale there is: zeros, or as good (448 * 2^-120 at most).  (The warp that
// copies V looks at the scales, which it has in registers.)
constexpr int kVDown = 15 - kVUp;
constexpr int kMostUnit = 20;             // beside a block; its V of 2^-106 and more is exact then
constexpr float kUp = -5.0f;              // P is 2^kUp at the reference;
constexpr float kUpSum = 15.0f;           // where the sums gave the reference, they are 2^kUpSum,
constexpr float kUpWide = 0.0f;           // or, in the last pass, 2^kUpWide;
constexpr float kSlack = 4.0f;            // where it rises with the maximum, it stays up to that far below
// A row's P sum to kLost times the keys or the run is done again: roundings below f16's smallest
// steps, 2^-25 at most for each key, then move the row by at most 2^-8 of the mean |V| if all of
// them went one way, and by that over the root of the keys as they do.  (A row that sees one of
// 4096 keys alone, by the reference, sums to 2^-5, which is kLost times those.  Single tokens
// have one key of the block for a reference: 64 of them x 28 heads, whose K had a few dims six
// times the others, had one done again, 51 us for 44, in every eighth call with kUp = -4, in one of
// thirty with -5.)
constexpr float kLost = 0x1p-17f;
// So is one that sums to kMostSum: the block's P is bf16 and reaches 2^128, where the row's own
// key is not among those that give its reference, and 1 / sum is 0 from 2^126 on.
constexpr float kMostSum = 0x1p64f;
constexpr float kLeastSum = 0x1p-100f;    // sums from here on give a reference for that,
constexpr int kKept = 4;                  // and so many runs of a CTA keep theirs
constexpr int kRecFloats = kRows * (kQ8D + 2);   // a partial: O [64][128], then (m, l) [64]
constexpr int kCombineThreads = 256;
constexpr int kMaxCluster = 8;

// TMEM columns: two V operands (64 columns: 128 f16 each), kSBufs S^T, one O^T
constexpr int kSBufs = 3;
constexpr uint32_t kColV = 0, kColS = 128, kColO = kColS + kSBufs * 64, kTmemCols = 512;

constexpr int kOffQ = 0;                                  // 2 x [2 parts][64 rows][128 B], swizzled
constexpr int kQBytes = 2 * kRows * kQ8D;
constexpr int kOffP = kOffQ + 2 * kQBytes;                // kPBufs x [128 keys][128 B], swizzled
constexpr int kPBufs = 3;
constexpr int kPBytes = kStepKeys * kRows * 2;
constexpr int kOffRing = kOffP + kPBufs * kPBytes;        // kStages x [K 128 keys][V 2 pages]
// Scales of a step: of a context step K's two pages [2][4], V's [2][4]; of a block
// [128 rows].  More slots than ring stages: a stage is free when its codes have been
// read, which the scores' readers are up to kSBufs steps behind.
constexpr int kOffScl = kOffRing + kStages * kStageBytes;
constexpr int kSclSlots = 8, kSclBytes = 512;
constexpr int kOffBar = kOffScl + kSclSlots * kSclBytes;
constexpr int kOffNm = kOffBar + 320;                     // [64] -m, m the rows' references
constexpr int kOffMove = kOffNm + kRows * 4;              // [64] what O and l of the row are multiplied by
constexpr int kOffRed = kOffMove + kRows * 4;             // [4 quadrants][64]
// [12] (bit r) run r failed; where the runs start [5]; its sums give no references; a wait gave up; f16
// does not hold its V; it failed in the second pass
constexpr int kFailed = 0, kNoSums = 6, kNoF16 = 8, kFailedAgain = 9;
constexpr int kOffFail = kOffRed + 4 * kRows * 4;
constexpr int kOffPar = kOffFail + 48;                    // [128] parents
constexpr int kOffAnc = kOffPar + kMaxR * 4;              // [128][2] 64-bit path masks
constexpr int kOffRow = kOffAnc + kMaxR * 16;             // [64] (sequence, block row, head) of a tile row, -1 past the last
constexpr int kOffUnit = kOffRow + kRows * 4;             // [2][64] units of the query rows
// [3 runs][128 dims][2] block rows whose V is not finite there.  Three, as V is converted up to
// two steps ahead of O^T, which can be two runs, and the epilogue behind that reads this.
constexpr int kOffInf = kOffUnit + 2 * kRows * 4;
constexpr int kOffVExp = kOffInf + 3 * kQ8D * 16;         // [3 runs] exponent of V's unit
constexpr int kOffKept = kOffVExp + 16;           // [kKept][64] -m that the sums gave
constexpr int kSmemBytes = kOffKept + kKept * kRows * 4;
static_assert(kOffInf % 16 == 0, "16-byte masks");
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
static_assert(kOffRing % 1024 == 0, "swizzled tiles");
static_assert(kRecFloats * 4 <= kPBufs * kPBytes, "a partial in P's place");
// a slot is written again kSclSlots steps on, by when the scores of the step kStages +
// kSBufs before that one have been read
static_assert(kSclSlots >= kStages + kSBufs, "scale slots");

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

// Instruction descriptor of tcgen05.mma kind::f16: f16 A and B (MN-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32_bmn(int M, int N) {
    return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// two codes (16 bits) as an f16 pair: exact
__device__ __forceinline__ uint32_t f16x2_of_codes(uint32_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(c)));
    return r;
}

// A bounded wait on an mbarrier phase, of 2 s of wall time as the library's others; one that gives
// up is noted for the kernel's end, and the others then give up soon.  There are many, and code
// that is run once a step, or once, has to be short to be there in time.
__device__ __forceinline__ void bar_wait(uint64_t* bar, uint32_t parity, volatile int* late) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1; i < (1u << 28); ++i) {
        if (mbar_try_wait(bar, parity)) return;
        if ((i & 255u) != 0u) continue;
        if (*late != 0) return;
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > 2000000000ull) break;
    }
    *late = 1;
}

// A bulk copy of what is read once: it takes the place of other such lines in L2, not of
// the kernel's code or the partials (64 single tokens: 49.0 us without, 46.7 with).
__device__ __forceinline__ void bulk_g2s_once(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// Which of n buffers the next step uses, and the parity of that use.
struct Turn {
    int x = 0;
    uint32_t parity = 0u;
    __device__ __forceinline__ void next(int n) {
        if (++x == n) x = 0, parity ^= 1u;
    }
};

// A row of bf16, 8 dims in each lane of a half-warp (dims 8 (lane & 15) ..).
// Its largest magnitude's bits:
__device__ __forceinline__ uint32_t row_most(uint4 x) {
    uint32_t m2 = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    return max(m2 >> 16, m2 & 0xffffu);
}
// The row in units of 2^e as row r of two swizzled tiles of e4m3, `second` bytes apart.
// One that holds NaN or infinity is NaN.
__device__ __forceinline__ void split_row(uint4 x, bool bad, int e, int r, uint8_t* tile, int second) {
    const int ch = threadIdx.x & 15;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
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
}

// A bulk copy shared -> global by one thread, the wait for all of that thread's to have read
// their source, and for all of them.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(dst),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int kN>
struct Rows {
    uint4 v[kN];
};

// V of a context step as bf16 into tensor memory at `to`: dim l of 128 positions, `have` of which exist.
// A function of its own, as it is rare: an SM's instruction cache does not hold all that a CTA's warps
// run (64 single tokens 44 us; with this in line 46 to 55, by where it came to lie).
__device__ __noinline__ void wide_v(const uint8_t* v, const float* scale, int have, int l, uint32_t to) {
    const uint32_t up = q8_pow2_pair(120);
#pragma unroll 1
    for (int h = 0; h < 8; ++h) {   // 16 keys: a run
        const uint32_t sb = have > 16 * h ? __float_as_uint(scale[h]) >> 16 : 0u, s2 = sb | sb << 16;
        auto value = [&](uint32_t p) { return q8_nan_pair(p, q8_mul2(q8_mul2(p, up), s2)); };
        uint32_t r[8];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const uint2 w = *reinterpret_cast<const uint2*>(v + q8_v_off(2 * h + o, l));
            r[4 * o] = value(q8_pair<0, 1>(w.x, 0u));
            r[4 * o + 1] = value(q8_pair<2, 3>(w.x, 0u));
            r[4 * o + 2] = value(q8_pair<0, 1>(w.y, 0u));
            r[4 * o + 3] = value(q8_pair<2, 3>(w.y, 0u));
        }
        tmem_st8(to + 8 * h, r);
    }
}

// kRT: rows a softmax thread takes; the tile's rows past 2 kRT do not exist (what their
// columns of P and O hold is not looked at)
template <int kRT, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1) attn_q8_kernel(CacheAttnArgs a, Work wk, float* __restrict__ ws) {
    constexpr int kLive = 2 * kRT;
    // Q's two parts side by side in N, sixteen rows of one beside those of the other, and the scores
    // in two columns that are added when they are read: K then passes shared memory once a step
    // (four products of 63 cycles for eight of 40; 64 single tokens 45.7 -> 43.1 us, 100001 positions 19.3
    // -> 18.6).  The larger tile has no room for three such S^T in tensor memory, and with two its
    // steps take as long as with the parts one after the other (16 sequences 35.9 and 35.7 us).
    constexpr bool kStacked = kRT == 16;
    // (aligned by its declaration: addresses are then constants, not registers)
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* ring_full = bars;                   // [kStages]
    uint64_t* ring_empty = ring_full + kStages;   // [kStages] V converted and S^T formed
    uint64_t* ring_go = ring_empty + kStages;     // [kStages] free for a block's K
    uint64_t* v_full = ring_go + kStages;         // [2] V operand there
    uint64_t* s_full = v_full + 2;                // [kSBufs] S^T formed
    uint64_t* s_empty = s_full + kSBufs;          // [kSBufs] scores read
    uint64_t* p_full = s_empty + kSBufs;          // [kPBufs] P written (and O rescaled)
    uint64_t* pv_done = p_full + kPBufs;          // [kPBufs] O^T has the step (P and the V operand read)
    uint64_t* q_ready = pv_done + kPBufs;         // [2] query rows there
    uint64_t* q_free = q_ready + 2;               // [2] the run's S^T are formed, and what was found of it no longer wanted
    uint64_t* o_free = q_free + 2;                // O^T read by the epilogue
    uint64_t* o_done = o_free + 1;                // O^T has the run's last step
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(o_done + 1);
    static_assert((3 * kStages + 8 + 2 * kSBufs + 2 * kPBufs) * 8 + 4 <= 320, "barrier area");
    float* nm_s = reinterpret_cast<float*>(smem + kOffNm);
    float* move_s = reinterpret_cast<float*>(smem + kOffMove);
    float* red_s = reinterpret_cast<float*>(smem + kOffRed);
    int32_t* par_s = reinterpret_cast<int32_t*>(smem + kOffPar);
    uint64_t* anc_s = reinterpret_cast<uint64_t*>(smem + kOffAnc);
    int* row_s = reinterpret_cast<int*>(smem + kOffRow);
    uint64_t* inf_s = reinterpret_cast<uint64_t*>(smem + kOffInf);
    int* vexp_s = reinterpret_cast<int*>(smem + kOffVExp);
    auto scales = [](int it) { return reinterpret_cast<float*>(smem + kOffScl + it % kSclSlots * kSclBytes); };
    auto stage = [](int it) { return smem + kOffRing + it % kStages * kStageBytes; };
    auto stage_use = [](int it) { return static_cast<uint32_t>(it / kStages) & 1u; };

    volatile int* fail_s = reinterpret_cast<volatile int*>(smem + kOffFail);
    volatile int* late = fail_s + 7;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        volatile int* f = reinterpret_cast<volatile int*>(smem + kOffFail);
        f[kFailed] = f[kNoSums] = f[7] = f[kNoF16] = f[kFailedAgain] = 0;
        auto init = [](uint64_t* b, int n, int count) {
#pragma unroll 1
            for (int i = 0; i < n; ++i) mbar_init(b + i, count);
        };
        init(ring_full, kStages, 2);
        init(ring_empty, kStages, kConvWarps + 1);
        init(ring_go, kStages, 1);
        init(v_full, 2, kConvWarps);
        init(s_full, kSBufs, 1);
        init(s_empty, kSBufs, kSoftWarps);
        init(p_full, kPBufs, kSoftWarps);
        init(pv_done, kPBufs, 1);
        init(q_ready, 2, kConvWarps);
        init(q_free, 2, 1 + kSoftWarps);
        init(o_free, 1, kSoftWarps);
        init(o_done, 1, 1);
        fence_mbar_init();
    }
    if (warp == kPvWarp) tmem_alloc(tmem_s, kTmemCols);
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
    Walk walk;
    const int rank = kCluster ? blockIdx.x % wk.cluster : 0;
    if (!early) pdl_wait();
    if constexpr (kCluster) walk.start_unit(a, wk, blockIdx.x / wk.cluster, rank);
    else walk.start(a, wk, blockIdx.x, gridDim.x);
    if (threadIdx.x == 0) walk.save(fail_s + 1);
    if (kCluster && warp >= kConvWarp && warp <= kTmaWarp) {
        // what does not hang on the lengths is sent for with them: the page table's row, the query
        // rows, the block
        const int u = blockIdx.x / wk.cluster, b = u / wk.U, ub = u - b * wk.U, g = ub / wk.row_tiles;
        auto near = [](const void* at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); };
        const int x = threadIdx.x - 32 * kConvWarp;
        if (warp == kTmaWarp) {
            if (32 * lane < a.max_pages) near(a.pages + static_cast<size_t>(b) * a.max_pages + 32 * lane);
        } else if (!early) {
            const int gr = (ub - g * wk.row_tiles) * wk.tile_rows + (x >> 1), j = gr * wk.inv_g >> 16;
            if (j < a.R) near(a.q + (static_cast<size_t>(b * a.R + j) * a.Hq + g * a.G + gr - j * a.G) * kQ8D + 64 * (x & 1));
            if (x < 2 * a.R) {
                const size_t at = ((static_cast<size_t>(b) * a.Hkv + g) * a.R) * kQ8D + 64 * x;
                near(a.k_blk + at);
                near(a.v_blk + at);
            }
        }
    }
    // Each role does the CTA's runs once.  Those of them that failed (found while they are done, looked
    // at after all have finished) are done a second time, with references that the first pass's sums
    // give; those to which they give none, or V's scales no f16, or which fail again, `wide`.
    int run = -1;               // the current one
    uint32_t todo = ~0u;        // (bit r) run r is to be done; bit 31: those from there on
    bool by_sums = false;       // the second pass
    auto next_run = [&]() {
        do {
            if (!walk.next(a, wk)) return false;
            run = min(run + 1, 31);
        } while ((todo >> run & 1u) == 0u);
        return true;
    };
    auto note_run = [&](int word) { atomicOr(reinterpret_cast<int*>(smem + kOffFail) + word, 1 << run); };
    // a warp's wait; its lanes go on together (what follows is warp-collective)
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        bar_wait(bar, parity, late);
        __syncwarp();
    };
    auto restart = [&]() {
        // (bulk copies are not ordered among themselves: the failed run's partial has to have arrived
        // before the next one is sent to its place)
        if (threadIdx.x == 0) bulk_wait();
        __syncwarp();
        walk.load(a, fail_s + 1);
        run = -1;
    };
    // (The last pass has code of its own, so that the others' is short.)
    auto passes = [&](auto&& runs) {
        uint32_t last = 0u;
        while (true) {
            runs(std::false_type{});
            __syncwarp();
            named_barrier(2, kThreads);
            if (by_sums) {
                last |= static_cast<uint32_t>(fail_s[kFailedAgain]);
                break;
            }
            const uint32_t failed = fail_s[kFailed], no_sums = fail_s[kNoSums], no_f16 = fail_s[kNoF16];
            todo = failed & ~(no_sums | no_f16) & ((1u << kKept) - 1u);
            last = (failed | no_f16) & ~todo;
            if (todo == 0u) break;
            by_sums = true;
            restart();
        }
        if (last == 0u) return;
        todo = last;
        by_sums = false;
        restart();
        runs(std::true_type{});
    };

    // The rows of Q of a run, by half-warps: rows hw, hw + 64 / kN .. of the tile (of its kLive).
    auto load_q = [&](auto& x, const Walk& of, int hw) {
        constexpr int kN = sizeof(x.v) / 16;
        const int g = of.cur_unit / wk.row_tiles, row0 = of.cur_unit % wk.row_tiles * wk.tile_rows;
        const int nrows = min(wk.tile_rows, a.R * a.G - row0);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int r = hw + kLive / kN * i, gr = row0 + r, j = gr * wk.inv_g >> 16;
            x.v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < nrows)
                x.v[i] = __ldg(reinterpret_cast<const uint4*>(
                                   a.q + (static_cast<size_t>(of.cur_b * a.R + j) * a.Hq + g * a.G + gr - j * a.G) * kQ8D) +
                               (lane & 15));
        }
    };
    auto split_q = [&](const auto& x, int seg, int hw) {
        constexpr int kN = sizeof(x.v) / 16, kAtOnce = kN < 4 ? kN : 4;   // (side by side: a row is a chain of some 300 cycles)
        float* unit = reinterpret_cast<float*>(smem + kOffUnit) + (seg & 1) * kRows;
        uint32_t most[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) most[i] = row_most(x.v[i]);
#pragma unroll 1
        for (int i0 = 0; i0 < kN; i0 += kAtOnce) {
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                uint4 y = x.v[i];
                uint32_t m = most[i];
                if (kN > kAtOnce && i0 > 0) y = x.v[kN - kAtOnce + i], m = most[kN - kAtOnce + i];
                const bool bad = m >= 0x7f80u;
                const int e = q8_exponent(__uint_as_float(bad ? 0u : m << 16)), r = hw + kLive / kN * (i0 + i);
                split_row(y, bad, e, kStacked ? 2 * r - (r & 15) : r, smem + kOffQ + (seg & 1) * kQBytes,
                          kStacked ? 16 * 128 : kQBytes / 2);
                if ((lane & 15) == 0) unit[r] = q8_pow2(e);
            }
        }
    };

    // Every step, of the context or a block, has a ring stage: step `it` stage it %
    // kStages in its it / kStages-th use.
    if (warp == kTmaWarp || warp == kTmaWarp + 1) {
        // ---------------- page copies ----------------
        const bool is_v = warp > kTmaWarp;
        const uint8_t* pool = is_v ? a.v_pool : a.k_pool;
        uint64_t once;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        int it = 0;
        passes([&](auto wide) {
            while (next_run()) {
                const int g = walk.cur_unit / wk.row_tiles;
                const int32_t* tab = a.pages + static_cast<size_t>(walk.cur_b) * a.max_pages;
                const int np = walk.p1 - walk.p0;
                if (lane == 0 && walk.bad_len) raise_error(a.err, SV_DEVERR_LENGTH);
                // lane l holds page p0 + 32 k + l, 32 table entries at once, and its scales (a copy of
                // their 16 bytes would take as long to issue as one of 8 KB)
                int pg = 0, i = walk.block ? -2 : 0;
                uint4 f = make_uint4(0u, 0u, 0u, 0u);
                float least = 0.f;   // (V, first pass) scales from here on are held by f16
#pragma unroll 1
                for (; i < np; i += 2, ++it) {
                    if ((i & 31) == 0) {
                        pg = -1;
                        if (i + lane < np) {
                            pg = __ldg(tab + walk.p0 + i + lane);
                            if (pg < 0 || pg >= a.num_pages) {
                                raise_error(a.err, SV_DEVERR_PAGE);
                                pg = -1;
                            }
                        }
                        f = make_uint4(0u, 0u, 0u, 0u);
                        if (pg >= 0)
                            f = __ldg(reinterpret_cast<const uint4*>(pool + (static_cast<size_t>(pg) * a.Hkv + g) * kQ8Bytes + kQ8Codes));
                        __syncwarp();
                    }
                    const int s = it % kStages;
                    const int pa = __shfl_sync(0xffffffffu, pg, i & 31), pb = __shfl_sync(0xffffffffu, pg, (i + 1) & 31);
                    // (once the ring is full this warp waits for those that wait for the preceding kernel, and a
                    // wait's limit must not count that kernel's time)
                    if (early && it == kStages) pdl_wait();
                    wait(&ring_empty[s], stage_use(it) ^ 1u);
                    if (i < 0) {   // the stage of the block's K, whose writers do not follow the others' use of it
                        if (lane == 0 && !is_v) mbar_arrive(&ring_go[s]);
                        __syncwarp();
                        continue;
                    }
                    uint8_t* st = stage(it) + (is_v ? kTileBytes : 0);
                    const int bytes = (pa >= 0 ? kQ8Codes : 0) + (pb >= 0 ? kQ8Codes : 0);
                    if (lane == 0) {
                        mbar_expect_tx(&ring_full[s], bytes);
                        if (pa >= 0) bulk_g2s_once(st, pool + (static_cast<size_t>(pa) * a.Hkv + g) * kQ8Bytes, kQ8Codes, &ring_full[s], once);
                        if (pb >= 0)
                            bulk_g2s_once(st + kQ8Codes, pool + (static_cast<size_t>(pb) * a.Hkv + g) * kQ8Bytes, kQ8Codes, &ring_full[s], once);
                    }
                    if (bytes < 2 * kQ8Codes) {   // a page outside the pool reads as zeros
#pragma unroll 1
                        for (int p = 0; p < 2; ++p) {
                            if ((p == 0 ? pa : pb) >= 0 || i + p >= np) continue;
#pragma unroll 1
                            for (int x = lane; x < kQ8Codes / 16; x += 32)
                                reinterpret_cast<uint4*>(st + p * kQ8Codes)[x] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                    if ((lane ^ (i & 31)) < 2)   // lanes i and i + 1 (i is even)
                        reinterpret_cast<uint4*>(scales(it))[(is_v ? 2 : 0) + (lane & 1)] = f;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ring_full[s]);
                    __syncwarp();
                    if (is_v && !wide && !by_sums && (i & 31) == 0) {
                        const uint32_t w[4] = {f.x, f.y, f.z, f.w};
                        const int left = pg < 0 ? 0 : walk.cur_t - (walk.p0 + i + lane) * kQ8Page;
                        if (i == 0) {   // the largest of the first two pages, as the unit is found
                            uint32_t top = 0u;
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (lane < 2 && left > kQ8Run * r) top = max(top, w[r]);
                            least = q8_pow2(max(q8_stored_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, top))) - kVDown, kQ8MinExp));
                        }
                        bool low = false;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            low |= left > kQ8Run * r && __uint_as_float(w[r]) < least && __uint_as_float(w[r]) > q8_pow2(kQ8MinExp);
                        if (low) note_run(kNoF16);
                    }
                }
            }
        });
    } else if (warp == kQkWarp) {
        // ---------------- S^T = K Q^T ----------------
        if (early) pdl_wait();   // (as all that it waits for do)
        constexpr uint32_t id_s = idesc_e4m3_f32(128, kStacked ? 2 * kLive : kLive);
        int it = 0, seg = 0;
        Turn sb;
        static_assert(kSBufs == kPBufs, "one turn for both");
        passes([&](auto wide) {
            while (next_run()) {
                const int n = walk.ctx_steps() + (walk.block ? 1 : 0);
                if (elect_one()) {
                    const uint64_t qd = smem_desc_sw128(smem_u32(smem + kOffQ + (seg & 1) * kQBytes), 16, 1024);
                    bar_wait(&q_ready[seg & 1], (seg >> 1) & 1, late);
#pragma unroll 1
                    for (int st = 0; st < n; ++st) {
                        const int i = it + st, s = i % kStages;
                        bar_wait(&ring_full[s], stage_use(i), late);
                        bar_wait(&s_empty[sb.x], sb.parity ^ 1u, late);
                        // (and for the buffer that these scores' P will take: P V of kPBufs steps before)
                        bar_wait(&pv_done[sb.x], sb.parity ^ 1u, late);
                        tc_fence_after();
                        const uint64_t kd = smem_desc_sw128(smem_u32(stage(i)), 16, 1024);
                        // K by either part of Q, and the remainders of a block's K
                        const int parts = (walk.block && st == 0 ? 2 : 1) * (kStacked ? 1 : 2);
#pragma unroll 1
                        for (int p = 0; p < parts; ++p) {
                            const uint64_t kp = kd + (kStacked ? p : p >> 1) * (kTileBytes >> 4);
                            const uint64_t qp = qd + (kStacked ? 0 : p & 1) * (kQBytes / 2 >> 4);
#pragma unroll
                            for (int kc = 0; kc < kQ8D / 32; ++kc)
                                tc_mma_e4m3(tS(sb.x), kp + kc * 2, qp + kc * 2, id_s, (p > 0 || kc > 0) ? 1u : 0u);
                        }
                        tc_commit(&s_full[sb.x]);
                        tc_commit(&ring_empty[s]);
                        sb.next(kSBufs);
                    }
                    tc_commit(&q_free[seg & 1]);
                }
                __syncwarp();
                sb.x = __shfl_sync(0xffffffffu, sb.x, 0), sb.parity = __shfl_sync(0xffffffffu, sb.parity, 0);
                it += n;
                ++seg;
            }
        });
    } else if (warp == kPvWarp) {
        // ---------------- O^T += V^T P^T ----------------
        if (early) pdl_wait();
        constexpr uint32_t id_o = idesc_f16_f32_bmn(128, kLive), id_two = idesc_bf16_f32(128, kLive, false, true);
        int it = 0, seg = 0;
        Turn pb;
        passes([&](auto wide) {
            while (next_run()) {
                const int n = walk.ctx_steps() + (walk.block ? 1 : 0);
                if (elect_one()) {
                    bar_wait(o_free, (seg & 1) ^ 1, late);
#pragma unroll 1
                    for (int st = 0; st < n; ++st) {
                        const int i = it + st, x = i & 1;
                        const bool two = (walk.block && st == 0) || wide;   // bf16, P in two parts
                        bar_wait(&v_full[x], (i >> 1) & 1, late);
                        bar_wait(&p_full[pb.x], pb.parity, late);
                        tc_fence_after();
                        uint64_t pd = smem_desc_sw128(smem_u32(smem + kOffP + pb.x * kPBytes), 16, 1024);
                        uint32_t more = st > 0 ? 1u : 0u;
#pragma unroll 1
                        for (int p = two ? 0 : 1; p < 2; ++p) {
#pragma unroll
                            for (int kc = 0; kc < kStepKeys / 16; ++kc) {
                                tc_mma_ts(tO, tV(x) + kc * 8, pd + kc * (2048 >> 4), two ? id_two : id_o, more);
                                more = 1u;
                            }
                            pd = smem_desc_sw128(smem_u32(stage(i)), 16, 1024);
                        }
                        if (two) tc_commit(&ring_empty[i % kStages]);
                        tc_commit(&pv_done[pb.x]);
                        pb.next(kPBufs);
                    }
                    tc_commit(o_done);
                }
                __syncwarp();
                pb.x = __shfl_sync(0xffffffffu, pb.x, 0), pb.parity = __shfl_sync(0xffffffffu, pb.parity, 0);
                it += n;
                ++seg;
            }
        });
    } else if (warp >= kConvWarp) {
        // ---------------- to e4m3 pairs and to f16 ----------------
        if (early) pdl_wait();
        const int cw = warp - kConvWarp, hw = 2 * cw + (lane >> 4), ch = lane & 15;
        const int l = q4 * 32 + lane;        // V: the TMEM lane, a dim
        int it = 0, seg = 0;
        Turn pb;                             // of step it - 2
        uint32_t gone = 0;                   // (bit s) parity of the next block in stage s
        auto conv_sync = []() {
            __syncwarp();
            named_barrier(3, 32 * kConvWarps);
        };
        // the V operand of this step is free: P V of two steps before is done
        auto v_free = [&]() {
            if (it >= 2) {
                wait(&pv_done[pb.x], pb.parity);
                pb.next(kPBufs);
            }
            tc_fence_after();
        };
        auto v_done = [&](bool free) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&v_full[it & 1]);
                if (free) mbar_arrive(&ring_empty[it % kStages]);
            }
            ++it;
        };
        passes([&](auto wide) {
            while (next_run()) {
                const int g = walk.cur_unit / wk.row_tiles;
                const size_t blk0 = (static_cast<size_t>(walk.cur_b) * a.Hkv + g) * a.R * kQ8D;
                // half-warps take the query rows, and the block's rows of K
                auto k_row = [&](int r) {
                    return walk.block && r < a.R ? __ldg(reinterpret_cast<const uint4*>(a.k_blk + blk0 + r * kQ8D) + ch)
                                                 : make_uint4(0u, 0u, 0u, 0u);
                };
                uint4 ahead[2] = {k_row(hw), k_row(hw + 8)};
                const int s = it % kStages;
                // (a cluster's first run, mostly its only one, leaves them to the softmax warps, who have nothing
                // else to do yet: 16 sequences 34.6 -> 34.0 us, a tree 24.8 -> 24.0, batch 1 10.0 -> 9.7.  Where
                // more runs follow, this code is better run, and fetched, before memory is busy: 64 single
                // tokens 43.4 us, 57 with the softmax warps' help)
                if (!kCluster || seg > 0) {
                    Rows<kLive / 8> rows;
                    load_q(rows, walk, hw);
                    wait(&q_free[seg & 1], ((seg >> 1) & 1) ^ 1);
                    split_q(rows, seg, hw);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&q_ready[seg & 1]);
                }
                if (walk.block) {   // the block's K, into the stage that is kept for it
                    wait(&ring_go[s], gone >> s & 1u);
                    gone ^= 1u << s;
#pragma unroll 1
                    for (int r0 = hw; r0 - hw < a.R; r0 += 16) {
                        const uint4 y[2] = {ahead[0], ahead[1]};
                        ahead[0] = k_row(r0 + 16), ahead[1] = k_row(r0 + 24);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t m = row_most(y[i]);
                            const bool bad = m >= 0x7f80u;
                            const int e = q8_exponent(__uint_as_float(bad ? 0u : m << 16));
                            split_row(y[i], bad, e, r0 + 8 * i, stage(it), kTileBytes);
                            if (ch == 0) scales(it)[r0 + 8 * i] = q8_pow2(e);
                        }
                    }
                    fence_proxy_async_smem();
                    conv_sync();
                    if (warp < kConvWarp + 2 && lane == 0) mbar_arrive(&ring_full[s]);
                }
                // V is in units of 2^ev: of the largest scale of the first pages (their live runs) with
                // kVUp powers of two to spare; in the last pass of 1.  Every warp finds it by itself.
                int ev = 0;
                if (walk.ctx_steps() > 0 && !wide) {
                    const int first = it + (walk.block ? 1 : 0);
                    uint32_t top = 0u;
                    wait(&ring_full[first % kStages], stage_use(first));
                    const int left = walk.cur_t - walk.p0 * kQ8Page - kQ8Run * lane;
                    if (lane < 8 && left > 0 && (lane < 4 || walk.p0 + 1 < walk.p1)) top = reinterpret_cast<const uint32_t*>(scales(first))[8 + lane];
                    ev = q8_stored_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, top))) + kVUp;
                }
                if (cw == 0 && lane == 0) vexp_s[seg % 3] = ev;
                const float to = q8_pow2(-ev);
                if (walk.block) {
                    if (ev > kMostUnit) note_run(kNoF16);
                    // V stays bf16: drafts that no row sees may be of any size.  Rows past the last are
                    // zeros.  What is not finite would reach the rows that do not see it (0 times it is
                    // NaN): it stays out of the product, and the epilogue adds it where it is seen
                    v_free();
                    const uint16_t* vsrc = a.v_blk + blk0 + l;
                    uint64_t inf0 = 0ull, inf1 = 0ull;
#pragma unroll 1
                    for (int k0 = 0; k0 < kStepKeys; k0 += 16) {
                        uint32_t r[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                        if (k0 < a.R) {
                            uint32_t w[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) w[k] = k0 + k < a.R ? __ldg(vsrc + (k0 + k) * kQ8D) : 0u;
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                if ((w[k] & 0x7f80u) == 0x7f80u) (k0 < 64 ? inf0 : inf1) |= 1ull << ((k0 & 63) + k), w[k] = 0u;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                r[k] = pack_bf16x2(__uint_as_float(w[2 * k] << 16) * to, __uint_as_float(w[2 * k + 1] << 16) * to);
                        }
                        tmem_st8(tV(it & 1) + lane_off + (k0 >> 1), r);
                    }
                    inf_s[(seg % 3 * kQ8D + l) * 2] = inf0;
                    inf_s[(seg % 3 * kQ8D + l) * 2 + 1] = inf1;
                    // (the stage's place is kept for P's second part: one arrival comes from its product)
                    v_done(cw != 0);
                }
#pragma unroll 1
                for (int st = 0; st < walk.ctx_steps(); ++st) {
                    uint8_t* v = stage(it) + kTileBytes;
                    wait(&ring_full[it % kStages], stage_use(it));
                    // keys of the step that exist: what the others' codes hold is not looked at (0 * a
                    // V that is not finite would be NaN)
                    const int have = min(walk.cur_t - (walk.p0 + 2 * st) * kQ8Page, (walk.p1 - walk.p0 - 2 * st) * kQ8Page);
                    if (have < kStepKeys) {
#pragma unroll 1
                        for (int o = have >> 3; o < kStepKeys / 8; ++o) {   // (this thread's dim alone)
                            uint64_t* w = reinterpret_cast<uint64_t*>(v + q8_v_off(o, l));
                            const int left = have - 8 * o;
                            *w = left <= 0 ? 0ull : *w & ((1ull << 8 * left) - 1ull);
                        }
                        // (the next copy into the stage comes by the other proxy: these stores before it)
                        fence_proxy_async_smem();
                    }
                    const float2* f2 = reinterpret_cast<const float2*>(scales(it) + 8);
                    if (wide) {
                        v_free();
                        wide_v(v, scales(it) + 8, have, l, tV(it & 1) + lane_off);
                        v_done(cw != 0);   // (P's second part goes to the stage, as a block's)
                        continue;
                    }
                    v_free();
#pragma unroll
                    for (int h = 0; h < 4; ++h) {   // 32 keys: two runs
                        const float2 f = f2[h];
                        const uint32_t m[2] = {have > 32 * h ? pack_f16x2(f.x * to, f.x * to) : 0u,
                                               have > 32 * h + 16 ? pack_f16x2(f.y * to, f.y * to) : 0u};
                        uint32_t r[16];
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            const uint2 w = *reinterpret_cast<const uint2*>(v + q8_v_off(4 * h + o, l));
                            r[4 * o] = mul_f16x2(f16x2_of_codes(w.x), m[o >> 1]);
                            r[4 * o + 1] = mul_f16x2(f16x2_of_codes(w.x >> 16), m[o >> 1]);
                            r[4 * o + 2] = mul_f16x2(f16x2_of_codes(w.y), m[o >> 1]);
                            r[4 * o + 3] = mul_f16x2(f16x2_of_codes(w.y >> 16), m[o >> 1]);
                        }
                        tmem_st16(tV(it & 1) + lane_off + 16 * h, r);
                    }
                    v_done(true);
                }
                ++seg;
            }
        });
    } else {
        // ---------------- softmax, epilogue ----------------
        // (the barrier counts whole warps: they arrive converged)
        auto soft_sync = []() {
            __syncwarp();
            named_barrier(1, 32 * kSoftWarps);
        };
        auto soft_any = [](bool x) {   // the same, and whether x holds in any of the threads
            uint32_t r;
            __syncwarp();
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(r)
                : "r"(x ? 1u : 0u), "n"(32 * kSoftWarps)
                : "memory");
            return r != 0u;
        };
        if (early) pdl_wait();
        // A cluster's successor may start now.  (Not before the wait: the successor may
        // read a cache that only this kernel's predecessor must not be writing.)
        if constexpr (kCluster) pdl_launch_dependents();
        const int hh = warp >> 2;              // rows hh * kRT .. of the tile (of its halves)
        const int l = q4 * 32 + lane;          // key of the step; dim in the epilogue
        const int tid = threadIdx.x;
        const float sc = a.scale_log2;
        const int rows = a.R * a.G;
        int it = 0, seg = 0;
        Turn sb;
        // The rows' means over the run, each thread's dim: store(row of the tile, mean), which cannot
        // pass V's largest.  True where something was not finite.
        auto means = [&](int b, int g, int row0, bool tree, auto&& store) {
            const float v_unit = q8_pow2(vexp_s[seg % 3]);
            uint64_t inf0 = 0ull, inf1 = 0ull;
            if (walk.block) inf0 = inf_s[(seg % 3 * kQ8D + l) * 2], inf1 = inf_s[(seg % 3 * kQ8D + l) * 2 + 1];
            bool bad = false;
#pragma unroll 1
            for (int c0 = 0; c0 < kRT; c0 += 8) {
                uint32_t o[8];
                tmem_ld8_sync(tO + lane_off + hh * kRT + c0, o);
                float mean[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = __uint_as_float(o[e]) * move_s[hh * kRT + c0 + e];
                    bad |= !(fabsf(x) < INFINITY);
                    mean[e] = x * v_unit;
                }
                if ((inf0 | inf1) != 0ull) {   // (rare) V that is not finite and that the row sees
#pragma unroll 1
                    for (int e = 0; e < 8; ++e) {
                        const int j = (row0 + hh * kRT + c0 + e) * wk.inv_g >> 16;   // (any row past the tile's last)
                        if (j >= a.R) continue;
                        uint64_t m0 = inf0, m1 = inf1;
                        if (tree) m0 &= anc_s[2 * j], m1 &= anc_s[2 * j + 1];
                        else m0 &= ~0ull >> (63 - min(j, 63)), m1 &= j < 64 ? 0ull : ~0ull >> (127 - j);
                        float add = 0.f;
#pragma unroll 1
                        for (; m0 | m1; (m0 ? m0 : m1) &= (m0 ? m0 : m1) - 1ull) {
                            const int key = m0 ? __ffsll(m0) - 1 : 63 + __ffsll(m1);
                            add += __uint_as_float(static_cast<uint32_t>(__ldg(
                                a.v_blk + ((static_cast<size_t>(b) * a.Hkv + g) * a.R + key) * kQ8D + l)) << 16);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i == e) mean[i] += add;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) store(hh * kRT + c0 + e, mean[e]);
            }
            return bad;
        };
        float* kept_s = reinterpret_cast<float*>(smem + kOffKept);
        passes([&](auto wide) {
            while (next_run()) {
                // done again: with the references that the sums gave, or, in the last pass, moving ones
                const bool kept = run < kKept && (wide ? (fail_s[kNoSums] >> run & 1) == 0 : by_sums), safe = wide && !kept;
                const int b = walk.cur_b, g = walk.cur_unit / wk.row_tiles, rt = walk.cur_unit % wk.row_tiles;
                const int row0 = rt * wk.tile_rows, nrows = min(wk.tile_rows, rows - row0);
                const bool first = kCluster && seg == 0;
                Rows<kLive / 16> qrows;
                if (first) load_q(qrows, walk, 2 * warp + (lane >> 4));
                // (a partial of the run before may still be on its way out of P's place)
                if (tid == 0) bulk_wait_read();
                if (tid < kRows) {
                    const int gr = row0 + tid, j = gr * wk.inv_g >> 16;
                    row_s[tid] = tid < nrows ? (b * a.R + j) * a.Hq + g * a.G + gr - j * a.G : -1;
                    nm_s[tid] = kept ? kept_s[run * kRows + tid] + (wide ? kUpWide : kUpSum) : 0.f;
                }
                const bool tree = walk.block && a.parent != nullptr;
                if (tree && tid < a.R) par_s[tid] = __ldg(a.parent + static_cast<size_t>(b) * a.R + tid);
                if (first) {
                    split_q(qrows, 0, 2 * warp + (lane >> 4));
                    fence_proxy_async_smem();
                }
                soft_sync();   // row_s, nm_s, par_s
                if (first && warp < kConvWarps && lane == 0) mbar_arrive(&q_ready[0]);
                if (tree) {
                    if (tid < a.R) {
                        uint64_t m0 = 0, m1 = 0;
                        int i = tid;
                        bool bad = false;
#pragma unroll 1
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
                // (the rows' units; all else that the convert warps write comes by way of S^T)
                const float* unit_s = reinterpret_cast<const float*>(smem + kOffUnit) + (seg & 1) * kRows;
                wait(&q_ready[seg & 1], (seg >> 1) & 1);
                float2 sums[kRT / 2];
#pragma unroll
                for (int i = 0; i < kRT / 2; ++i) sums[i] = make_float2(0.f, 0.f);
                bool found = false;   // (safe) row tid has a reference
                const int lead = walk.block ? 1 : 0, n = walk.ctx_steps() + lead;
                // the rows that see this thread's key (bit e: row hh * kRT + e): of the context, keys
                // before the length (the second page of a step may be missing); block row l is seen
                // from query rows l G on, or by the tree rows on whose path it lies
                auto seen_by = [&](int st) {
                    if (st >= lead)
                        return (walk.p0 + 2 * (st - lead)) * kQ8Page + l < min(walk.cur_t, walk.p1 * kQ8Page) ? ~0u : 0u;
                    if (!tree) {
                        const int lo = l < a.R ? l * a.G - row0 - hh * kRT : kRT;
                        return lo >= kRT ? 0u : lo > 0 ? ~0u << lo : ~0u;
                    }
                    // block row by block row: its G query rows see the same keys
                    uint32_t seen = 0u;
                    const int r0 = row0 + hh * kRT, r1 = min(r0 + kRT, rows);
                    int j = r0 * wk.inv_g >> 16;
#pragma unroll 1
                    for (int r = j * a.G - r0; l < a.R && r + r0 < r1; ++j, r += a.G) {
                        if ((anc_s[2 * j + (l >> 6)] >> (l & 63) & 1ull) == 0ull) continue;
                        const uint32_t run = (1u << a.G) - 1u;   // (G <= 16)
                        seen |= r >= 0 ? run << r : run >> -r;
                    }
                    return seen;
                };
                // the key's scale: of its run, or of the block's row
                auto key_scale = [&](int st) { return sc * scales(it)[st < lead ? l : l >> 4]; };
                auto scores = [&](uint32_t(&s)[kRT]) {
                    if constexpr (!kStacked) {
                        tmem_ld32_sync(tS(sb.x) + lane_off + hh * kRT, s);
                    } else {
                        uint32_t z[32];
                        tmem_ld32_sync(tS(sb.x) + lane_off + hh * 32, z);
#pragma unroll
                        for (int i = 0; i < kRT / 2; ++i) {
                            const float2 y = __fadd2_rn(make_float2(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1])),
                                                        make_float2(__uint_as_float(z[16 + 2 * i]), __uint_as_float(z[17 + 2 * i])));
                            s[2 * i] = __float_as_uint(y.x), s[2 * i + 1] = __float_as_uint(y.y);
                        }
                    }
                };
                auto scores8 = [&](int c0, uint32_t(&s)[8]) {
                    tmem_ld8_sync(tS(sb.x) + lane_off + hh * 32 + c0, s);
                    if constexpr (kStacked) {
                        uint32_t z[8];
                        tmem_ld8_sync(tS(sb.x) + lane_off + hh * 32 + 16 + c0, z);
#pragma unroll
                        for (int i = 0; i < 8; ++i) s[i] = __float_as_uint(__fadd_rn(__uint_as_float(s[i]), __uint_as_float(z[i])));
                    }
                };
                auto s_wait = [&]() {
                    wait(&s_full[sb.x], sb.parity);
                    tc_fence_after();
                };
                // The references (until now none, -m + kUp = 0): the maxima over the run's first 32 keys
                // where those are finite, or, with `safe`, over all so far.  A score is rounded before
                // anything is done with it, here and in the steps with masks, so that with `safe` the
                // largest gives kUp however large it is (the scales first: codes times one of them can
                // pass fp32's largest).
                auto references = [&](int st, uint32_t seen) {
                    const float ks = key_scale(st);
                    if (wide || q4 == 0) {
                        float most = 0.f;   // lane e's: row e's
#pragma unroll (kRT == 16 ? 2 : 1)
                        for (int c0 = 0; c0 < kRT; c0 += 8) {
                            uint32_t s[8];
                            scores8(c0, s);
                            const float4* un = reinterpret_cast<const float4*>(unit_s + hh * kRT + c0);
                            const float4 ua = un[0], ub = un[1];
                            const float u[8] = {ua.x, ua.y, ua.z, ua.w, ub.x, ub.y, ub.z, ub.w};
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float z = __fmul_rn(__uint_as_float(s[i]), __fmul_rn(u[i], ks));
                                const float m = warp_max(seen >> (c0 + i) & 1u ? z : -INFINITY);
                                if (lane == c0 + i) most = m;
                            }
                        }
                        if (lane < kRT) {
                            if (wide) red_s[q4 * kRows + hh * kRT + lane] = most;
                            else if (fabsf(most) < INFINITY) nm_s[hh * kRT + lane] = kUp - most;
                        }
                    }
                    soft_sync();
                    if (!wide) return;
                    bool moved = false;
                    if (tid < kLive) {
                        // up where the maximum has risen by more than kSlack, or where no score was finite so
                        // far (P, the sum and O are 0 then) to wherever it is
                        const float m = fmaxf(fmaxf(red_s[tid], red_s[kRows + tid]), fmaxf(red_s[2 * kRows + tid], red_s[3 * kRows + tid]));
                        const float was = kUp - nm_s[tid];
                        float move = 1.0f;
                        if (m > -INFINITY && (!found || m > was + kSlack)) {
                            if (found) move = fast_exp2(was - m);
                            moved = found;
                            nm_s[tid] = kUp - m;
                            found = true;
                        }
                        move_s[tid] = move;
                    }
                    if (!soft_any(moved)) return;
#pragma unroll
                    for (int i = 0; i < kRT / 2; ++i)
                        sums[i] = __fmul2_rn(sums[i], reinterpret_cast<const float2*>(move_s + hh * kRT)[i]);
                    // O^T (lane = dim) once the step before is in it
                    wait(&pv_done[(it - 1) % kPBufs], ((it - 1) / kPBufs) & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < kRT; c0 += 8) {
                        uint32_t o[8];
                        tmem_ld8_sync(tO + lane_off + hh * kRT + c0, o);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * move_s[hh * kRT + c0 + e]);
                        tmem_st8(tO + lane_off + hh * kRT + c0, o);
                    }
                    tmem_st_wait();
                };
                auto step_done = [&]() {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[sb.x]);
                    sb.next(kSBufs);
                    ++it;
                };
                // a step that every row sees whole.  (A key's line of P takes eight rows in 16 bytes.)
                auto plain_step = [&](int st) {
                    s_wait();
                    const float ks = key_scale(st);
                    uint32_t s[kRT];
                    scores(s);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_empty[sb.x]);   // the scores are read
                    const float2 k2 = make_float2(ks, ks);
                    const float2* nm = reinterpret_cast<const float2*>(nm_s + hh * kRT);
                    const float2* un = reinterpret_cast<const float2*>(unit_s + hh * kRT);
                    uint8_t* prow = smem + kOffP + sb.x * kPBytes + l * 128;
#pragma unroll
                    for (int q = 0; q < kRT / 8; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 4 * q; i < 4 * q + 4; ++i) {
                            // exponents of two rows against their references
                            const float2 e = __ffma2_rn(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])),
                                                        __fmul2_rn(un[i], k2), nm[i]);
                            const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                            sums[i] = __fadd2_rn(sums[i], p);
                            w[i & 3] = pack_f16x2(p.x, p.y);
                        }
                        *reinterpret_cast<uint4*>(prow + (((hh * (kRT / 8) + q) ^ (l & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    step_done();
                };
                // any step, the block's among them, whose P is bf16 (range) in two parts (16 bits), the second
                // in the place of the step's K, which has been read; so is all P of the last pass.  Eight
                // rows at a time; the sums go round, so that the loop's code serves them all (unrolled, the
                // larger tile's spills).
                auto any_step = [&](int st) {
                    s_wait();
                    const bool two = st < lead || wide;
                    const uint32_t seen = seen_by(st);
                    if (safe || (st == 0 && !kept)) references(st, seen);
                    const float ks = key_scale(st);
                    uint8_t* prow = smem + kOffP + sb.x * kPBytes + l * 128;
                    uint8_t* rest = stage(it) + l * 128;
                    const bool none = !__any_sync(0xffffffffu, seen != 0u);
#pragma unroll (kRT == 16 ? 2 : 1)
                    for (int c0 = 0; c0 < kRT; c0 += 8) {
                        uint32_t w[4] = {0u, 0u, 0u, 0u}, v[4] = {0u, 0u, 0u, 0u};
                        float2 now[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) now[i] = sums[i];
                        if (!none) {
                            uint32_t s[8];
                            scores8(c0, s);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                // (one by one: the packed product and sum would be fused)
                                const float2 un = reinterpret_cast<const float2*>(unit_s + hh * kRT + c0)[i];
                                const float2 nm = reinterpret_cast<const float2*>(nm_s + hh * kRT + c0)[i];
                                const float ex = __fadd_rn(__fmul_rn(__uint_as_float(s[2 * i]), __fmul_rn(un.x, ks)), nm.x);
                                const float ey = __fadd_rn(__fmul_rn(__uint_as_float(s[2 * i + 1]), __fmul_rn(un.y, ks)), nm.y);
                                const float2 p = make_float2(seen >> (c0 + 2 * i) & 1u ? fast_exp2(ex) : 0.f,
                                                             seen >> (c0 + 2 * i + 1) & 1u ? fast_exp2(ey) : 0.f);
                                now[i] = __fadd2_rn(now[i], p);
                                if (two) {
                                    w[i] = pack_bf16x2(p.x, p.y);
                                    v[i] = pack_bf16x2(p.x - __uint_as_float(w[i] << 16), p.y - __uint_as_float(w[i] & 0xffff0000u));
                                } else {
                                    w[i] = pack_f16x2(p.x, p.y);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < kRT / 2 - 4; ++i) sums[i] = sums[i + 4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) sums[kRT / 2 - 4 + i] = now[i];
                        const int to = ((hh * (kRT / 8) + c0 / 8) ^ (l & 7)) << 4;
                        *reinterpret_cast<uint4*>(prow + to) = make_uint4(w[0], w[1], w[2], w[3]);
                        if (two) *reinterpret_cast<uint4*>(rest + to) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_empty[sb.x]);
                    step_done();
                };
                // whole context steps apart, so that they carry no masks
                const bool ragged = (walk.p1 - walk.p0) & 1 || walk.p1 * kQ8Page > walk.cur_t;
                const int nwhole = wide ? 0 : n - (ragged ? 1 : 0);
#pragma unroll 1
                for (int st = 0; st < n; ++st) {
                    if (st >= lead && st < nwhole) {
                        if (st == 0 && !kept) {
                            s_wait();
                            references(0, ~0u);
                        }
                        plain_step(st);
                    } else {
                        any_step(st);
                    }
                }
                // the rows' sums over the keys: lane e of a warp ends with its row e's
                // (halving the rows and the lanes that differ, step by step)
                float sum[kRT];
#pragma unroll
                for (int i = 0; i < kRT / 2; ++i) sum[2 * i] = sums[i].x, sum[2 * i + 1] = sums[i].y;
                fold_sums(sum);
#pragma unroll
                for (int o = kRT; o < 32; o <<= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
                if (lane < kRT) red_s[q4 * kRows + hh * kRT + lane] = sum[0];
                // Partials go by way of P's place, where a cluster's stay; so do the rows of a unit that
                // is whole, as bf16.
                float* rec = reinterpret_cast<float*>(smem + kOffP);
                const bool direct = kCluster ? wk.cluster == 1 : walk.whole;
                soft_sync();
                bool bad = false;
                float lsum = 0.f;
                if (tid < kLive) {
                    lsum = (red_s[tid] + red_s[kRows + tid]) + (red_s[2 * kRows + tid] + red_s[3 * kRows + tid]);
                    const float least = kLost * static_cast<float>(kStepKeys * n);
                    bad = !(lsum < kMostSum) || (lsum < least && tid < nrows);
                    if (!wide && !by_sums && run < kKept) {
                        if ((lsum >= kLeastSum && lsum < INFINITY) || tid >= nrows)
                            kept_s[run * kRows + tid] = nm_s[tid] - __log2f(fmaxf(lsum, kLeastSum));
                        else
                            note_run(kNoSums);
                    }
                    move_s[tid] = lsum != 0.f ? __fdividef(1.0f, lsum) : 0.f;
                }
                wait(o_done, seg & 1);
                // (only now has all of P been read)
                if (!direct && tid < kLive)
                    *reinterpret_cast<float2*>(rec + kRows * kQ8D + 2 * tid) = make_float2(-nm_s[tid], lsum);   // (kUp below the reference)
                tc_fence_after();
                soft_sync();
                bad |= means(b, g, row0, tree, [&](int r, float mean) {
                    if (direct) reinterpret_cast<uint16_t*>(rec)[r * kQ8D + l] = f32_bf16_bits(mean);
                    else rec[r * kQ8D + l] = mean;   // (rows past the tile's last too, never read)
                });
                if (bad && !wide) note_run(by_sums ? kFailedAgain : kFailed);
                tc_fence_before();
                if (!kCluster && !direct) fence_proxy_async_smem();
                soft_sync();   // red_s and nm_s read by everyone before the next run writes them; the rows are there
                if (lane == 0) {
                    mbar_arrive(o_free);
                    mbar_arrive(&q_free[seg & 1]);
                }
                if (direct) {
#pragma unroll 1
                    for (int r = warp; r < nrows; r += kSoftWarps)
                        reinterpret_cast<uint2*>(a.out + static_cast<size_t>(row_s[r]) * kQ8D)[lane] =
                            reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(rec) + r * kQ8D)[lane];
                    soft_sync();   // (P's place and row_s are free)
                } else if (!kCluster) {
                    // (a partial run that is not the CTA's first is its last)
                    if (tid == 0) bulk_s2g(ws + (static_cast<size_t>(blockIdx.x) * 2 + (run > 0 ? 1 : 0)) * kRecFloats, rec, kRecFloats * 4);
                }
                ++seg;
            }
        });
        if (tid == 0) bulk_wait();
        if constexpr (kCluster) {   // no page of the unit fell to this CTA
            if (seg == 0 && tid < kRows)
                *reinterpret_cast<float2*>(smem + kOffP + (kRows * kQ8D + 2 * tid) * 4) = make_float2(-INFINITY, 0.f);
        }
    }
    __syncwarp();
    if (kCluster && wk.cluster > 1) {
        cluster_sync_warp();   // every CTA's partial is there
        cg::cluster_group cluster = cg::this_cluster();
        const int u = blockIdx.x / wk.cluster, b = u / wk.U, ub = u - b * wk.U, g = ub / wk.row_tiles;
        const int row0 = (ub - g * wk.row_tiles) * wk.tile_rows, nrows = min(wk.tile_rows, a.R * a.G - row0);
        auto dst = [&](int r) {
            const int gr = row0 + r, j = gr * wk.inv_g >> 16;
            return a.out + (static_cast<size_t>(b * a.R + j) * a.Hq + g * a.G + gr - j * a.G) * kQ8D;
        };
        auto partial = [&](int i, int r, float2& ml, float4& o) {
            const float* rec = reinterpret_cast<const float*>(cluster.map_shared_rank(smem + kOffP, i));
            ml = *reinterpret_cast<const float2*>(rec + kRows * kQ8D + 2 * r);
            o = *(reinterpret_cast<const float4*>(rec + r * kQ8D) + lane);
        };
        const int step = wk.cluster * (kThreads / 32), r0 = rank + wk.cluster * warp;
        if (wk.cluster < 4) {   // a warp may have two rows: both on their way at once (16 sequences 35.4 -> 34.6 us)
            static_assert(2 * 2 * (kThreads / 32) >= kRows, "two rows of a warp");
            PartialRows<3> x, y;
            const bool two = r0 + step < nrows;
            if (r0 < nrows) x.load(wk.cluster, [&](int i, float2& ml, float4& o) { partial(i, r0, ml, o); });
            if (two) y.load(wk.cluster, [&](int i, float2& ml, float4& o) { partial(i, r0 + step, ml, o); });
            RowSum sum;
            if (r0 < nrows) x.add_to<true>(sum), store_row(sum, dst(r0));
            sum = RowSum();
            if (two) y.add_to<true>(sum), store_row(sum, dst(r0 + step));
        } else if (r0 < nrows) {
            auto get = [&](int i, float2& ml, float4& o) { partial(i, r0, ml, o); };
            join_partials<true>(wk.cluster, get, dst(r0));
        }
        __syncwarp();
        cluster_sync_warp();   // this CTA's partial has been read
    }
    if constexpr (!kCluster) pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == kPvWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
        if (*late != 0) {
            raise_error(a.err, SV_DEVERR_TIMEOUT);
            // copies may be on their way into this CTA's shared memory: some thousand times as long as one takes
            const uint64_t t0 = global_timer_ns();
            for (int i = 0; i < (1 << 20) && global_timer_ns() - t0 < 2000000ull; ++i) {}
        }
    }
}

// Joins the partial rows of the units that lie in several CTAs' runs: kWide warps a row.
// (One sequence of 100001 positions, whose two units lie in 77 runs each: 8 us less with
// 8 warps a row than with one.)  Which CTAs had a unit follows from the lengths, which the
// attention does not write and was past its own wait for: they are read before the wait here
// (the same 20.3 -> 19.5 us, 64 single tokens 46.4 -> 45.6).
template <int kWide>
__global__ void __launch_bounds__(kCombineThreads)
    combine_q8_kernel(CacheAttnArgs a, Work wk, const float* __restrict__ ws, int grid) {
    __shared__ float2 ml_s[kWide];
    __shared__ float4 o_s[kWide][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gr = blockIdx.x * (kCombineThreads / 32 / kWide) + warp / kWide, part = warp % kWide;
    const int b = blockIdx.y / a.Hkv, g = blockIdx.y % a.Hkv;
    const int rt = gr / wk.tile_rows, r = gr % wk.tile_rows;
    const int2 sums = work_sums(a, b);
    const int W = sums.x * wk.U, n = active_ctas(wk, W, grid);
    const int np = ctx_pages(ctx_len(a, b));
    const int w0 = sums.y * wk.U + (g * wk.row_tiles + rt) * (np + 1), w1 = w0 + np + 1;
    const int i0 = cta_of(W, w0, n), i1 = cta_of(W, w1 - 1, n);
    const bool later = static_cast<int64_t>(w0) * n > static_cast<int64_t>(W) * i0;   // w0 is past CTA i0's first page
    pdl_wait();
    pdl_launch_dependents();
    if (gr >= a.R * a.G) return;   // (a whole CTA where a row has one)
    if (i0 == i1) return;   // one CTA had the whole unit and wrote its rows
    auto get = [&](int k, float2& ml, float4& o) {
        // a unit that starts inside CTA i0's run is its second partial
        const int i = k * kWide + part;
        const float* rec = ws + (static_cast<size_t>(i0 + i) * 2 + (i == 0 && later ? 1 : 0)) * kRecFloats;
        ml = __ldcg(reinterpret_cast<const float2*>(rec + kRows * kQ8D + 2 * r));
        o = __ldcg(reinterpret_cast<const float4*>(rec + r * kQ8D) + lane);
    };
    const int count = i1 - i0 + 1;
    RowSum x = add_partials<true>((count - part + kWide - 1) / kWide, get);
    if constexpr (kWide > 1) {
        if (lane == 0) ml_s[part] = make_float2(x.m, x.l);
        o_s[part][lane] = x.o;
        __syncthreads();
        if (warp != 0) return;
        x = add_partials<false>(kWide, [&](int k, float2& ml, float4& o) { ml = ml_s[k], o = o_s[k][lane]; });
    }
    store_row(x, a.out + ((static_cast<size_t>(b) * a.R + gr / a.G) * a.Hq + g * a.G + gr % a.G) * kQ8D);
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

// How the work is split: a cluster of up to 8 CTAs for each unit, joined on chip, or all
// pages evenly over the SMs and partials joined by a second kernel, whichever is expected to
// take less time.  The terms, in ns, were fitted to some sixty shapes:
//   - a page takes a CTA 300, or, where CTAs that read at the same time fill HBM, 2.8 for each
//     of them; 2.3 and 2.55 where they are out of step (units in several waves, the even split);
//   - a CTA's start and end and a cluster's join take 6500, 11000 with tiles of more than 32 rows;
//   - the even split's, with the second kernel, 11500 and 17000, and a CTA that goes on to
//     another unit 5500 and 10000 more, beside steps of 250 and 375 a page.  A single sequence's
//     units are alike, and a multiple of their number of CTAs splits them without such CTAs:
//     9000 and 13500 (9 x 28 heads over 4, 4096 positions: 18.2 -> 14.4 us when that came in).
// Measured in us, the side that the rule takes first: 5 x 12 heads over 2 of 4096 positions,
// clusters 9.4, split 10.2; of 8192, split 10.1, clusters 11.6; of 16384, split 11.6, clusters
// 16.0; 9 x 28 over 4, 8192: split 14.9, clusters 15.4; four such: clusters 19.7, split 21.1;
// 16: clusters of two 34.5, split 40.5; 64 of 4096: one CTA a unit 64.5, split 75.8; 40: split 51.1,
// one a unit 61.4; 65 x 28 over 4, 8192: clusters 24.4, split 25.9; 32 single tokens of 2048: one
// a unit 17.6, split 23.5; 64 of 256: 16.8 and 22.8; 64 of 4096: split 53.2, one a unit 55.0.  The
// table's capacity decides, as the lengths are on the device.
void plan(Work& w, int B, int max_pages, int& grid) {
    const int64_t units = static_cast<int64_t>(B) * w.U, pages = units * (static_cast<int64_t>(max_pages) + 1);
    const int64_t sms = device_sm_count();
    const bool tall = w.tile_rows > 32;
    auto page_ns = [](int64_t ctas, int64_t ps) { return ctas * ps > 300000 ? ctas * ps / 1000 : int64_t(300); };
    const int64_t most = pages / kGrain;
    grid = static_cast<int>(most < 1 ? 1 : most < sms ? most : sms);
    w.cluster = 0;
    w.even = B == 1 ? w.U : 1;
    if (grid > w.even) grid -= grid % w.even;
    const int64_t each = (pages + grid - 1) / grid, stream = each * page_ns(grid, 2550);
    const int64_t steps = each * (tall ? 375 : 250) + (B == 1 ? 0 : units * (tall ? 10000 : 5500) / grid);
    int64_t best = (stream > steps ? stream : steps) + (B == 1 ? (tall ? 13500 : 9000) : (tall ? 17000 : 11500));
    auto cost = [&](int64_t n, int c, int64_t ps) { return (max_pages + c) / c * page_ns(n * c, ps) + (tall ? 11000 : 6500); };
    for (int c = 1; c <= kMaxCluster; ++c) {
        int64_t t;
        if (units <= (c == 1 ? sms : resident_clusters(c))) t = cost(units, c, 2800);
        else if (c == 1) t = units / sms * cost(sms, 1, 2300) + (units % sms ? cost(units % sms, 1, 2300) : 0);
        else continue;
        if (t >= best) continue;
        best = t;
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
    constexpr int kWarps = kCombineThreads / 32;
    if (grid > 2 * kWarps * a.B * w.U)
        return launch_pdl(combine_q8_kernel<kWarps>, dim3(a.R * a.G, a.B * a.Hkv), dim3(kCombineThreads), 0, st, a, w, part, grid);
    return launch_pdl(combine_q8_kernel<1>, dim3((a.R * a.G + kWarps - 1) / kWarps, a.B * a.Hkv), dim3(kCombineThreads), 0, st, a, w,
                      part, grid);
}

}  // namespace sv
