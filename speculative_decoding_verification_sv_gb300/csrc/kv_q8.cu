// kv_q8.cu -- writing and reading the 8-bit paged KV cache (format: kv_q8.cuh).
//
//   append  new rows of a layer, K rotated by position (as kv_append.cu), the bf16
//           rows that the bf16 cache would hold rounded to e4m3 on the way
//   commit  the accepted rows of a verify block, every layer (as kv_commit.cu)
//   gather  a window of positions read back as bf16 rows
//
// The unit of writing is a run, the sixteen aligned positions of one (sequence, head)
// that share a scale: one warp owns it, takes the largest magnitude of the new rows
// over its lanes, and where an earlier row's scale is too small for them holds the
// earlier codes anew.  V's words hold eight positions of a dim: what a partly filled
// octet held before is read back and merged.  No two warps of a launch share a run, and
// none waits for another.
//
// Measured, graph replays over inputs larger than L2: append of 8 prompts of 2048 rows (4
// heads; 34 MB read, 17 MB written, 7.4 us at copy rate) 16.1 us; of 4 chunks of 1000 rows 6.5,
// of one token in each of 64 sequences 4.8.  A run of K is 16 rows of angles beside 16
// rows of data, and both come from L2 or beyond before a code can leave: latency and, at
// 0.5 instructions a cycle, issue bound it, so warps hold eight rows' angles on their way
// (23.5 us with the read-back for the prompts; four 24.9, two 27.1, sixteen 26.3: fewer warps
// fit or registers spill) in CTAs of four warps, which leave room for 20 on an SM (three of
// eight 26.7, with spills).  With lanes of four dims side by side, whose rotation takes two
// shuffles and eight selects a row and loads every angle twice, the same took 32.2.
// Commit of 28 layers x 4 heads, 16 sequences of up to 9 rows: 13.7 us, of which the launch, len
// and the cluster's barriers are 2.9: three rounds of scattered rows and runs for each of 2048
// warps.  Fetching the later rounds' lines to L2 first gained nothing (25.6 and 25.1 us with
// the read-back), 1024 threads a CTA lost (28.6), 256 too (25.5).
// Gather of 8 x 8192 positions: 32.3 us, 196 MB at 6.1 TB/s.
#include <cooperative_groups.h>

#include "kv_append.cuh"
#include "kv_q8.cuh"
#include "sv_internal.h"

namespace cg = cooperative_groups;

namespace sv {
namespace {

constexpr int kThreads = 128;
constexpr int kCommitThreads = 512;
constexpr int kMaxR = 128;
constexpr int kCluster = 8;

// Largest magnitude in the rows, over the warp, and which rows hold NaN or infinity:
// such rows become NaN and do not count.
__device__ __forceinline__ float run_amax(uint2 (&x)[kQ8Run], uint32_t& bad) {
    uint32_t m2 = 0u;   // a maximum in each half
#pragma unroll
    for (int i = 0; i < kQ8Run; ++i) {
        m2 = __vmaxu2(m2, x[i].x & 0x7fff7fffu);
        m2 = __vmaxu2(m2, x[i].y & 0x7fff7fffu);
    }
    uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 >> 16, m2 & 0xffffu));
    bad = 0u;
    if (m >= 0x7f80u) {   // (rare) without the rows that are not finite
        uint32_t mine = 0u;
#pragma unroll
        for (int i = 0; i < kQ8Run; ++i) {
            const uint32_t r = __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu);
            if (max(r >> 16, r & 0xffffu) >= 0x7f80u) mine |= 1u << i;
        }
        bad = __reduce_or_sync(0xffffffffu, mine);
        m2 = 0u;
#pragma unroll
        for (int i = 0; i < kQ8Run; ++i) {
            if (bad >> i & 1u) {
                x[i] = make_uint2(0x7fc07fc0u, 0x7fc07fc0u);
            } else {
                m2 = __vmaxu2(m2, x[i].x & 0x7fff7fffu);
                m2 = __vmaxu2(m2, x[i].y & 0x7fff7fffu);
            }
        }
        m = __reduce_max_sync(0xffffffffu, max(m2 >> 16, m2 & 0xffffu));
    }
    return __uint_as_float(m << 16);
}

// The four dims that a lane has of a row of K, in two pairs: dims a, a + 1 and b, b + 1.
// In a row whose halves are turned against each other (dims d and d + rot / 2) both
// members of two rotation pairs, so that no value and no angle passes between lanes;
// else four dims side by side.
struct KDims {
    int a, b;
};
__device__ __forceinline__ KDims k_dims(const AppendArgs& g) {
    const int l = threadIdx.x & 31, half = g.rot / 2;
    if (!g.rope || g.interleaved) return {4 * l, 4 * l + 2};
    if (2 * l < half) return {2 * l, 2 * l + half};
    return {2 * l + half, 2 * l + 64};   // of the dims from rot on, which are not turned
}

// Turns the lane's dims of the sixteen rows of K and rounds them to bf16: the rows that
// the bf16 cache would hold.  cs is the rope table's row of the run's first position;
// rows outside first .. last are copies of the first or last one, and so are their angles.
__device__ __forceinline__ void turn_run(uint2 (&x)[kQ8Run], int first, int last, const float* cs, int rot, bool interleaved) {
    const int f = 2 * (threadIdx.x & 31), half = rot / 2;   // two angles: f, f + 1
    if (f >= half) return;
    constexpr int kAhead = 8;   // rows whose angles are on their way at a time
#pragma unroll
    for (int i0 = 0; i0 < kQ8Run; i0 += kAhead) {
        float2 co[kAhead], si[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const float* c = cs + min(max(i0 + i, first), last) * rot + f;
            co[i] = __ldg(reinterpret_cast<const float2*>(c));
            si[i] = __ldg(reinterpret_cast<const float2*>(c + half));
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            uint2& w = x[i0 + i];
            float v[4];
            unpack4(w, v);
            if (interleaved) {
                rope_turn(v[0], v[1], co[i].x, si[i].x);
                rope_turn(v[2], v[3], co[i].y, si[i].y);
            } else {
                rope_turn(v[0], v[2], co[i].x, si[i].x);
                rope_turn(v[1], v[3], co[i].y, si[i].y);
            }
            w = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
    }
}

// One warp writes positions first .. last (of the sixteen) of a run of a (page, head)
// block; x holds the lane's four dims (packed bf16; of V four side by side, of K those
// of kd) of the sixteen rows, zeros or copies of the first or last one outside first .. last.
// Positions before `first` keep their values, held anew where the
// scale grows; where the run's first position is written, what the run held is gone.
// Returns whether a row was not finite.
template <bool kV, bool kApart = false>
__device__ __forceinline__ bool write_run(uint8_t* blk, int run, int first, int last, uint2 (&x)[kQ8Run], KDims kd = {0, 0}) {
    const int lane = threadIdx.x & 31;
    float* scale = reinterpret_cast<float*>(blk + q8_scale_off(run));
    const float s_old = first > 0 ? *scale : 0.f;
    // V: what the octets that are not written whole hold
    uint4 old[2][2];
    bool part[2];
    if constexpr (kV) {
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            part[o] = last >= 8 * o && !(first <= 8 * o && last >= 8 * o + 7);
            if (part[o]) {
                const uint4* src = reinterpret_cast<const uint4*>(blk + q8_v_off(2 * run + o, 4 * lane));
                old[o][0] = src[0];
                old[o][1] = src[1];
            }
        }
    }
    uint32_t bad;
    const int need = q8_exponent(run_amax(x, bad));
    const int e_old = q8_stored_exponent(s_old), e = first > 0 ? max(need, e_old) : need;
    const bool again = first > 0 && e != e_old;   // the earlier codes are held anew
    // x 2^-e by one product, or two where 2^-e has no normal form (e > 126 does not occur)
    const float rs = q8_pow2(-e), f = q8_pow2(max(e_old - e, -126));
    if (lane == 0) *scale = q8_pow2(e);
    if constexpr (!kV) {
        uint8_t* rows = blk + q8_k_off(kQ8Run * run, 0);   // dim d of row i: at 128 i + (d ^ i % 8 * 16)
        if (again) {
#pragma unroll 4
            for (int i = 0; i < first; ++i) {
                uint32_t* p = reinterpret_cast<uint32_t*>(rows + 128 * i + (4 * lane ^ (i & 7) << 4));
                *p = q8_rescale4(*p, f);
            }
        }
#pragma unroll
        for (int i = 0; i < kQ8Run; ++i) {
            if (i < first || i > last) continue;
            float v[4];
            unpack4(x[i], v);
            const uint32_t lo = q8_codes2(v[0] * rs, v[1] * rs), hi = q8_codes2(v[2] * rs, v[3] * rs);
            if constexpr (kApart) {
                *reinterpret_cast<uint16_t*>(rows + 128 * i + (kd.a ^ (i & 7) << 4)) = static_cast<uint16_t>(lo);
                *reinterpret_cast<uint16_t*>(rows + 128 * i + (kd.b ^ (i & 7) << 4)) = static_cast<uint16_t>(hi);
            } else {
                *reinterpret_cast<uint32_t*>(rows + 128 * i + (4 * lane ^ (i & 7) << 4)) = lo | hi << 16;
            }
        }
    } else {
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            uint8_t* at = blk + q8_v_off(2 * run + o, 4 * lane);
            if (last < 8 * o) continue;
            if (first > 8 * o + 7 && !again) continue;
            uint32_t w[4][2];   // [dim][positions 0..3, 4..7]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) unpack4(x[8 * o + 4 * h + i], v[i]);
#pragma unroll
                for (int d = 0; d < 4; ++d) w[d][h] = q8_codes4(v[0][d] * rs, v[1][d] * rs, v[2][d] * rs, v[3][d] * rs);
            }
            if (part[o]) {
                const uint32_t ow[4][2] = {{old[o][0].x, old[o][0].y}, {old[o][0].z, old[o][0].w},
                                           {old[o][1].x, old[o][1].y}, {old[o][1].z, old[o][1].w}};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t fresh = 0u, before = 0u;   // the bytes that are new, those of positions before
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = 8 * o + 4 * h + i;
                        if (p >= first && p <= last) fresh |= 0xffu << 8 * i;
                        if (p < first) before |= 0xffu << 8 * i;
                    }
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        uint32_t k = ow[d][h];
                        if (again && before) k = (q8_rescale4(k, f) & before) | (k & ~before);
                        w[d][h] = (w[d][h] & fresh) | (k & ~fresh);
                    }
                }
            }
            uint4* dst = reinterpret_cast<uint4*>(at);
            dst[0] = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
            dst[1] = make_uint4(w[2][0], w[2][1], w[3][0], w[3][1]);
        }
    }
    return bad != 0u && lane == 0;
}

// Append: warp items (slot, head, K or V).  A sequence of n rows touches at most
// n / 16 + 2 runs, so slots row_off[b] / 16 + 2 b .. hold its runs, and no count has
// to be summed over the sequences before a warp finds its own.
__global__ void __launch_bounds__(kThreads, 5) append_q8_kernel(AppendArgs a, uint8_t* __restrict__ k_pool,
                                                             uint8_t* __restrict__ v_pool, uint32_t items) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t item_blocks = (items - 1) / (kThreads / 32) + 1;
    if (blockIdx.x >= item_blocks) {
        check_rows(a, (blockIdx.x - item_blocks) * kThreads + threadIdx.x);
        return;
    }
    const uint32_t it = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (it >= items) return;
    const uint32_t slot = it / (2u * a.Hkv), sub = it - slot * (2u * a.Hkv), h = sub >> 1;
    auto first_slot = [&](int i) { return static_cast<int64_t>(__ldg(a.row_off + i) >> 4) + 2 * static_cast<int64_t>(i); };
    const int b = warp_last_at_most(a.B, slot, first_slot);
    if (b < 0) return;
    int r0, r1;
    if (!append_rows(a, b, r0, r1)) return;
    const int t = __ldg(a.len + b);
    const int64_t run = static_cast<int64_t>(t >> 4) + (slot - first_slot(b));
    const int64_t end = static_cast<int64_t>(t) + (r1 - r0);
    const int64_t b0 = max(static_cast<int64_t>(t), kQ8Run * run), b1 = min(end, kQ8Run * run + kQ8Run);
    if (b0 >= b1) return;
    if (t < 0 || b1 > a.cap) {
        if (lane == 0) raise_error(a.err, SV_DEVERR_LENGTH);
        if (t < 0 || b0 >= a.cap) return;
    }
    const int p0 = static_cast<int>(b0), p1 = static_cast<int>(min(b1, static_cast<int64_t>(a.cap)));
    const int pg = __ldg(a.pages + static_cast<size_t>(b) * a.max_pages + p0 / kQ8Page);
    if (pg < 0 || pg >= a.num_pages) {
        if (lane == 0) raise_error(a.err, SV_DEVERR_PAGE);
        return;
    }
    const size_t blk = (static_cast<size_t>(pg) * a.Hkv + h) * kQ8Bytes;
    const int base = p0 & ~(kQ8Run - 1), first = p0 - base, last = p1 - 1 - base, r = (p0 & (kQ8Page - 1)) / kQ8Run;
    const bool is_v = sub & 1;
    const KDims kd = is_v ? KDims{4 * lane, 4 * lane + 2} : k_dims(a);
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const uint16_t* src = (is_v ? a.v : a.k) + h * kQ8D + (r0 + (base - t)) * stride;
    uint2 x[kQ8Run];
#pragma unroll
    for (int i = 0; i < kQ8Run; ++i) {
        const uint16_t* row = src + min(max(i, first), last) * stride;
        x[i] = make_uint2(__ldg(reinterpret_cast<const uint32_t*>(row + kd.a)), __ldg(reinterpret_cast<const uint32_t*>(row + kd.b)));
    }
    bool bad;
    if (is_v) {
        bad = write_run<true>(v_pool + blk, r, first, last, x);
    } else {
        if (a.rope) turn_run(x, first, last, a.rope + static_cast<int64_t>(base) * a.rot, a.rot, a.interleaved);
        bad = write_run<false, true>(k_pool + blk, r, first, last, x, kd);
    }
    if (bad) raise_error(a.err, SV_DEVERR_NONFINITE);
}

// Commit: one cluster per sequence, its warps taking (layer, head, run, K or V)
// items; every CTA reads len[b] before rank 0 advances it.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kCommitThreads)
    commit_q8_kernel(uint8_t* __restrict__ k_pool, uint8_t* __restrict__ v_pool, const uint16_t* __restrict__ k_blk,
                     const uint16_t* __restrict__ v_blk, int L, int B, int Hkv, int R, const int32_t* __restrict__ path,
                     const int32_t* __restrict__ n_acc, int32_t* len, const int32_t* __restrict__ pages, int max_pages,
                     int num_pages, unsigned int* err) {
    __shared__ int path_s[kMaxR], page_s[kMaxR];
    __shared__ int path_ok_s, page_ok_s;
    pdl_wait();
    pdl_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / kCluster;
    const int lane = threadIdx.x & 31;
    const int t = len[b], m = n_acc[b];
    cluster.barrier_arrive();   // len[b] has been read
    const bool m_ok = m >= 0 && m < R;
    const bool len_ok = t >= 0 && static_cast<int64_t>(t) + m + 1 <= static_cast<int64_t>(max_pages) * kQ8Page;
    if (threadIdx.x == 0) path_ok_s = page_ok_s = 1;
    __syncthreads();
    if (m_ok && len_ok && threadIdx.x <= m) {
        const int p = path[static_cast<size_t>(b) * R + threadIdx.x];
        path_s[threadIdx.x] = p;
        if (p < 0 || p >= R) path_ok_s = 0;
        const int pg = pages[static_cast<size_t>(b) * max_pages + (t + threadIdx.x) / kQ8Page];
        page_s[threadIdx.x] = pg;
        if (pg < 0 || pg >= num_pages) page_ok_s = 0;
    }
    __syncthreads();
    if (!m_ok || !len_ok || !path_ok_s || !page_ok_s) {   // uniform across the cluster: nobody writes
        if (rank == 0 && threadIdx.x == 0)
            raise_error(err, !m_ok || (len_ok && !path_ok_s) ? SV_DEVERR_PATH
                                                             : !len_ok ? SV_DEVERR_LENGTH : SV_DEVERR_PAGE);
        cluster.barrier_wait();
        return;
    }
    const uint32_t o0 = t / kQ8Run, nrun = (t + m) / kQ8Run - o0 + 1;
    const uint32_t items = static_cast<uint32_t>(L) * Hkv * 2 * nrun;
    bool bad = false;
    for (uint32_t it = rank * (kCommitThreads / 32) + (threadIdx.x >> 5); it < items; it += kCluster * (kCommitThreads / 32)) {
        const uint32_t kv = it & 1, x1 = it >> 1, lh = x1 / nrun, o = x1 - lh * nrun, l = lh / Hkv, h = lh - l * Hkv;
        const int base = kQ8Run * static_cast<int>(o0 + o), off = base - t, first = max(-off, 0), last = min(m - off, kQ8Run - 1);
        const size_t blk = ((static_cast<size_t>(l) * num_pages + page_s[off + first]) * Hkv + h) * kQ8Bytes;
        const uint16_t* src = (kv ? v_blk : k_blk) +
                              ((static_cast<size_t>(l) * B + b) * Hkv + h) * R * static_cast<size_t>(kQ8D) + 4 * lane;
        uint2 x[kQ8Run];
#pragma unroll
        for (int i = 0; i < kQ8Run; ++i) {
            x[i] = make_uint2(0u, 0u);
            if (i >= first && i <= last) x[i] = __ldg(reinterpret_cast<const uint2*>(src + path_s[off + i] * kQ8D));
        }
        const int r = (base & (kQ8Page - 1)) / kQ8Run;
        bad |= kv ? write_run<true>(v_pool + blk, r, first, last, x) : write_run<false>(k_pool + blk, r, first, last, x);
    }
    if (bad) raise_error(err, SV_DEVERR_NONFINITE);
    cluster.barrier_wait();   // every CTA has read len[b]
    if (rank == 0 && threadIdx.x == 0) len[b] = t + m + 1;
}

// Gather: warp items (layer, sequence, head, K or V, run).  A lane has eight dims
// (8 (lane & 15) ..), so it stores 16 bytes a row and two rows leave with one
// instruction: of K rows 2 i + lane / 16, of V rows i of octet lane / 16.
__global__ void __launch_bounds__(kThreads)
    gather_q8_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool, uint32_t B, uint32_t Hkv,
                     const int32_t* __restrict__ start, const int32_t* __restrict__ len, int n, uint32_t nrun,
                     const int32_t* __restrict__ pages, int max_pages, int num_pages, uint16_t* __restrict__ k_out,
                     uint16_t* __restrict__ v_out, uint32_t items, unsigned int* err) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane >> 4, d = 8 * (lane & 15);
    const uint32_t it = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (it >= items) return;
    const uint32_t lbhk = it / nrun, o = it - lbhk * nrun;
    const uint32_t kv = lbhk & 1, lbh = lbhk >> 1;   // lbh: (layer * B + sequence) * Hkv + head
    const uint32_t lb = lbh / Hkv, h = lbh - lb * Hkv, l = lb / B, b = lb - l * B;
    const int st = __ldg(start + b);
    int t = __ldg(len + b);
    if (t < 0 || t > max_pages * kQ8Page || st < 0) {
        if (lane == 0) raise_error(err, SV_DEVERR_LENGTH);
        t = st < 0 ? 0 : max(0, min(t, max_pages * kQ8Page));
    }
    const int64_t q0 = static_cast<int64_t>(st & ~(kQ8Run - 1)) + kQ8Run * static_cast<int64_t>(o);   // the run's first position
    const uint8_t* blk = nullptr;
    if (q0 >= 0 && q0 < t) {
        const int pg = __ldg(pages + static_cast<size_t>(b) * max_pages + q0 / kQ8Page);
        if (pg < 0 || pg >= num_pages) {
            if (lane == 0) raise_error(err, SV_DEVERR_PAGE);
        } else {
            blk = (kv ? v_pool : k_pool) + ((static_cast<size_t>(l) * num_pages + pg) * Hkv + h) * kQ8Bytes;
        }
    }
    const int run = static_cast<int>(q0 & (kQ8Page - 1)) / kQ8Run;
    uint16_t* out = (kv ? v_out : k_out) + static_cast<size_t>(lbh) * n * kQ8D + d;
    auto store = [&](int pos, uint4 y) {
        const int64_t r = q0 + pos - st;
        if (r < 0 || r >= n) return;
        if (q0 + pos >= t) y = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(out + r * kQ8D) = y;
    };
    if (!blk) {
#pragma unroll
        for (int i = 0; i < kQ8Run / 2; ++i) store(2 * i + sub, make_uint4(0u, 0u, 0u, 0u));
        return;
    }
    // a pair's value: 2^120 takes the code to its own, then the scale (exact both, and
    // one product would not do: 2^(120 + e) can pass bf16's largest)
    const uint32_t up = q8_pow2_pair(120);
    const uint32_t sb = __float_as_uint(__ldg(reinterpret_cast<const float*>(blk + q8_scale_off(run)))) >> 16;
    const uint32_t s2 = sb | sb << 16;
    auto value = [&](uint32_t p) { return q8_mul2(q8_mul2(p, up), s2); };
    if (kv) {
        uint4 c[4];
        const uint4* src = reinterpret_cast<const uint4*>(blk + q8_v_off(2 * run + sub, d));
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = __ldg(src + i);
        const uint32_t w[8][2] = {{c[0].x, c[0].y}, {c[0].z, c[0].w}, {c[1].x, c[1].y}, {c[1].z, c[1].w},
                                  {c[2].x, c[2].y}, {c[2].z, c[2].w}, {c[3].x, c[3].y}, {c[3].z, c[3].w}};
        auto row = [&](int pos, const uint32_t (&p)[4]) {
            store(8 * sub + pos, make_uint4(q8_nan_pair(p[0], value(p[0])), q8_nan_pair(p[1], value(p[1])), q8_nan_pair(p[2], value(p[2])),
                                            q8_nan_pair(p[3], value(p[3]))));
        };
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t p[4][4];   // [position][pair of dims]
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[0][e] = q8_pair<0, 4>(w[2 * e][g], w[2 * e + 1][g]);
                p[1][e] = q8_pair<1, 5>(w[2 * e][g], w[2 * e + 1][g]);
                p[2][e] = q8_pair<2, 6>(w[2 * e][g], w[2 * e + 1][g]);
                p[3][e] = q8_pair<3, 7>(w[2 * e][g], w[2 * e + 1][g]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) row(4 * g + i, p[i]);
        }
    } else {
        uint2 w[kQ8Run / 2];
#pragma unroll
        for (int i = 0; i < kQ8Run / 2; ++i)
            w[i] = __ldg(reinterpret_cast<const uint2*>(blk + q8_k_off(kQ8Run * run + 2 * i + sub, d >> 4) + (d & 8)));
#pragma unroll
        for (int i = 0; i < kQ8Run / 2; ++i) {
            const uint32_t p[4] = {q8_pair<0, 1>(w[i].x, 0u), q8_pair<2, 3>(w[i].x, 0u), q8_pair<0, 1>(w[i].y, 0u),
                                   q8_pair<2, 3>(w[i].y, 0u)};
            store(2 * i + sub, make_uint4(q8_nan_pair(p[0], value(p[0])), q8_nan_pair(p[1], value(p[1])), q8_nan_pair(p[2], value(p[2])),
                                          q8_nan_pair(p[3], value(p[3]))));
        }
    }
}

unsigned int warp_grid(int64_t items) {
    return static_cast<unsigned int>((items + kThreads / 32 - 1) / (kThreads / 32));
}

}  // namespace

int64_t append_q8_items(int N, int B, int Hkv) {
    return (static_cast<int64_t>(N) / kQ8Run + 2 * static_cast<int64_t>(B)) * 2 * Hkv;
}

cudaError_t launch_append_q8(const AppendArgs& a, uint8_t* k_pool, uint8_t* v_pool, cudaStream_t st) {
    const int64_t items = append_q8_items(a.N, a.B, a.Hkv);
    const uint32_t checks = (a.B - 1) / kThreads + 1;
    return launch_pdl(append_q8_kernel, dim3(warp_grid(items) + checks), dim3(kThreads), 0, st, a, k_pool, v_pool,
                      static_cast<uint32_t>(items));
}

cudaError_t launch_commit_q8(uint8_t* k_pool, uint8_t* v_pool, const uint16_t* k_blk, const uint16_t* v_blk, int L,
                             int B, int Hkv, int R, const int32_t* path, const int32_t* n_acc, int32_t* len,
                             const int32_t* pages, int max_pages, int num_pages, cudaStream_t st) {
    return launch_pdl(commit_q8_kernel, dim3(B * kCluster), dim3(kCommitThreads), 0, st, k_pool, v_pool, k_blk, v_blk, L, B,
                      Hkv, R, path, n_acc, len, pages, max_pages, num_pages, device_error_word());
}

int64_t gather_q8_items(int L, int B, int Hkv, int n) {
    return static_cast<int64_t>(L) * B * Hkv * 2 * ((static_cast<int64_t>(n) + kQ8Run - 1) / kQ8Run + 1);
}

cudaError_t launch_gather_q8(const uint8_t* k_pool, const uint8_t* v_pool, int L, int B, int Hkv, const int32_t* start,
                             const int32_t* len, int n, const int32_t* pages, int max_pages, int num_pages,
                             uint16_t* k_out, uint16_t* v_out, cudaStream_t st) {
    const int64_t items = gather_q8_items(L, B, Hkv, n);
    return launch_pdl(gather_q8_kernel, dim3(warp_grid(items)), dim3(kThreads), 0, st, k_pool, v_pool,
                      static_cast<uint32_t>(B), static_cast<uint32_t>(Hkv), start, len, n,
                      static_cast<uint32_t>((static_cast<int64_t>(n) + kQ8Run - 1) / kQ8Run + 1), pages, max_pages, num_pages,
                      k_out, v_out, static_cast<uint32_t>(items), device_error_word());
}

}  // namespace sv
