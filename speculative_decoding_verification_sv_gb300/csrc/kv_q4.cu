// kv_q4.cu -- writing and reading the 4-bit paged KV cache (format: kv_q4.cuh).
//
//   append  new rows of a layer, K rotated by position (as kv_append.cu), the
//           bf16 rows that the bf16 cache would hold quantised on the way
//   commit  the accepted rows of a verify block, every layer (as kv_commit.cu)
//   gather  a window of positions read back as bf16 rows
//
// V's words hold eight positions of a dim, so the unit of writing is an octet
// (eight aligned positions of one (sequence, head)): one warp owns it, reads
// back the words of an octet that was partly filled before, and writes each
// word once.  No two warps of a launch share a word, and none waits for
// another.
//
// Measured.  append, 4 x 1024 new rows of 4 heads at position 7168: 7.3 us, held up by
// the chain that finds an octet's place, loads its rows and angles, quantises and (at
// the ends of a sequence) merges; the rows are all sent for before the first is looked
// at, and the scales are formed once a lane for eight rows (quantising row by row took
// 15 us under the profiler, this 11.6).  gather, 32768 rows of 4 heads back to bf16: 15
// us, 4.5 TB/s of stores, bound by them.  commit, 16 sequences of 28 layers: 12.4 us,
// for one sequence 3.6 us: the 448 octets of a sequence whose rows lie in two (28
// layers, 4 heads, K and V) are four rounds of the 128 warps of its cluster, each a
// chain of the path, the row, the quantising and V's merge, and the SMs beside the 128
// CTAs are idle.  A warp an octet over the whole grid, with the lengths advanced by a
// second launch, took 4 us less for 16 sequences, 1 us more for one, and a launch more
// on the host; one launch could do the same with a counter of each sequence's CTAs.
#include <cooperative_groups.h>

#include "kv_append.cuh"
#include "kv_q4.cuh"
#include "sv_internal.h"

namespace cg = cooperative_groups;

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kCommitThreads = 512;
constexpr int kMaxR = 128;
constexpr int kCluster = 8;

// Turns the lane's four dims (4 lane .., packed bf16) of the rows of positions
// base + first .. base + last of a K octet and rounds them to bf16: the rows that
// the bf16 cache would hold.  cs is the table's row of position base.  Two rows'
// cosines and sines are on their way at a time (four took 104 bytes of spills).
template <bool kInterleaved>
__device__ __forceinline__ void turn_rows(uint2 (&x)[8], int first, int last, const float* cs, int rot) {
    const int lane = threadIdx.x & 31, d = 4 * lane, half = rot / 2;
    const bool in = d < rot, lower = d < half;   // lower: the first member of its pair (halves)
    const int mate = !in ? lane : lower ? lane + half / 4 : lane - half / 4;
    const int f = !in ? 0 : kInterleaved ? d / 2 : lower ? d : d - half;
#pragma unroll
    for (int i0 = 0; i0 < 8; i0 += 2) {
        float4 co[2], si[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i0 + i < first || i0 + i > last) continue;
            const float* c = cs + static_cast<int64_t>(i0 + i) * rot + f;
            if constexpr (kInterleaved) {
                const float2 a = __ldg(reinterpret_cast<const float2*>(c));
                const float2 b = __ldg(reinterpret_cast<const float2*>(c + half));
                co[i] = make_float4(a.x, a.y, 0.0f, 0.0f);
                si[i] = make_float4(b.x, b.y, 0.0f, 0.0f);
            } else {
                co[i] = __ldg(reinterpret_cast<const float4*>(c));
                si[i] = __ldg(reinterpret_cast<const float4*>(c + half));
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i0 + i < first || i0 + i > last) continue;
            uint2& w = x[i0 + i];
            float v[4];
            unpack4(w, v);
            if constexpr (kInterleaved) {
                rope_turn(v[0], v[1], co[i].x, si[i].x);
                rope_turn(v[2], v[3], co[i].y, si[i].y);
            } else {
                float y[4];
                unpack4(make_uint2(__shfl_sync(0xffffffffu, w.x, mate), __shfl_sync(0xffffffffu, w.y, mate)), y);
                const float cc[4] = {co[i].x, co[i].y, co[i].z, co[i].w}, ss[4] = {si[i].x, si[i].y, si[i].z, si[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float a = lower ? v[e] : y[e], b = lower ? y[e] : v[e];
                    rope_turn(a, b, cc[e], ss[e]);
                    v[e] = lower ? a : b;
                }
            }
            const uint2 r = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            w = in ? r : w;
        }
    }
}

// One warp writes positions first .. last (of the eight) of an octet of a
// (page, head) block; rows holds the lane's four dims (packed bf16) of the eight
// rows, zeros outside first .. last.  Returns whether a group held NaN or
// infinity.
template <bool kV>
__device__ __forceinline__ bool write_octet(uint8_t* blk, int octet, int first, int last, const uint2 (&rows)[8]) {
    const int lane = threadIdx.x & 31, g = lane >> 3, row = lane & 7;
    const bool whole = first == 0 && last == 7;
    uint4 old = make_uint4(0u, 0u, 0u, 0u);   // V: words that hold positions of before
    if (kV && !whole) old = *reinterpret_cast<const uint4*>(blk + q4_v_code_off(octet, 4 * lane));
    float x[8][4], s, rs;
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack4(rows[i], x[i]);
    q4_scales8(x, s, rs);
    const bool mine = row >= first && row <= last;   // the lane stores this row's scale
    if (mine)
        *reinterpret_cast<uint16_t*>(blk + (kV ? q4_v_scale_off(g, 8 * octet + row) : q4_k_scale_off(g, 8 * octet + row))) =
            f32_bf16_bits(s);
    if constexpr (kV) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < first || i > last) continue;   // (its nibbles are taken from before)
            const float si = __shfl_sync(0xffffffffu, s, i, 8), ri = __shfl_sync(0xffffffffu, rs, i, 8);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] += (q4_code(x[i][e], si, ri) - kQ4CodeBase) * (1u << q4_shift(i));
        }
        uint4* dst = reinterpret_cast<uint4*>(blk + q4_v_code_off(octet, 4 * lane));
        if (!whole) {
            uint32_t keep = 0u;   // the nibbles of positions that are not written
#pragma unroll
            for (int i = 0; i < 8; ++i) keep |= i < first || i > last ? 15u << q4_shift(i) : 0u;
            w[0] |= old.x & keep;
            w[1] |= old.y & keep;
            w[2] |= old.z & keep;
            w[3] |= old.w & keep;
        }
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        uint32_t h[8];   // a row's four codes of this lane, in the half word that they take
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = 0u;
            if (i < first || i > last) continue;
            const float si = __shfl_sync(0xffffffffu, s, i, 8), ri = __shfl_sync(0xffffffffu, rs, i, 8);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[i] += (q4_code(x[i][e], si, ri) - kQ4CodeBase) * (1u << q4_shift(e));
            h[i] <<= 8 * (lane & 1);
        }
        // eight lanes' half words of eight rows turned: lane (g, row) ends up with
        // the 16 bytes of its row's group
        const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
        uint32_t p[4], q[2][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)   // rows 2 i + (lane & 1)
            p[i] = (b0 ? h[2 * i + 1] : h[2 * i]) | __shfl_xor_sync(0xffffffffu, b0 ? h[2 * i] : h[2 * i + 1], 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // rows 4 i + (lane & 3)
            const uint32_t own = b1 ? p[2 * i + 1] : p[2 * i];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? p[2 * i] : p[2 * i + 1], 2);
            q[i][0] = b1 ? got : own;
            q[i][1] = b1 ? own : got;
        }
        const uint32_t o0 = b2 ? q[1][0] : q[0][0], o1 = b2 ? q[1][1] : q[0][1];
        const uint32_t g0 = __shfl_xor_sync(0xffffffffu, b2 ? q[0][0] : q[1][0], 4);
        const uint32_t g1 = __shfl_xor_sync(0xffffffffu, b2 ? q[0][1] : q[1][1], 4);
        if (mine)
            *reinterpret_cast<uint4*>(blk + q4_k_code_off(g, 8 * octet + row)) =
                b2 ? make_uint4(g0, g1, o0, o1) : make_uint4(o0, o1, g0, g1);
    }
    return mine && s != s;
}

// Append: warp items (slot, head, K or V).  A sequence of n rows touches at
// most n / 8 + 2 octets, so slots row_off[b] / 8 + 2 b .. hold its octets, and
// no count has to be summed over the sequences before a warp finds its own.
__global__ void __launch_bounds__(kThreads, 4) append_q4_kernel(AppendArgs a, uint8_t* __restrict__ k_pool,
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
    auto first_slot = [&](int i) { return static_cast<int64_t>(__ldg(a.row_off + i) >> 3) + 2 * static_cast<int64_t>(i); };
    const int b = warp_last_at_most(a.B, slot, first_slot);
    if (b < 0) return;
    int r0, r1;
    if (!append_rows(a, b, r0, r1)) return;
    const int t = __ldg(a.len + b);
    const int64_t octet = static_cast<int64_t>(t >> 3) + (slot - first_slot(b));
    const int64_t end = static_cast<int64_t>(t) + (r1 - r0);
    const int64_t b0 = max(static_cast<int64_t>(t), 8 * octet), b1 = min(end, 8 * octet + 8);
    if (b0 >= b1) return;
    if (t < 0 || b1 > a.cap) {
        if (lane == 0) raise_error(a.err, SV_DEVERR_LENGTH);
        if (t < 0 || b0 >= a.cap) return;
    }
    const int p0 = static_cast<int>(b0), p1 = static_cast<int>(min(b1, static_cast<int64_t>(a.cap)));
    const int pg = __ldg(a.pages + static_cast<size_t>(b) * a.max_pages + p0 / kQ4Page);
    if (pg < 0 || pg >= a.num_pages) {
        if (lane == 0) raise_error(a.err, SV_DEVERR_PAGE);
        return;
    }
    const size_t blk = (static_cast<size_t>(pg) * a.Hkv + h) * kQ4Bytes;
    const int base = p0 & ~7, first = p0 - base, last = p1 - 1 - base, oct = (p0 & (kQ4Page - 1)) >> 3;
    const int64_t stride = sub & 1 ? a.v_stride : a.k_stride;
    const uint16_t* src = (sub & 1 ? a.v : a.k) + h * kQ4D + 4 * lane + (r0 + (base - t)) * stride;
    uint2 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = make_uint2(0u, 0u);
        if (i >= first && i <= last) x[i] = __ldg(reinterpret_cast<const uint2*>(src + i * stride));
    }
    bool bad;
    if (sub & 1) {
        bad = write_octet<true>(v_pool + blk, oct, first, last, x);
    } else {
        if (a.rope) {
            const float* cs = a.rope + static_cast<int64_t>(base) * a.rot;
            if (a.interleaved) turn_rows<true>(x, first, last, cs, a.rot);
            else turn_rows<false>(x, first, last, cs, a.rot);
        }
        bad = write_octet<false>(k_pool + blk, oct, first, last, x);
    }
    if (bad) raise_error(a.err, SV_DEVERR_NONFINITE);
}

// Commit: one cluster per sequence, its warps taking (layer, head, octet, K or
// V) items; every CTA reads len[b] before rank 0 advances it.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kCommitThreads)
    commit_q4_kernel(uint8_t* __restrict__ k_pool, uint8_t* __restrict__ v_pool, const uint16_t* __restrict__ k_blk,
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
    const bool len_ok = t >= 0 && static_cast<int64_t>(t) + m + 1 <= static_cast<int64_t>(max_pages) * kQ4Page;
    if (threadIdx.x == 0) path_ok_s = page_ok_s = 1;
    __syncthreads();
    if (m_ok && len_ok && threadIdx.x <= m) {
        const int p = path[static_cast<size_t>(b) * R + threadIdx.x];
        path_s[threadIdx.x] = p;
        if (p < 0 || p >= R) path_ok_s = 0;
        const int pg = pages[static_cast<size_t>(b) * max_pages + (t + threadIdx.x) / kQ4Page];
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
    const uint32_t o0 = t >> 3, noct = ((t + m) >> 3) - o0 + 1;
    const uint32_t items = static_cast<uint32_t>(L) * Hkv * 2 * noct;
    bool bad = false;
    for (uint32_t it = rank * (kCommitThreads / 32) + (threadIdx.x >> 5); it < items; it += kCluster * (kCommitThreads / 32)) {
        const uint32_t kv = it & 1, x1 = it >> 1, lh = x1 / noct, o = x1 - lh * noct, l = lh / Hkv, h = lh - l * Hkv;
        const int base = 8 * static_cast<int>(o0 + o), off = base - t, first = max(-off, 0), last = min(m - off, 7);
        const size_t blk = ((static_cast<size_t>(l) * num_pages + page_s[off + first]) * Hkv + h) * kQ4Bytes;
        const uint16_t* src = (kv ? v_blk : k_blk) +
                              ((static_cast<size_t>(l) * B + b) * Hkv + h) * R * static_cast<size_t>(kQ4D) + 4 * lane;
        uint2 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = make_uint2(0u, 0u);
            if (i >= first && i <= last) x[i] = __ldg(reinterpret_cast<const uint2*>(src + path_s[off + i] * kQ4D));
        }
        const int oct = (base & (kQ4Page - 1)) >> 3;
        bad |= kv ? write_octet<true>(v_pool + blk, oct, first, last, x)
                  : write_octet<false>(k_pool + blk, oct, first, last, x);
    }
    if (bad) raise_error(err, SV_DEVERR_NONFINITE);
    cluster.barrier_wait();   // every CTA has read len[b]
    if (rank == 0 && threadIdx.x == 0) len[b] = t + m + 1;
}

// Gather: warp items (layer, sequence, head, K or V, octet of positions); a lane
// has eight dims (8 (lane & 15) ..) of four of the octet's positions, so it
// stores 16 bytes a row and two rows leave with one instruction.  A word's codes
// become bf16 two at a time: or-ed into the low bits of bf16 128, 136 taken off
// and the scale multiplied, all exact.
__device__ __forceinline__ uint32_t q4_pair(uint32_t codes, __nv_bfloat162 s) {
    const uint32_t x = (codes & 0x000f000fu) | 0x43004300u, off = 0x43084308u;
    const __nv_bfloat162 y = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                             *reinterpret_cast<const __nv_bfloat162*>(&off)), s);
    return *reinterpret_cast<const uint32_t*>(&y);
}

__global__ void __launch_bounds__(kThreads)
    gather_q4_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool, uint32_t B, uint32_t Hkv,
                     const int32_t* __restrict__ start, const int32_t* __restrict__ len, int n, uint32_t noct,
                     const int32_t* __restrict__ pages, int max_pages, int num_pages, uint16_t* __restrict__ k_out,
                     uint16_t* __restrict__ v_out, uint32_t items, unsigned int* err) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane >> 4, d = 8 * (lane & 15), g = d >> 5;
    const uint32_t it = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (it >= items) return;
    const uint32_t lbhk = it / noct, o = it - lbhk * noct;
    const uint32_t kv = lbhk & 1, lbh = lbhk >> 1;   // lbh: (layer * B + sequence) * Hkv + head
    const uint32_t lb = lbh / Hkv, h = lbh - lb * Hkv, l = lb / B, b = lb - l * B;
    const int st = __ldg(start + b);
    int t = __ldg(len + b);
    if (t < 0 || t > max_pages * kQ4Page || st < 0) {
        if (lane == 0) raise_error(err, SV_DEVERR_LENGTH);
        t = st < 0 ? 0 : max(0, min(t, max_pages * kQ4Page));
    }
    const int64_t q0 = static_cast<int64_t>(st & ~7) + 8 * static_cast<int64_t>(o);   // the octet's first position
    const uint8_t* blk = nullptr;
    if (q0 >= 0 && q0 < t) {
        const int pg = __ldg(pages + static_cast<size_t>(b) * max_pages + q0 / kQ4Page);
        if (pg < 0 || pg >= num_pages) {
            if (lane == 0) raise_error(err, SV_DEVERR_PAGE);
        } else {
            blk = (kv ? v_pool : k_pool) + ((static_cast<size_t>(l) * num_pages + pg) * Hkv + h) * kQ4Bytes;
        }
    }
    const int oct = static_cast<int>(q0 & (kQ4Page - 1)) >> 3;
    uint16_t* out = (kv ? v_out : k_out) + static_cast<size_t>(lbh) * n * kQ4D + d;
    // row i of the lane's four is position q0 + pos(i)
    auto store = [&](int pos, uint4 y) {
        const int64_t r = q0 + pos - st;
        if (r < 0 || r >= n) return;
        if (q0 + pos >= t) y = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(out + r * kQ4D) = y;
    };
    if (!blk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) store(2 * i + sub, make_uint4(0u, 0u, 0u, 0u));
    } else if (kv) {
        // positions 4 sub .. 4 sub + 3: bits 8 sub .. of the words' halves
        const uint4* src = reinterpret_cast<const uint4*>(blk + q4_v_code_off(oct, d));
        const uint4 lo = __ldg(src), hi = __ldg(src + 1);
        const uint2 sc = __ldg(reinterpret_cast<const uint2*>(blk + q4_v_scale_off(g, 8 * oct + 4 * sub)));
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // element 4 sub + i of a word: half i & 1, bit 4 (2 sub + i / 2)
            const uint32_t sb = __byte_perm(i < 2 ? sc.x : sc.y, 0u, i & 1 ? 0x3232 : 0x1010);
            const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&sb);
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = q4_pair(__byte_perm(w[2 * e], w[2 * e + 1], i & 1 ? 0x7632 : 0x5410) >> (8 * sub + 4 * (i >> 1)), s);
            store(4 * sub + i, make_uint4(y[0], y[1], y[2], y[3]));
        }
    } else {
        uint32_t w[4];
        uint16_t sb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int slot = 8 * oct + 2 * i + sub;
            w[i] = __ldg(reinterpret_cast<const uint32_t*>(blk + q4_k_code_off(g, slot) + 4 * (lane & 3)));
            sb[i] = __ldg(reinterpret_cast<const uint16_t*>(blk + q4_k_scale_off(g, slot)));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 s = __bfloat162bfloat162(__ushort_as_bfloat16(sb[i]));
            store(2 * i + sub, make_uint4(q4_pair(w[i], s), q4_pair(w[i] >> 4, s), q4_pair(w[i] >> 8, s),
                                          q4_pair(w[i] >> 12, s)));
        }
    }
}

unsigned int warp_grid(int64_t items) {
    return static_cast<unsigned int>((items + kThreads / 32 - 1) / (kThreads / 32));
}

}  // namespace

int64_t append_q4_items(int N, int B, int Hkv) { return (static_cast<int64_t>(N) / 8 + 2 * static_cast<int64_t>(B)) * 2 * Hkv; }

cudaError_t launch_append_q4(const AppendArgs& a, uint8_t* k_pool, uint8_t* v_pool, cudaStream_t st) {
    const int64_t items = append_q4_items(a.N, a.B, a.Hkv);
    const uint32_t checks = (a.B - 1) / kThreads + 1;
    return launch_pdl(append_q4_kernel, dim3(warp_grid(items) + checks), dim3(kThreads), 0, st, a, k_pool, v_pool,
                      static_cast<uint32_t>(items));
}

cudaError_t launch_commit_q4(uint8_t* k_pool, uint8_t* v_pool, const uint16_t* k_blk, const uint16_t* v_blk, int L,
                             int B, int Hkv, int R, const int32_t* path, const int32_t* n_acc, int32_t* len,
                             const int32_t* pages, int max_pages, int num_pages, cudaStream_t st) {
    return launch_pdl(commit_q4_kernel, dim3(B * kCluster), dim3(kCommitThreads), 0, st, k_pool, v_pool, k_blk, v_blk, L, B,
                      Hkv, R, path, n_acc, len, pages, max_pages, num_pages, device_error_word());
}

int64_t gather_q4_items(int L, int B, int Hkv, int n) {
    return static_cast<int64_t>(L) * B * Hkv * 2 * ((static_cast<int64_t>(n) + 7) / 8 + 1);
}

cudaError_t launch_gather_q4(const uint8_t* k_pool, const uint8_t* v_pool, int L, int B, int Hkv, const int32_t* start,
                             const int32_t* len, int n, const int32_t* pages, int max_pages, int num_pages,
                             uint16_t* k_out, uint16_t* v_out, cudaStream_t st) {
    const int64_t items = gather_q4_items(L, B, Hkv, n);
    return launch_pdl(gather_q4_kernel, dim3(warp_grid(items)), dim3(kThreads), 0, st, k_pool, v_pool,
                      static_cast<uint32_t>(B), static_cast<uint32_t>(Hkv), start, len, n,
                      static_cast<uint32_t>((n + 7) / 8 + 1), pages, max_pages, num_pages, k_out, v_out,
                      static_cast<uint32_t>(items), device_error_word());
}

}  // namespace sv
