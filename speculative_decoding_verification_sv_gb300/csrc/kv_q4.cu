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
#include <cooperative_groups.h>

#include "kv_append.cuh"
#include "kv_q4.cuh"
#include "sv_internal.h"

namespace cg = cooperative_groups;

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxR = 128;
constexpr int kCluster = 8;

// Four bf16 dims (4 lane ..) of a row.
__device__ __forceinline__ void load4(const uint16_t* row, int d, float (&x)[4]) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + d));
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// The lane's four dims of a K row at position pos, rotated and rounded to
// bf16: the row that the bf16 cache would hold.
__device__ __forceinline__ void load4_turned(const uint16_t* row, const float* cs, int rot, bool interleaved,
                                             float (&x)[4]) {
    const int d = 4 * (threadIdx.x & 31), half = rot / 2;
    load4(row, d, x);
    if (d >= rot) return;
    if (interleaved) {
        const float2 co = __ldg(reinterpret_cast<const float2*>(cs + d / 2));
        const float2 si = __ldg(reinterpret_cast<const float2*>(cs + half + d / 2));
        rope_turn(x[0], x[1], co.x, si.x);
        rope_turn(x[2], x[3], co.y, si.y);
    } else {
        // the pair's other member, the first (d < half) or the second of its pair
        const bool first = d < half;
        const int f = first ? d : d - half;
        float y[4];
        load4(row, first ? d + half : f, y);
        const float4 co = __ldg(reinterpret_cast<const float4*>(cs + f));
        const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + f));
        const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a = first ? x[e] : y[e], b = first ? y[e] : x[e];
            rope_turn(a, b, cc[e], ss[e]);
            x[e] = first ? a : b;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = bf16_bits_f32(f32_bf16_bits(x[e]));
}

// One warp writes positions [p0, p1) of an octet (same octet, same page) into
// the (page, head) block: row(p, x) loads the lane's four dims of position p.
// Returns whether a group held NaN or infinity.
template <bool kV, typename Row>
__device__ __forceinline__ bool write_octet(uint8_t* blk, int p0, int p1, Row&& row) {
    const int lane = threadIdx.x & 31;
    const int first = p0 & 7, n = p1 - p0, slot = p0 & (kQ4Page - 1);
    float x[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) row(p0 + i, x[i]);
    bool bad = false;
    if constexpr (kV) {
        uint4* dst = reinterpret_cast<uint4*>(blk + q4_v_code_off(slot >> 3, 4 * lane));
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        uint32_t mine = 0u;   // the nibbles of the new positions
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= n) break;
            uint32_t c[4];
            float s;
            q4_quantise4(x[i], c, s);
            bad |= s != s;
            const int sh = q4_shift(first + i);
            mine |= 15u << sh;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] |= c[e] << sh;
            if ((lane & 7) == 0)
                *reinterpret_cast<uint16_t*>(blk + q4_v_scale_off(lane >> 3, slot + i)) = f32_bf16_bits(s);
        }
        if (n < 8) {
            const uint4 old = *dst;
            w[0] |= old.x & ~mine;
            w[1] |= old.y & ~mine;
            w[2] |= old.z & ~mine;
            w[3] |= old.w & ~mine;
        }
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= n) break;
            uint32_t c[4];
            float s;
            q4_quantise4(x[i], c, s);
            bad |= s != s;
            uint32_t h = (c[0] | (c[1] << 16) | (c[2] << 4) | (c[3] << 20)) << (8 * (lane & 1));
            h |= __shfl_xor_sync(0xffffffffu, h, 1);
            if ((lane & 1) == 0)
                *reinterpret_cast<uint32_t*>(blk + q4_k_code_off(lane >> 3, slot + i) + 2 * (lane & 7)) = h;
            if ((lane & 7) == 0)
                *reinterpret_cast<uint16_t*>(blk + q4_k_scale_off(lane >> 3, slot + i)) = f32_bf16_bits(s);
        }
    }
    return bad;
}

// Append: warp items (slot, head, K or V).  A sequence of n rows touches at
// most n / 8 + 2 octets, so slots row_off[b] / 8 + 2 b .. hold its octets, and
// no count has to be summed over the sequences before a warp finds its own.
__global__ void __launch_bounds__(kThreads) append_q4_kernel(AppendArgs a, uint8_t* __restrict__ k_pool,
                                                             uint8_t* __restrict__ v_pool, int64_t items) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (it >= items) return;
    const int64_t slot = it / (2 * a.Hkv);
    const int sub = static_cast<int>(it % (2 * a.Hkv)), h = sub >> 1;
    auto first_slot = [&](int i) { return static_cast<int64_t>(__ldg(a.row_off + i) >> 3) + 2 * static_cast<int64_t>(i); };
    const int b = warp_last_at_most(a.B, slot, first_slot);
    if (b < 0) return;
    int r0, r1;
    if (!append_rows(a, b, r0, r1)) {
        if (lane == 0) raise_error(a.err, SV_DEVERR_ROWS);
        return;
    }
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
    bool bad;
    if (sub & 1) {
        bad = write_octet<true>(v_pool + blk, p0, p1, [&](int p, float(&x)[4]) {
            load4(a.v + static_cast<int64_t>(r0 + (p - t)) * a.v_stride + h * kQ4D, 4 * lane, x);
        });
    } else {
        bad = write_octet<false>(k_pool + blk, p0, p1, [&](int p, float(&x)[4]) {
            const uint16_t* row = a.k + static_cast<int64_t>(r0 + (p - t)) * a.k_stride + h * kQ4D;
            if (a.rope) load4_turned(row, a.rope + static_cast<size_t>(p) * a.rot, a.rot, a.interleaved, x);
            else load4(row, 4 * lane, x);
        });
    }
    if (bad) raise_error(a.err, SV_DEVERR_NONFINITE);
}

// Commit: one cluster per sequence, its warps taking (layer, head, K or V,
// octet) items; every CTA reads len[b] before rank 0 advances it.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
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
    if (!m_ok || !len_ok || !path_ok_s || !page_ok_s) {   // uniform across the cluster: nobody writes or waits
        if (rank == 0 && threadIdx.x == 0)
            raise_error(err, !m_ok || (len_ok && !path_ok_s) ? SV_DEVERR_PATH
                                                             : !len_ok ? SV_DEVERR_LENGTH : SV_DEVERR_PAGE);
        return;
    }
    const int o0 = t >> 3, noct = ((t + m) >> 3) - o0 + 1;
    const int items = L * Hkv * 2 * noct;
    bool bad = false;
    for (int it = rank * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += kCluster * (kThreads / 32)) {
        const int o = it % noct, kv = it / noct & 1, lh = it / noct >> 1;
        const int l = lh / Hkv, h = lh % Hkv;
        const int p0 = max(t, 8 * (o0 + o)), p1 = min(t + m + 1, 8 * (o0 + o) + 8);
        const size_t blk = ((static_cast<size_t>(l) * num_pages + page_s[p0 - t]) * Hkv + h) * kQ4Bytes;
        const uint16_t* src = (kv ? v_blk : k_blk) + (static_cast<size_t>(l) * B + b) * Hkv * R * kQ4D +
                              static_cast<size_t>(h) * R * kQ4D;
        auto row = [&](int p, float(&x)[4]) { load4(src + path_s[p - t] * kQ4D, 4 * lane, x); };
        bad |= kv ? write_octet<true>(v_pool + blk, p0, p1, row) : write_octet<false>(k_pool + blk, p0, p1, row);
    }
    if (bad) raise_error(err, SV_DEVERR_NONFINITE);
    cluster.sync();   // every CTA has read len[b]
    if (rank == 0 && threadIdx.x == 0) len[b] = t + m + 1;
}

// Gather: warp items (layer, sequence, head, K or V, octet of positions).
__global__ void __launch_bounds__(kThreads)
    gather_q4_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool, int L, int B, int Hkv,
                     const int32_t* __restrict__ start, const int32_t* __restrict__ len, int n, int noct,
                     const int32_t* __restrict__ pages, int max_pages, int num_pages, uint16_t* __restrict__ k_out,
                     uint16_t* __restrict__ v_out, int64_t items, unsigned int* err) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, d = 4 * lane;
    const int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (it >= items) return;
    const int o = static_cast<int>(it % noct);
    int64_t x = it / noct;
    const int kv = static_cast<int>(x & 1);
    x >>= 1;                                    // (layer * B + sequence) * Hkv + head
    const int h = static_cast<int>(x % Hkv);
    const int b = static_cast<int>(x / Hkv % B), l = static_cast<int>(x / Hkv / B);
    const int st = __ldg(start + b);
    int t = __ldg(len + b);
    if (t < 0 || t > max_pages * kQ4Page || st < 0) {
        if (lane == 0) raise_error(err, SV_DEVERR_LENGTH);
        t = st < 0 ? 0 : max(0, min(t, max_pages * kQ4Page));
    }
    const int64_t q0 = static_cast<int64_t>(st & ~7) + 8 * o;   // the octet's first position
    uint16_t* out = (kv ? v_out : k_out) + x * n * static_cast<int64_t>(kQ4D) + d;
    const uint8_t* blk = nullptr;
    if (q0 >= 0 && q0 < t) {
        const int pg = __ldg(pages + static_cast<size_t>(b) * max_pages + q0 / kQ4Page);
        if (pg < 0 || pg >= num_pages) {
            if (lane == 0) raise_error(err, SV_DEVERR_PAGE);
        } else {
            blk = (kv ? v_pool : k_pool) + ((static_cast<size_t>(l) * num_pages + pg) * Hkv + h) * kQ4Bytes;
        }
    }
    const int slot = static_cast<int>(q0 & (kQ4Page - 1)), g = lane >> 3;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (blk && kv) w = __ldg(reinterpret_cast<const uint4*>(blk + q4_v_code_off(slot >> 3, d)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = q0 + i - st;
        if (r < 0 || r >= n) continue;
        uint2 y = make_uint2(0u, 0u);
        if (blk && q0 + i < t) {
            uint32_t c[4];
            uint16_t sb;
            if (kv) {
                const int sh = q4_shift(i);
                c[0] = w.x >> sh & 15u;
                c[1] = w.y >> sh & 15u;
                c[2] = w.z >> sh & 15u;
                c[3] = w.w >> sh & 15u;
                sb = __ldg(reinterpret_cast<const uint16_t*>(blk + q4_v_scale_off(g, slot + i)));
            } else {
                const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(blk + q4_k_code_off(g, slot + i) +
                                                                           4 * ((lane & 7) >> 1))) >> (8 * (lane & 1));
                c[0] = q & 15u;
                c[1] = q >> 16 & 15u;
                c[2] = q >> 4 & 15u;
                c[3] = q >> 20 & 15u;
                sb = __ldg(reinterpret_cast<const uint16_t*>(blk + q4_k_scale_off(g, slot + i)));
            }
            const float s = bf16_bits_f32(sb);
            y.x = pack_bf16x2((static_cast<int>(c[0]) - 8) * s, (static_cast<int>(c[1]) - 8) * s);
            y.y = pack_bf16x2((static_cast<int>(c[2]) - 8) * s, (static_cast<int>(c[3]) - 8) * s);
        }
        *reinterpret_cast<uint2*>(out + r * kQ4D) = y;
    }
}

unsigned int warp_grid(int64_t items) {
    return static_cast<unsigned int>((items + kThreads / 32 - 1) / (kThreads / 32));
}

}  // namespace

int64_t append_q4_items(int N, int B, int Hkv) { return (static_cast<int64_t>(N) / 8 + 2 * static_cast<int64_t>(B)) * 2 * Hkv; }

cudaError_t launch_append_q4(const AppendArgs& a, uint8_t* k_pool, uint8_t* v_pool, cudaStream_t st) {
    const int64_t items = append_q4_items(a.N, a.B, a.Hkv);
    return launch_pdl(append_q4_kernel, dim3(warp_grid(items)), dim3(kThreads), 0, st, a, k_pool, v_pool, items);
}

cudaError_t launch_commit_q4(uint8_t* k_pool, uint8_t* v_pool, const uint16_t* k_blk, const uint16_t* v_blk, int L,
                             int B, int Hkv, int R, const int32_t* path, const int32_t* n_acc, int32_t* len,
                             const int32_t* pages, int max_pages, int num_pages, cudaStream_t st) {
    return launch_pdl(commit_q4_kernel, dim3(B * kCluster), dim3(kThreads), 0, st, k_pool, v_pool, k_blk, v_blk, L, B,
                      Hkv, R, path, n_acc, len, pages, max_pages, num_pages, device_error_word());
}

int64_t gather_q4_items(int L, int B, int Hkv, int n) {
    return static_cast<int64_t>(L) * B * Hkv * 2 * ((static_cast<int64_t>(n) + 7) / 8 + 1);
}

cudaError_t launch_gather_q4(const uint8_t* k_pool, const uint8_t* v_pool, int L, int B, int Hkv, const int32_t* start,
                             const int32_t* len, int n, const int32_t* pages, int max_pages, int num_pages,
                             uint16_t* k_out, uint16_t* v_out, cudaStream_t st) {
    const int64_t items = gather_q4_items(L, B, Hkv, n);
    const int noct = (n + 7) / 8 + 1;
    return launch_pdl(gather_q4_kernel, dim3(warp_grid(items)), dim3(kThreads), 0, st, k_pool, v_pool, L, B, Hkv, start,
                      len, n, noct, pages, max_pages, num_pages, k_out, v_out, items, device_error_word());
}

}  // namespace sv
