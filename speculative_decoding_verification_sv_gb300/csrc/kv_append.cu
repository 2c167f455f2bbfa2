// kv_append.cu -- new rows of K and V into a paged bf16 cache, K rotated by
// its position on the way.
//
// A prompt, a prefill chunk or single decoded tokens: N rows of B sequences,
// sequence b's being rows row_off[b] .. row_off[b + 1], at the positions from
// len[b] on.  Pure movement: 1 KB read and 1 KB written per row and pair of KV
// heads, bound by HBM for prompts and by latency for single tokens.
#include "kv_append.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = 8;   // one warp finds one row's place
constexpr int kPage = 64;

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Work items of a row are 16-byte pieces: of each K head the rotated dims (half
// split: both pieces of a pair in one item), then the rest, then the pieces
// of V.
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a, uint16_t* __restrict__ k_pool,
                                                             uint16_t* __restrict__ v_pool) {
    __shared__ int64_t dst_s[kRowsPerCta];   // element offset of (page, head 0, position) in a pool; -1: no place
    __shared__ int pos_s[kRowsPerCta];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = blockIdx.x * kRowsPerCta;
    const int nrows = min(kRowsPerCta, a.N - row0);
    if (warp < nrows) {
        const int row = row0 + warp;
        const int b = warp_last_at_most(a.B, row, [&](int i) { return static_cast<int64_t>(__ldg(a.row_off + i)); });
        int64_t dst = -1;
        int pos = 0;
        if (b >= 0) {
            int r0, r1;
            if (!append_rows(a, b, r0, r1)) {
                if (lane == 0) raise_error(a.err, SV_DEVERR_ROWS);
            } else if (row >= r0 && row < r1) {
                const int t = __ldg(a.len + b);
                const int64_t p = static_cast<int64_t>(t) + (row - r0);
                if (t < 0 || p >= a.cap) {
                    if (lane == 0) raise_error(a.err, SV_DEVERR_LENGTH);
                } else {
                    pos = static_cast<int>(p);
                    const int pg = __ldg(a.pages + static_cast<size_t>(b) * a.max_pages + pos / kPage);
                    if (pg < 0 || pg >= a.num_pages) {
                        if (lane == 0) raise_error(a.err, SV_DEVERR_PAGE);
                    } else {
                        dst = (static_cast<int64_t>(pg) * a.Hkv * kPage + pos % kPage) * a.D;
                    }
                }
            }
        }
        if (lane == 0) {
            dst_s[warp] = dst;
            pos_s[warp] = pos;
        }
    }
    __syncthreads();
    const int rot = a.rope ? a.rot : 0, half = rot / 2;
    const int turned = a.interleaved ? rot / 8 : half / 8;     // rotated items of a head
    const int kper = turned + (a.D - rot) / 8, vper = a.D / 8;
    const int per_row = a.Hkv * (kper + vper);
    const int64_t head_stride = static_cast<int64_t>(kPage) * a.D;
    for (int it = threadIdx.x; it < nrows * per_row; it += kThreads) {
        const int r = it / per_row;
        int x = it % per_row;
        const int64_t d0 = dst_s[r];
        if (d0 < 0) continue;
        const int64_t row = row0 + r;
        if (x >= a.Hkv * kper) {   // V
            x -= a.Hkv * kper;
            const int h = x / vper, d = x % vper * 8;
            *reinterpret_cast<uint4*>(v_pool + d0 + h * head_stride + d) =
                __ldg(reinterpret_cast<const uint4*>(a.v + row * a.v_stride + h * a.D + d));
            continue;
        }
        const int h = x / kper, c = x % kper;
        const uint16_t* src = a.k + row * a.k_stride + h * a.D;
        uint16_t* dst = k_pool + d0 + h * head_stride;
        if (c >= turned) {         // dims past the rotated ones
            const int d = rot + (c - turned) * 8;
            *reinterpret_cast<uint4*>(dst + d) = __ldg(reinterpret_cast<const uint4*>(src + d));
            continue;
        }
        const float* cs = a.rope + static_cast<size_t>(pos_s[r]) * rot;
        if (a.interleaved) {
            const int d = c * 8;
            float v[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(src + d)), v);
            const float4 co = __ldg(reinterpret_cast<const float4*>(cs + d / 2));
            const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + d / 2));
            rope_turn(v[0], v[1], co.x, si.x);
            rope_turn(v[2], v[3], co.y, si.y);
            rope_turn(v[4], v[5], co.z, si.z);
            rope_turn(v[6], v[7], co.w, si.w);
            *reinterpret_cast<uint4*>(dst + d) = pack8(v);
        } else {
            const int d = c * 8;
            float v[8], w[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(src + d)), v);
            unpack8(__ldg(reinterpret_cast<const uint4*>(src + half + d)), w);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 co = __ldg(reinterpret_cast<const float4*>(cs + d + e));
                const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + d + e));
                rope_turn(v[e], w[e], co.x, si.x);
                rope_turn(v[e + 1], w[e + 1], co.y, si.y);
                rope_turn(v[e + 2], w[e + 2], co.z, si.z);
                rope_turn(v[e + 3], w[e + 3], co.w, si.w);
            }
            *reinterpret_cast<uint4*>(dst + d) = pack8(v);
            *reinterpret_cast<uint4*>(dst + half + d) = pack8(w);
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, uint16_t* k_pool, uint16_t* v_pool, cudaStream_t st) {
    return launch_pdl(kv_append_kernel, dim3((a.N + kRowsPerCta - 1) / kRowsPerCta), dim3(kThreads), 0, st, a, k_pool,
                      v_pool);
}

}  // namespace sv
