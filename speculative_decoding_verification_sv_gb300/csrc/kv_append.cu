// kv_append.cu -- new rows of K and V into a paged bf16 cache, K rotated by
// its position on the way.
//
// A prompt, a prefill chunk or single decoded tokens: N rows of B sequences,
// sequence b's being rows row_off[b] .. row_off[b + 1], at the positions from
// len[b] on.  Pure movement: 1 KB read and 1 KB written per row and pair of KV
// heads.  Held up by the chain of loads that finds a row's place (offsets, length,
// page), done for each row by itself, three rounds of warps an SM deep for a long
// prompt: 8 x 2048 rows of 4 heads take 14.1 us (4.5 TB/s), 64 single tokens 3.0 us.
// A row is sent for once it is known to be no padding (the first offset and the last one, a round trip that
// costs single tokens 0.3 us) and before its place is: sent for after that, the
// prompts took 16.1 us; with more warps an SM (48, for spills) 15.1 us; a thread a
// 16-byte piece in place of a warp a row 26 us.
#include "kv_append.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kThreads = 128;
constexpr int kPage = 64;
constexpr int kAhead = 4;   // 16-byte pieces of V a lane has in flight

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

// One warp a row, in 16-byte pieces.  K is turned by 16 bytes of the first half of
// a pair and 16 of the second (half split), or 16 bytes of pairs; then the dims that
// stay.
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a, uint16_t* __restrict__ k_pool,
                                                             uint16_t* __restrict__ v_pool) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t row_blocks = (a.N - 1) / (kThreads / 32) + 1;
    if (blockIdx.x >= row_blocks) {
        check_rows(a, (blockIdx.x - row_blocks) * kThreads + threadIdx.x);
        return;
    }
    const int row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= a.N) return;
    // padding is not read
    if (row < __ldg(a.row_off) || row >= __ldg(a.row_off + a.B)) return;
    // the row itself is sent for before its place is known
    const uint16_t* vrow = a.v + static_cast<int64_t>(row) * a.v_stride;
    const uint16_t* krow = a.k + static_cast<int64_t>(row) * a.k_stride;
    const int per = a.D / 8, pieces = a.Hkv * per;
    const int rot = a.rope ? a.rot : 0, half = rot / 2;
    const int turned = a.interleaved ? rot / 8 : half / 8, kper = turned + (a.D - rot) / 8;
    const bool split = !a.interleaved;   // a piece's pairs: 16 bytes here, 16 bytes half a rotation on
    uint4 v[kAhead], k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0;
    auto load_v = [&](int x0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (x0 + 32 * u < pieces) v[u] = __ldg(reinterpret_cast<const uint4*>(vrow) + x0 + 32 * u);
    };
    auto load_k = [&](int x) {
        if (x >= a.Hkv * kper) return;
        const int h = x / kper, c = x - h * kper;
        const uint16_t* src = krow + h * a.D + (c < turned ? c * 8 : rot + (c - turned) * 8);
        k0 = __ldg(reinterpret_cast<const uint4*>(src));
        if (split && c < turned) k1 = __ldg(reinterpret_cast<const uint4*>(src + half));
    };
    load_k(lane);
    load_v(lane);
    // the row's place: its sequence, position and page
    const int b = warp_last_at_most(a.B, row, [&](int i) { return static_cast<int64_t>(__ldg(a.row_off + i)); });
    if (b < 0) return;
    int r0, r1;
    if (!append_rows(a, b, r0, r1) || row < r0 || row >= r1) return;
    const int t = __ldg(a.len + b);
    const int64_t p = static_cast<int64_t>(t) + (row - r0);
    if (t < 0 || p >= a.cap) {
        if (lane == 0) raise_error(a.err, SV_DEVERR_LENGTH);
        return;
    }
    const int pos = static_cast<int>(p);
    const int pg = __ldg(a.pages + static_cast<size_t>(b) * a.max_pages + pos / kPage);
    if (pg < 0 || pg >= a.num_pages) {
        if (lane == 0) raise_error(a.err, SV_DEVERR_PAGE);
        return;
    }
    const int64_t head_stride = static_cast<int64_t>(kPage) * a.D;   // of a page
    const int64_t dst = (static_cast<int64_t>(pg) * a.Hkv * kPage + pos % kPage) * a.D;
    const float* cs = a.rope + static_cast<size_t>(pos) * rot;
    for (int x = lane; x < a.Hkv * kper; x += 32) {
        if (x != lane) load_k(x);
        const int h = x / kper, c = x - h * kper;
        const int d = c < turned ? c * 8 : rot + (c - turned) * 8;
        uint4* to = reinterpret_cast<uint4*>(k_pool + dst + h * head_stride + d);
        float y[8], z[8];
        if (c >= turned) {
            *to = k0;
        } else if (!split) {
            const float4 co = __ldg(reinterpret_cast<const float4*>(cs + d / 2));
            const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + d / 2));
            unpack8(k0, y);
            rope_turn(y[0], y[1], co.x, si.x);
            rope_turn(y[2], y[3], co.y, si.y);
            rope_turn(y[4], y[5], co.z, si.z);
            rope_turn(y[6], y[7], co.w, si.w);
            *to = pack8(y);
        } else {
            float4 co[2], si[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                co[e] = __ldg(reinterpret_cast<const float4*>(cs + d) + e);
                si[e] = __ldg(reinterpret_cast<const float4*>(cs + half + d) + e);
            }
            unpack8(k0, y);
            unpack8(k1, z);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rope_turn(y[4 * e], z[4 * e], co[e].x, si[e].x);
                rope_turn(y[4 * e + 1], z[4 * e + 1], co[e].y, si[e].y);
                rope_turn(y[4 * e + 2], z[4 * e + 2], co[e].z, si[e].z);
                rope_turn(y[4 * e + 3], z[4 * e + 3], co[e].w, si[e].w);
            }
            *to = pack8(y);
            *reinterpret_cast<uint4*>(k_pool + dst + h * head_stride + d + half) = pack8(z);
        }
    }
    for (int x0 = lane; x0 < pieces; x0 += 32 * kAhead) {
        if (x0 != lane) load_v(x0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int x = x0 + 32 * u;
            if (x >= pieces) continue;
            const int h = x / per;
            *reinterpret_cast<uint4*>(v_pool + dst + h * head_stride + (x - h * per) * 8) = v[u];
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, uint16_t* k_pool, uint16_t* v_pool, cudaStream_t st) {
    const uint32_t row_blocks = (a.N - 1) / (kThreads / 32) + 1, checks = (a.B - 1) / kThreads + 1;
    return launch_pdl(kv_append_kernel, dim3(row_blocks + checks), dim3(kThreads), 0, st, a, k_pool, v_pool);
}

}  // namespace sv
