// kv_append.cuh -- what the append kernels share: where a new row goes, and its
// rotation.
#pragma once

#include <stdint.h>

#include "sv_device.cuh"

namespace sv {

struct AppendArgs {
    const uint16_t* k;         // [N] rows of [Hkv][D], row strides below
    const uint16_t* v;
    int64_t k_stride, v_stride;
    int N, B, Hkv, D;
    const int32_t* row_off;    // [B + 1]
    const int32_t* len;        // [B] position of each sequence's first new row
    const float* rope;         // [positions][rot]: cosines, then sines (nullptr: no rotation)
    int rot, cap;              // cap: positions the page table and the rope table both reach
    bool interleaved;
    const int32_t* pages;      // [B][max_pages]
    int max_pages, num_pages;
    unsigned int* err;
};

// Rows of sequence b, or false where the offsets do not name rows.
__device__ __forceinline__ bool append_rows(const AppendArgs& a, int b, int& r0, int& r1) {
    r0 = __ldg(a.row_off + b);
    r1 = __ldg(a.row_off + b + 1);
    return r0 >= 0 && r0 <= r1 && r1 <= a.N;
}

// Reports a sequence whose offsets do not name rows, thread i sequence i.  The
// search for a row's sequence need not meet it: blocks of their own look at all of
// them.
__device__ __forceinline__ void check_rows(const AppendArgs& a, uint32_t i) {
    int r0, r1;
    if (i < static_cast<uint32_t>(a.B) && !append_rows(a, static_cast<int>(i), r0, r1)) raise_error(a.err, SV_DEVERR_ROWS);
}

// The largest b in [0, B) with key(b) <= x, -1 where there is none; one warp,
// 32 probes a round.  With keys out of order some b is still returned.
template <typename F>
__device__ __forceinline__ int warp_last_at_most(int B, int64_t x, F&& key) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;
    while (true) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, i < n && key(lo + i) <= x);
        if (m == 0u) return -1;
        const int k = 31 - __clz(m);
        lo += k * step;
        n = min(step, n - k * step);
        if (step == 1) return lo;
    }
}

// One pair of a row turned by its position's angle; every product and sum is
// rounded to fp32 by itself, so the result is the same wherever it is formed.
__device__ __forceinline__ void rope_turn(float& x, float& y, float c, float s) {
    const float nx = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = nx;
}

__device__ __forceinline__ void unpack4(uint2 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// Turns the lane's four dims (4 lane .., packed bf16) of the rows of positions
// base + first .. base + last of kN rows of K and rounds them to bf16: the rows that
// the bf16 cache would hold.  cs is the table's row of position base.  Two rows'
// cosines and sines are on their way at a time (four took 104 bytes of spills).
template <bool kInterleaved, int kN>
__device__ __forceinline__ void turn_rows(uint2 (&x)[kN], int first, int last, const float* cs, int rot) {
    const int lane = threadIdx.x & 31, d = 4 * lane, half = rot / 2;
    const bool in = d < rot, lower = d < half;   // lower: the first member of its pair (halves)
    const int mate = !in ? lane : lower ? lane + half / 4 : lane - half / 4;
    const int f = !in ? 0 : kInterleaved ? d / 2 : lower ? d : d - half;
#pragma unroll
    for (int i0 = 0; i0 < kN; i0 += 2) {
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

}  // namespace sv
