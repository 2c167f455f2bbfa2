// kv_append.cuh -- what the append kernels share: where a new row goes.
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

}  // namespace sv
