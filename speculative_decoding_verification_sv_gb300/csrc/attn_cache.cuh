// attn_cache.cuh -- what the attentions over the 4-bit and the 8-bit cache share: how
// the work is laid out over the CTAs, the walk over it, and the join of partial rows.
//
// A unit is one (sequence, KV head, tile of 64 query rows).  Either each unit has a
// cluster of CTAs, or the units' pages, and the block as one more, are laid end to end
// over all units and each CTA takes an equal run of them.
#pragma once

#include <math.h>
#include <stdint.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

constexpr int kHeadDim = 128;
constexpr int kPage = 64;                 // positions per page
constexpr int kRows = 64;                 // query rows of a tile
constexpr int kGrain = 4;                 // pages a CTA takes at least (where there are as many)

struct Work {
    int U;         // units of a sequence: Hkv * row tiles
    int row_tiles;
    int tile_rows; // rows of a tile but the last
    int cluster;   // CTAs of a unit where each unit has a cluster, 0 where the pages are split evenly
    int even;      // where more CTAs than this share the pages, a multiple of it do
    int inv_g;     // ceil(2^16 / G): r * inv_g >> 16 is r / G for every row r < 2048 of G <= 16
};

// Pages of sequence b (its length clamped into the table), the block not counted.
__device__ __forceinline__ int ctx_len(const CacheAttnArgs& a, int b) {
    const int t = a.len[b];
    return t < 0 ? 0 : min(t, a.max_pages * kPage);
}
__device__ __forceinline__ int ctx_pages(int t) { return (t + kPage - 1) / kPage; }

// Work of all sequences (sum of pages + 1), and of those before sequence
// `before`; one warp, every lane gets both.
__device__ __forceinline__ int2 work_sums(const CacheAttnArgs& a, int before) {
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
__device__ __forceinline__ int active_ctas(const Work& w, int W, int grid) {
    const int n = max(1, min(grid, W / kGrain));
    return n > w.even ? n - n % w.even : n;
}
// (n <= 2^15: products of remainders stay in 32 bits)
__device__ __forceinline__ int cta_first(int W, int i, int n) {
    const uint32_t q = static_cast<uint32_t>(W) / static_cast<uint32_t>(n), r = static_cast<uint32_t>(W) - q * n;
    return static_cast<int>(q * i + r * i / static_cast<uint32_t>(n));
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

    __device__ __forceinline__ void start(const CacheAttnArgs& a, const Work& w, int cta, int grid) {
        const int lane = threadIdx.x & 31;
        // (the first 32 lengths stay in registers: a round trip less for most batches)
        const int t0 = lane < a.B ? ctx_len(a, lane) : 0;
        const int w0 = lane < a.B ? (ctx_pages(t0) + 1) * w.U : 0;
        int W = w0;
        for (int i = 32 + lane; i < a.B; i += 32) W += (ctx_pages(ctx_len(a, i)) + 1) * w.U;
        W = __reduce_add_sync(0xffffffffu, W);
        const int n = active_ctas(w, W, grid);
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
        raw = a.len[b];
        bad_len = raw != t;
    }
    // Unit u's pages for CTA `rank` of the cluster that has the unit.
    __device__ __forceinline__ void start_unit(const CacheAttnArgs& a, const Work& w, int u, int rank) {
        b = u / w.U;
        unit = u - b * w.U;
        t = ctx_len(a, b);
        raw = a.len[b];
        bad_len = raw != t;
        np = ctx_pages(t);
        pos = off = cta_first(np + 1, rank, w.cluster);
        end = cta_first(np + 1, rank + 1, w.cluster);
    }
    __device__ __forceinline__ bool next(const CacheAttnArgs& a, const Work& w) {
        if (pos >= end) return false;
        if (fresh) {   // (the length was sent for when the run before began)
            t = max(0, min(raw, a.max_pages * kPage));
            bad_len = raw != t;
            np = ctx_pages(t);
            fresh = false;
        }
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
                raw = a.len[b];
                fresh = true;
            }
        }
        return true;
    }
    int raw;                           // length of sequence b as given
    bool fresh = false;                // which t and np do not follow yet
    bool bad_len = false;              // of the current run: the length was clamped
    int cur_b, cur_unit, cur_t;
    __device__ __forceinline__ void save(volatile int* to) const {
        to[0] = pos, to[1] = end, to[2] = b, to[3] = unit, to[4] = off;
    }
    __device__ __forceinline__ void load(const CacheAttnArgs& a, const volatile int* from) {
        pos = from[0], end = from[1], b = from[2], unit = from[3], off = from[4];
        fresh = true;
        raw = a.len[b];
    }
    __device__ __forceinline__ int ctx_steps() const { return (p1 - p0 + 1) / 2; }
};

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

__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What some partials of a row sum up to, a lane four dims of it: O, l, relative to m.
struct RowSum {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
};

// Up to kN partials of a row: get(i, ml, o) loads the i-th's (m, l) and the lane's four
// dims of its O: sums of P V, or, with kMeans, those over l.
template <int kN>
struct PartialRows {
    float2 ml[kN];
    float4 o[kN];
    template <typename Get>
    __device__ __forceinline__ void load(int n, Get&& get) {
#pragma unroll
        for (int u = 0; u < kN; ++u) {
            ml[u] = make_float2(-INFINITY, 0.f);
            o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (u < n) get(u, ml[u], o[u]);
        }
    }
    template <bool kMeans>
    __device__ __forceinline__ void add_to(RowSum& r) const {
        auto power = [](float x) { return kMeans ? fast_exp2(x) : exp2f(x); };
        // A mean weighs 2^m l, here the single power 2^(m + log2 l), of which the largest is 2^-8:
        // l can be large and a mean as large as V, so neither their product nor a sum of
        // 256 means may be formed.  (The difference of two m first, as m + log2 l rounds.)
        float lg[kN];
        float mn = r.m;
#pragma unroll
        for (int u = 0; u < kN; ++u) {
            lg[u] = kMeans ? fast_log2(ml[u].y) : 0.f;   // (-inf for 0)
            if constexpr (kMeans) mn = fmaxf(mn, ml[u].x + lg[u] + 8.0f);
            else if (ml[u].y != 0.f) mn = fmaxf(mn, ml[u].x);
        }
        const float c = r.m == -INFINITY ? 0.f : power(r.m - mn);
        r.o.x *= c, r.o.y *= c, r.o.z *= c, r.o.w *= c, r.l *= c;
#pragma unroll
        for (int u = 0; u < kN; ++u) {
            if (ml[u].y == 0.f) continue;   // all of the row's scores there are -inf
            const float w = power(kMeans ? (ml[u].x - mn) + lg[u] : ml[u].x - mn);
            r.l += kMeans ? w : w * ml[u].y;
            r.o.x += w * o[u].x;
            r.o.y += w * o[u].y;
            r.o.z += w * o[u].z;
            r.o.w += w * o[u].w;
        }
        r.m = mn;
    }
};

// Adds n partials of a row, eight in flight.
template <bool kMeans, typename Get>
__device__ __forceinline__ RowSum add_partials(int n, Get&& get) {
    RowSum r;
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += 8) {
        PartialRows<8> p;
        p.load(n - c0, [&](int u, float2& ml, float4& o) { get(c0 + u, ml, o); });
        p.template add_to<kMeans>(r);
    }
    return r;
}

__device__ __forceinline__ void store_row(const RowSum& r, uint16_t* dst) {
    const float inv = r.l != 0.f ? 1.0f / r.l : 0.f;
    *reinterpret_cast<uint2*>(dst + 4 * (threadIdx.x & 31)) =
        make_uint2(pack_bf16x2(r.o.x * inv, r.o.y * inv), pack_bf16x2(r.o.z * inv, r.o.w * inv));
}

template <bool kMeans, typename Get>
__device__ __forceinline__ void join_partials(int n, Get&& get, uint16_t* dst) {
    store_row(add_partials<kMeans>(n, get), dst);
}

inline Work work_of(int R, int G, int Hkv) {
    Work w{};
    const int rows = R * G;
    w.row_tiles = (rows + kRows - 1) / kRows;
    w.tile_rows = (rows + w.row_tiles - 1) / w.row_tiles;
    w.U = Hkv * w.row_tiles;
    w.even = 1;
    w.inv_g = (65536 + G - 1) / G;
    return w;
}

}  // namespace sv
