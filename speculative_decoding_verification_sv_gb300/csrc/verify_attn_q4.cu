// verify_attn_q4.cu -- attention of the k+1 verify rows over a 4-bit paged KV
// cache (format: kv_q4.cuh) and the block's own bf16 K/V.
//
// out = softmax(scale q K^T) V over the cached positions and the block rows
// that the row may see, as verify_attn.cu; the cache's bytes are 0.28 of the
// bf16 cache's.  One CTA per (sequence, head, row): 128 keys at a time, a
// thread a key for the scores and a dim for the values.
#include <math.h>

#include "kv_q4.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) attn_q4_kernel(AttnQ4Args a) {
    __shared__ float q_s[kQ4D], p_s[kThreads], red_s[4];
    pdl_wait();
    pdl_launch_dependents();
    const int j = blockIdx.x % a.R, h = blockIdx.x / a.R, b = blockIdx.y, g = h / a.G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int t = a.len[b];
    const int cap = a.max_pages * kQ4Page;
    if (t < 0 || t > cap) {
        if (tid == 0) raise_error(a.err, SV_DEVERR_LENGTH);
        t = t < 0 ? 0 : cap;
    }
    const size_t qo = ((static_cast<size_t>(b) * a.R + j) * a.Hq + h) * kQ4D + tid;
    q_s[tid] = bf16_bits_f32(a.q[qo]);
    // the row's path: bit i of anc set iff block row i is visible
    uint64_t anc[2] = {0ull, 0ull};
    if (a.parent) {
        const int32_t* par = a.parent + static_cast<size_t>(b) * a.R;
        int i = j;
        bool bad = false;
        for (int steps = 0; steps <= a.R && i >= 0; ++steps) {
            anc[i >> 6] |= 1ull << (i & 63);
            const int p = par[i];
            if ((i == 0 && p != -1) || (i > 0 && (p < 0 || p >= i))) {
                bad = true;
                break;
            }
            i = p;
        }
        if (bad) {
            if (tid == 0) raise_error(a.err, SV_DEVERR_TREE);
            anc[0] = j < 64 ? 1ull << j : 0ull;
            anc[1] = j >= 64 ? 1ull << (j - 64) : 0ull;
        }
    }
    __syncthreads();
    float m = -INFINITY, l = 0.f, o = 0.f;
    const size_t blk_row = (static_cast<size_t>(b) * a.Hkv + g) * a.R;
    for (int k0 = 0; k0 < t + a.R; k0 += kThreads) {
        const int key = k0 + tid;
        const int bi = key - t;   // block row, if >= 0
        float s = -INFINITY;
        auto block_of = [&](int p) -> const uint8_t* {
            const int pg = a.pages[static_cast<size_t>(b) * a.max_pages + p / kQ4Page];
            if (pg < 0 || pg >= a.num_pages) {
                raise_error(a.err, SV_DEVERR_PAGE);
                return nullptr;
            }
            return reinterpret_cast<const uint8_t*>((static_cast<size_t>(pg) * a.Hkv + g) * kQ4Bytes);
        };
        if (bi < 0) {
            const uint8_t* off = block_of(key);
            s = 0.f;
            const bool there = a.pages[static_cast<size_t>(b) * a.max_pages + key / kQ4Page] >= 0 &&
                               a.pages[static_cast<size_t>(b) * a.max_pages + key / kQ4Page] < a.num_pages;
            if (there) {
                const uint8_t* blk = a.k_pool + reinterpret_cast<size_t>(off);
                for (int gr = 0; gr < 4; ++gr) {
                    const float sc = bf16_bits_f32(
                        *reinterpret_cast<const uint16_t*>(blk + q4_k_scale_off(gr, key & 63)));
                    const uint32_t* w = reinterpret_cast<const uint32_t*>(blk + q4_k_code_off(gr, key & 63));
                    for (int d = 0; d < 32; ++d) {
                        const int c = static_cast<int>(w[d >> 3] >> q4_shift(d & 7) & 15u) - 8;
                        s = fmaf(q_s[gr * 32 + d], c * sc, s);
                    }
                }
            }
        } else if (bi < a.R && (a.parent ? (anc[bi >> 6] >> (bi & 63) & 1ull) != 0ull : bi <= j)) {
            s = 0.f;
            for (int d = 0; d < kQ4D; ++d) s = fmaf(q_s[d], bf16_bits_f32(a.k_blk[(blk_row + bi) * kQ4D + d]), s);
        }
        s *= a.scale_log2;
        float mt = s;
        for (int off = 16; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
        if (lane == 0) red_s[warp] = mt;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red_s[0], red_s[1]), fmaxf(red_s[2], red_s[3])));
        const float p = s == -INFINITY ? 0.f : exp2f(s - mn);
        p_s[tid] = p;
        const float c = m == -INFINITY ? 0.f : exp2f(m - mn);
        __syncthreads();
        float ps = 0.f;
        o *= c;
        for (int i = 0; i < kThreads; ++i) {
            const float pi = p_s[i];
            ps += pi;
            if (pi == 0.f) continue;
            const int ki = k0 + i;
            float v = 0.f;
            if (ki < t) {
                const int pg = a.pages[static_cast<size_t>(b) * a.max_pages + ki / kQ4Page];
                if (pg >= 0 && pg < a.num_pages) {
                    const uint8_t* blk = a.v_pool + (static_cast<size_t>(pg) * a.Hkv + g) * kQ4Bytes;
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + q4_v_code_off((ki & 63) >> 3, tid));
                    v = (static_cast<int>(w >> q4_shift(ki & 7) & 15u) - 8) *
                        bf16_bits_f32(*reinterpret_cast<const uint16_t*>(blk + q4_v_scale_off(tid >> 5, ki & 63)));
                }
            } else {
                v = bf16_bits_f32(a.v_blk[(blk_row + ki - t) * kQ4D + tid]);
            }
            o = fmaf(pi, v, o);
        }
        l = l * c + ps;
        m = mn;
        __syncthreads();
    }
    a.out[qo] = f32_bf16_bits(l > 0.f ? o / l : 0.f);
}

}  // namespace

size_t attn_q4_workspace(const sv_attn_shape&) { return 0; }

cudaError_t launch_verify_attn_q4(const AttnQ4Args& a, void*, cudaStream_t st) {
    return launch_pdl(attn_q4_kernel, dim3(a.Hq * a.R, a.B), dim3(kThreads), 0, st, a);
}

}  // namespace sv
