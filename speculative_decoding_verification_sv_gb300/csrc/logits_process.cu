// logits_process.cu -- sampling controls on a verify block's logits:
// repetition, frequency and presence penalties, biases and grammar masks,
// between the LM head and the acceptance.
//
// In a verify block the controls differ row by row: a draft on the row's own
// path (the chain before it, or its ancestors in a tree) has been said when
// the row's token is drawn, so it counts as repeated there and not elsewhere.
// For row j of sequence b and token v, with n the times v occurs among the
// sequence's generated tokens and the row's path, in this order, each step
// rounded to fp32 by itself:
//     x = l > 0 ? l / rep : l * rep       if v is in the prompt or n > 0
//     x = x - freq * n - pres             if n > 0
//     x = x + bias                        if v has one
//     x = mask_value                      if the row's grammar forbids v
//
// One pass over the logits (4 bytes read and 4 written an element: HBM is the
// bound; keys alone need no write).  A CTA takes a slice of the vocabulary of
// one sequence and all its rows: it counts the history's tokens of the slice
// in shared memory once (integer atomics: the same in any order), and each
// lane keeps its four tokens' words in registers over the rows.  Almost every
// word is 0, and those logits only pass through.
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxR = 128;
constexpr int kUnroll = 4;   // rows a lane has in flight

// A token's word: times generated in the low bits, and
constexpr uint32_t kPrompt = 1u << 31;   // it is in the prompt
constexpr uint32_t kBias = 1u << 30;     // it has a bias
constexpr uint32_t kBlock = 1u << 29;    // it is a token of the block
constexpr uint32_t kCount = kBlock - 1u;

struct Penalties {
    float rep, freq, pres;
};

template <bool kVec>
__global__ void __launch_bounds__(kThreads) logits_kernel(LogitsArgs a, int slice) {
    extern __shared__ uint32_t words[];          // [slice], then [slice] bias entries + 1
    __shared__ int tok_s[kMaxR];
    __shared__ uint64_t anc_s[kMaxR][2];         // tree: the row's path as a bit mask
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.y, v0 = blockIdx.x * slice, v1 = min(a.V, v0 + slice);
    const int width = v1 - v0;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool report = blockIdx.x == 0;         // one slice reports what every slice sees
    uint32_t* bidx = words + slice;
    const bool counted = a.hist || a.tok || a.bias_off;

    Penalties pen{1.0f, 0.0f, 0.0f};
    if (a.rep) pen.rep = __ldg(a.rep + b);
    if (a.freq) pen.freq = __ldg(a.freq + b);
    if (a.pres) pen.pres = __ldg(a.pres + b);
    bool bad_pen = false;
    if (!(pen.rep > 0.0f) || !isfinite(pen.rep)) pen.rep = 1.0f, bad_pen = true;
    if (!isfinite(pen.freq)) pen.freq = 0.0f, bad_pen = true;
    if (!isfinite(pen.pres)) pen.pres = 0.0f, bad_pen = true;
    if (bad_pen && report && tid == 0) raise_error(a.err, SV_DEVERR_PARAM);

    if (counted) {
        for (int i = tid; i < (a.bias_off ? 2 : 1) * slice; i += kThreads) words[i] = 0u;
        __syncthreads();
        bool bad_tok = false;
        if (a.tok) {
            for (int j = tid; j < a.R; j += kThreads) {
                const int t = __ldg(a.tok + static_cast<size_t>(b) * a.R + j);
                tok_s[j] = t;
                bad_tok |= t < 0 || t >= a.V;
                if (t >= v0 && t < v1) atomicOr(&words[t - v0], kBlock);
            }
            if (a.parent) {
                const int32_t* par = a.parent + static_cast<size_t>(b) * a.R;
                for (int j = tid; j < a.R; j += kThreads) {
                    uint64_t m[2] = {0ull, 0ull};
                    int i = j;
                    bool bad = false;
                    for (int steps = 0; steps <= a.R && i >= 0; ++steps) {
                        if (i < 64) m[0] |= 1ull << i;
                        else m[1] |= 1ull << (i - 64);
                        const int p = __ldg(par + i);
                        if ((i == 0 && p != -1) || (i > 0 && (p < 0 || p >= i))) {
                            bad = true;
                            break;
                        }
                        i = p;
                    }
                    if (bad) {   // a malformed path is the row's own token
                        if (report) raise_error(a.err, SV_DEVERR_TREE);
                        m[0] = j < 64 ? 1ull << j : 0ull;
                        m[1] = j >= 64 ? 1ull << (j - 64) : 0ull;
                    }
                    anc_s[j][0] = m[0];
                    anc_s[j][1] = m[1];
                }
            }
        }
        if (a.hist) {
            int hl = __ldg(a.hist_len + b);
            if (hl < 0 || hl > a.hist_cap) {
                if (report && tid == 0) raise_error(a.err, SV_DEVERR_LENGTH);
                hl = hl < 0 ? 0 : a.hist_cap;
            }
            const int pl = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
            const int32_t* hist = a.hist + static_cast<size_t>(b) * a.hist_cap;
            auto count = [&](int i, int t) {
                const uint32_t r = static_cast<uint32_t>(t) - static_cast<uint32_t>(v0);
                if (r < static_cast<uint32_t>(width)) {
                    if (i < pl) atomicOr(&words[r], kPrompt);
                    else atomicAdd(&words[r], 1u);
                }
                bad_tok |= t < 0 || t >= a.V;
            };
            int i0 = 0;
            if ((a.hist_cap & 3) == 0) {   // rows start on 16 bytes
                i0 = hl & ~3;
                for (int i = 4 * tid; i < i0; i += 4 * kThreads) {
                    const int4 t = __ldg(reinterpret_cast<const int4*>(hist + i));
                    count(i, t.x);
                    count(i + 1, t.y);
                    count(i + 2, t.z);
                    count(i + 3, t.w);
                }
            }
            for (int i = i0 + tid; i < hl; i += kThreads) count(i, __ldg(hist + i));
        }
        if (a.bias_off) {
            const int o0 = __ldg(a.bias_off + b), o1 = __ldg(a.bias_off + b + 1);
            if (o0 < 0 || o1 < o0 || o1 > a.n_bias) {
                if (report && tid == 0) raise_error(a.err, SV_DEVERR_ROWS);
            } else {
                for (int i = o0 + tid; i < o1; i += kThreads) {
                    const int t = __ldg(a.bias_tok + i);
                    bad_tok |= t < 0 || t >= a.V;
                    if (t >= v0 && t < v1) {   // of a token named twice the later entry holds
                        atomicOr(&words[t - v0], kBias);
                        atomicMax(&bidx[t - v0], static_cast<uint32_t>(i) + 1u);
                    }
                }
            }
        }
        if (bad_tok && report) raise_error(a.err, SV_DEVERR_TOKEN);
        __syncthreads();
    }

    // times token v occurs on row j's path in the block
    auto on_path = [&](int j, int v) {
        uint32_t n = 0;
        if (a.parent) {
            for (int i = 0; i <= j; ++i)
                n += tok_s[i] == v && (anc_s[j][i >> 6] >> (i & 63) & 1ull) != 0ull;
        } else {
            for (int i = 0; i <= j; ++i) n += tok_s[i] == v;
        }
        return n;
    };
    auto apply = [&](float x, uint32_t w, int j, int v) {
        uint32_t n = w & kCount;
        if (w & kBlock) n += on_path(j, v);
        if (n > 0 || (w & kPrompt)) x = x > 0.0f ? __fdiv_rn(x, pen.rep) : __fmul_rn(x, pen.rep);
        if (n > 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(pen.freq, static_cast<float>(n))), pen.pres);
        if (w & kBias) x = __fadd_rn(x, __ldg(a.bias_val + bidx[v - v0] - 1u));
        return x;
    };

    const float* in = a.logits + static_cast<size_t>(b) * a.R * a.V;
    float* out = a.out ? a.out + static_cast<size_t>(b) * a.R * a.V : nullptr;
    const int nslab = (a.V + kArgmaxSlab - 1) / kArgmaxSlab, mwords = (a.V + 31) / 32;
    bool nan = false;
    for (int s = warp; s * kArgmaxSlab < width; s += kWarps) {   // 128 columns, four a lane
        const int r0 = s * kArgmaxSlab + 4 * lane, c0 = v0 + r0;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (counted) {
            const uint4 ww = *reinterpret_cast<const uint4*>(words + r0);
            w[0] = ww.x, w[1] = ww.y, w[2] = ww.z, w[3] = ww.w;
        }
        const bool any = (w[0] | w[1] | w[2] | w[3]) != 0u;
        for (int j0 = 0; j0 < a.R; j0 += kUnroll) {
            float x[kUnroll][4];
            uint32_t ok[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int j = j0 + u;
                ok[u] = 15u;
                if (j >= a.R) continue;
                const float* src = in + static_cast<size_t>(j) * a.V + c0;
                if constexpr (kVec) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c0 < a.V) v = __ldcs(reinterpret_cast<const float4*>(src));
                    x[u][0] = v.x, x[u][1] = v.y, x[u][2] = v.z, x[u][3] = v.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[u][e] = c0 + e < a.V ? __ldcs(src + e) : 0.f;
                }
                if (a.mask && c0 < a.V)
                    ok[u] = __ldg(a.mask + (static_cast<size_t>(b) * a.R + j) * mwords + (c0 >> 5)) >> (c0 & 31) & 15u;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int j = j0 + u;
                if (j >= a.R) break;
                if (any) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (w[e] != 0u) x[u][e] = apply(x[u][e], w[e], j, c0 + e);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(ok[u] >> e & 1u)) x[u][e] = a.mask_value;
                if (out) {
                    float* dst = out + static_cast<size_t>(j) * a.V + c0;
                    if constexpr (kVec) {
                        if (c0 < a.V) __stcs(reinterpret_cast<float4*>(dst), make_float4(x[u][0], x[u][1], x[u][2], x[u][3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (c0 + e < a.V) __stcs(dst + e, x[u][e]);
                    }
                }
                if (a.argmax) {
                    uint64_t key = 0ull;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (c0 + e >= a.V) continue;
                        nan |= x[u][e] != x[u][e];
                        const uint64_t k = argmax_key(argmax_okey(x[u][e]), c0 + e);
                        key = k > key ? k : key;
                    }
                    key = warp_max_key(key);
                    if (lane == 0) a.argmax[(static_cast<size_t>(b) * a.R + j) * nslab + (c0 >> 7)] = key;
                }
            }
        }
    }
    if (nan) raise_error(a.err, SV_DEVERR_NONFINITE);
}

}  // namespace

cudaError_t launch_logits_process(const LogitsArgs& a, cudaStream_t st) {
    // slices of 512 to 4096 tokens, about eight CTAs an SM
    int64_t want = (static_cast<int64_t>(a.V) * a.B / (8 * kSmCount) + kArgmaxSlab - 1) / kArgmaxSlab * kArgmaxSlab;
    const int slice = static_cast<int>(want < 512 ? 512 : want > 4096 ? 4096 : want);
    const bool counted = a.hist || a.tok || a.bias_off;
    const size_t smem = counted ? static_cast<size_t>(slice) * 4 * (a.bias_off ? 2 : 1) : 0;
    const dim3 grid((a.V + slice - 1) / slice, a.B);
    if (a.V % 4 == 0) return launch_pdl(logits_kernel<true>, grid, dim3(kThreads), smem, st, a, slice);
    return launch_pdl(logits_kernel<false>, grid, dim3(kThreads), smem, st, a, slice);
}

}  // namespace sv
