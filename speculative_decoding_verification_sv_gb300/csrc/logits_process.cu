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
// A CTA takes a slice of the vocabulary of one sequence and all its rows.  It
// counts the history's tokens of the slice in shared memory (integer atomics:
// the same in any order) and lists those that some control touches -- few.  The
// rest is movement, bound by HBM (4 bytes read and 4 written an element; keys
// alone need no write): logits pass through with the mask alone, and the listed
// tokens are then done again, one by one.  (With the controls in the stream the
// kernel was bound by its instructions, 223 for each 128 logits: 64 x 9 rows of
// 151936 took 229 us.)
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxR = 128;
constexpr int kChunk = 512;      // columns a warp takes at a time: four slabs, eight lanes each
constexpr int kMaxSlice = 4096;
constexpr int kBatch = 8;        // touched tokens a thread has in flight

// A token's word: times generated in the low bits, and
constexpr uint32_t kPrompt = 1u << 31;   // it is in the prompt
constexpr uint32_t kBias = 1u << 30;     // it has a bias
constexpr uint32_t kBlock = 1u << 29;    // it is a token of the block
constexpr uint32_t kCount = kBlock - 1u;

// What the CTA knows of its slice, in dynamic shared memory: [slice] words,
// [slice] bias entries + 1 (with biases), [slice] 16-bit places of the touched.
struct Slice {
    uint32_t* word;
    uint32_t* bias;
    uint16_t* list;
    int v0, width;
};

// Lane l holds columns 4 (l % 8) + 32 k + e, e < 4, of slab l / 8 of a chunk as
// x[4 k + e], k < 4: four loads of a lane lie 128 bytes apart, its mask bits are
// bits 4 (l % 8) + e of the slab's word k, and its columns ascend.

// Key of each slab over the columns in `take`, in its eight lanes; the general
// form.  c0: the lane's first column.
__device__ __noinline__ uint64_t slab_key(const float (&x)[16], uint32_t take, int c0) {
    uint64_t key = 0ull;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint64_t k = take >> i & 1u ? argmax_key(argmax_okey(x[i]), c0 + 32 * (i >> 2) + (i & 3)) : 0ull;
        key = k > key ? k : key;
    }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, key, off);
        key = o > key ? o : key;
    }
    return key;
}

// max(a, b, c), NaN if one is
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The same where no value is NaN and each slab has one above -infinity (those
// that do not count are -infinity): its largest, then the lowest column of it.
// Returns whether that held in the whole warp.
__device__ __forceinline__ bool slab_key_fast(const float (&x)[16], int c0, uint64_t& key) {
    float m = x[15];
#pragma unroll
    for (int i = 0; i < 14; i += 2) m = fmax3_nan(m, x[i], x[i + 1]);
    m = fmax3_nan(m, x[14], x[14]);
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, m, off);
        m = fmax3_nan(m, o, o);
    }
    if (!__all_sync(0xffffffffu, m > -INFINITY)) return false;
    uint32_t at = 0x7fffffffu;
#pragma unroll
    for (int i = 15; i >= 0; --i) at = x[i] == m ? 32u * (i >> 2) + (i & 3) : at;
    at += static_cast<uint32_t>(c0);
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) at = min(at, __shfl_xor_sync(0xffffffffu, at, off));
    key = argmax_key(argmax_okey(m), static_cast<int>(at));
    return true;
}

// The lane's 16 logits of a row, p its first column's place, c that column.
template <bool kVec>
__device__ __forceinline__ void load_row(const float* p, int c, int V, float (&x)[16]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (kVec) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + 32 * k < V) v = __ldcs(reinterpret_cast<const float4*>(p + 32 * k));
            x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * k + e] = c + 32 * k + e < V ? __ldcs(p + 32 * k + e) : 0.f;
        }
    }
}
template <bool kVec>
__device__ __forceinline__ void store_row(float* p, int c, int V, const float (&x)[16]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (kVec) {
            if (c + 32 * k < V)
                __stcs(reinterpret_cast<float4*>(p + 32 * k),
                       make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + 32 * k + e < V) __stcs(p + 32 * k + e, x[4 * k + e]);
        }
    }
}

template <bool kVec, bool kKeys>
__global__ void __launch_bounds__(kThreads, 3) logits_kernel(LogitsArgs a, int slice) {
    extern __shared__ __align__(16) uint32_t words[];
    __shared__ int tok_s[kMaxR];
    __shared__ uint64_t anc_s[kMaxR][2];         // tree: the row's path as a bit mask
    __shared__ int touched_s;
    pdl_wait();
    pdl_launch_dependents();
    // the sequences' first slices start first: token ids are numbered by how often
    // they occur, so those slices have the most touched tokens
    const int b = blockIdx.x % a.B, si = blockIdx.x / a.B;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Slice sl;
    sl.v0 = si * slice;
    sl.width = min(a.V - sl.v0, slice);
    sl.word = words;
    sl.bias = words + slice;
    sl.list = reinterpret_cast<uint16_t*>(words + (a.bias_off ? 2 : 1) * slice);
    const bool report = si == 0;         // one slice reports what every slice sees
    const bool counted = a.hist || a.tok || a.bias_off;

    if (counted) {
        // the first 16 history tokens of each thread are on their way while the
        // words are cleared
        const int32_t* hist = a.hist + static_cast<size_t>(b) * a.hist_cap;
        int hl = 0, pl = 0;
        const bool vec = (a.hist_cap & 3) == 0;   // rows start on 16 bytes
        int4 ahead[4];
        if (a.hist) {
            hl = __ldg(a.hist_len + b);
            if (hl < 0 || hl > a.hist_cap) {
                if (report && tid == 0) raise_error(a.err, SV_DEVERR_LENGTH);
                hl = hl < 0 ? 0 : a.hist_cap;
            }
            pl = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
            if (vec) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = 4 * (tid + u * kThreads);
                    if (i + 4 <= hl) ahead[u] = __ldg(reinterpret_cast<const int4*>(hist + i));
                }
            }
        }
        const int clear = (a.bias_off ? 2 : 1) * slice / 4;
        for (int i = tid; i < clear; i += kThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (tid == 0) touched_s = 0;
        __syncthreads();
        bool bad_tok = false;
        // marks token t: its word gets `bits` (added where they are a count), and a
        // place in the list the first time
        auto mark = [&](int t, uint32_t bits) {
            bad_tok |= t < 0 || t >= a.V;
            const uint32_t r = static_cast<uint32_t>(t) - static_cast<uint32_t>(sl.v0);
            if (r >= static_cast<uint32_t>(sl.width)) return;
            const uint32_t old = bits == 1u ? atomicAdd(&sl.word[r], 1u) : atomicOr(&sl.word[r], bits);
            if (old == 0u) sl.list[atomicAdd(&touched_s, 1)] = static_cast<uint16_t>(r);
        };
        if (a.tok) {
            for (int j = tid; j < a.R; j += kThreads) {
                const int t = __ldg(a.tok + static_cast<size_t>(b) * a.R + j);
                tok_s[j] = t;
                mark(t, kBlock);
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
            auto said = [&](int i, int t) { mark(t, i < pl ? kPrompt : 1u); };
            auto said4 = [&](int i, const int4& t) {
                said(i, t.x);
                said(i + 1, t.y);
                said(i + 2, t.z);
                said(i + 3, t.w);
            };
            int done = 0;
            if (vec) {
                done = hl & ~3;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = 4 * (tid + u * kThreads);
                    if (i + 4 <= hl) said4(i, ahead[u]);
                }
                for (int i = 4 * (tid + 4 * kThreads); i < done; i += 4 * kThreads)
                    said4(i, __ldg(reinterpret_cast<const int4*>(hist + i)));
            }
            for (int i = done + tid; i < hl; i += kThreads) said(i, __ldg(hist + i));
        }
        if (a.bias_off) {
            const int o0 = __ldg(a.bias_off + b), o1 = __ldg(a.bias_off + b + 1);
            if (o0 < 0 || o1 < o0 || o1 > a.n_bias) {
                if (report && tid == 0) raise_error(a.err, SV_DEVERR_ROWS);
            } else {
                for (int i = o0 + tid; i < o1; i += kThreads) {
                    const int t = __ldg(a.bias_tok + i);
                    mark(t, kBias);
                    // of a token named twice the later entry holds
                    if (t >= sl.v0 && t < sl.v0 + sl.width) atomicMax(&sl.bias[t - sl.v0], static_cast<uint32_t>(i) + 1u);
                }
            }
        }
        if (bad_tok && report) raise_error(a.err, SV_DEVERR_TOKEN);
        __syncthreads();
    }

    const float* in = a.logits + static_cast<size_t>(b) * a.R * a.V;
    float* out = a.out ? a.out + static_cast<size_t>(b) * a.R * a.V : nullptr;
    const int nslab = (a.V + kArgmaxSlab - 1) / kArgmaxSlab, mwords = (a.V + 31) / 32;
    const uint32_t* mask = a.mask ? a.mask + static_cast<size_t>(b) * a.R * mwords : nullptr;
    uint64_t* keys = kKeys ? a.argmax + static_cast<size_t>(b) * a.R * nslab : nullptr;
    bool nan = false;

    // every logit with the mask alone; the touched ones do not count for the keys
    // (warp items: a chunk of columns and a span of rows, the next row's loads on
    // their way while one is worked on; short slices split the rows)
    const int chunks = (sl.width + kChunk - 1) / kChunk;
    const int split = min(a.R, (kWarps + chunks - 1) / chunks), span = (a.R + split - 1) / split;
    const int place = (lane >> 3) * kArgmaxSlab + 4 * (lane & 7);
    for (int it = warp; it < chunks * split; it += kWarps) {
        const int r0 = it / split * kChunk + place, c0 = sl.v0 + r0;
        const int j0 = it % split * span, j1 = min(a.R, j0 + span);
        if (j0 >= j1) continue;
        const float* src = in + static_cast<size_t>(j0) * a.V + c0;
        const uint32_t* msrc = mask ? mask + static_cast<size_t>(j0) * mwords + (c0 >> 5) : nullptr;
        size_t at = static_cast<size_t>(j0) * a.V + c0;
        float x[16];
        uint32_t ok[4];
        auto load = [&]() {
            load_row<kVec>(src, c0, a.V, x);
            src += a.V;
            if (mask) {
#pragma unroll
                for (int k = 0; k < 4; ++k) ok[k] = c0 + 32 * k < a.V ? __ldg(msrc + k) >> (c0 & 31) : 0u;
                msrc += mwords;
            }
        };
        load();
        // columns that exist, and those of them that are touched
        uint32_t take = 0xFFFFu, hit = 0u;
        if constexpr (kKeys) {
            if (c0 + 100 > a.V) {
                take = 0u;
#pragma unroll
                for (int i = 0; i < 16; ++i) take |= c0 + 32 * (i >> 2) + (i & 3) < a.V ? 1u << i : 0u;
            }
            if (counted) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (r0 + 32 * k >= slice) break;
                    const uint4 w = *reinterpret_cast<const uint4*>(sl.word + r0 + 32 * k);
                    hit |= ((w.x ? 1u : 0u) | (w.y ? 2u : 0u) | (w.z ? 4u : 0u) | (w.w ? 8u : 0u)) << (4 * k);
                }
            }
        }
        const bool some = __any_sync(0xffffffffu, hit != 0u || take != 0xFFFFu);
#pragma unroll 1
        for (int j = j0; j < j1; ++j) {
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = x[i];
            uint32_t count = take & ~hit;
            if (mask) {
                uint32_t allowed = 0u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    allowed |= (ok[k] & 15u) << (4 * k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[4 * k + e] = ok[k] >> e & 1u ? y[4 * k + e] : a.mask_value;
                }
                count = take & ~(hit & allowed);
            }
            if (j + 1 < j1) load();
            if (out) store_row<kVec>(out + at, c0, a.V, y);
            at += a.V;
            if constexpr (kKeys) {
                uint64_t key = 0ull;
                if (some) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = count >> i & 1u ? y[i] : -INFINITY;
                }
                if (!slab_key_fast(y, c0, key)) {
                    key = slab_key(y, count, c0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) nan |= y[i] != y[i];
                }
                if ((lane & 7) == 0 && c0 < a.V) keys[static_cast<size_t>(j) * nslab + (c0 >> 7)] = key;
            }
        }
    }

    if (counted) {
        // the touched tokens, rows by rows
        float rep = a.rep ? __ldg(a.rep + b) : 1.0f, freq = a.freq ? __ldg(a.freq + b) : 0.0f;
        float pres = a.pres ? __ldg(a.pres + b) : 0.0f;
        bool bad_param = false;
        if (!(rep > 0.0f) || !isfinite(rep)) rep = 1.0f, bad_param = true;
        if (!isfinite(freq)) freq = 0.0f, bad_param = true;
        if (!isfinite(pres)) pres = 0.0f, bad_param = true;
        if (bad_param && report && tid == 0) raise_error(a.err, SV_DEVERR_PARAM);
        __syncthreads();   // the pass above has read (and written) the slice
        const uint32_t n = static_cast<uint32_t>(touched_s);
        // several at a time: each is a load from wherever the token lies
        const uint32_t items = n * a.R;
        for (uint32_t base = tid; base < items; base += kThreads * kBatch) {
            float x[kBatch];
            uint32_t r[kBatch];
            int j[kBatch];
            bool ok[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t it = base + u * kThreads;
                ok[u] = it < items;
                if (!ok[u]) continue;
                j[u] = static_cast<int>(it / n);
                r[u] = sl.list[it - static_cast<uint32_t>(j[u]) * n];
                const int v = sl.v0 + static_cast<int>(r[u]);
                if (mask) ok[u] = (__ldg(mask + static_cast<size_t>(j[u]) * mwords + (v >> 5)) >> (v & 31) & 1u) != 0u;
                // (in place: what the pass above wrote there is the logit itself)
                x[u] = in[static_cast<size_t>(j[u]) * a.V + v];
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (!ok[u]) continue;
                const uint32_t w = sl.word[r[u]];
                const int v = sl.v0 + static_cast<int>(r[u]);
                uint32_t c = w & kCount;
                if (w & kBlock) {   // times on row j's path
                    for (int i = 0; i <= j[u]; ++i) {
                        const bool on = !a.parent || (anc_s[j[u]][i >> 6] >> (i & 63) & 1ull) != 0ull;
                        c += on && tok_s[i] == v;
                    }
                }
                float y = x[u];
                if (c > 0 || (w & kPrompt)) y = y > 0.0f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
                if (c > 0) y = __fsub_rn(__fsub_rn(y, __fmul_rn(freq, static_cast<float>(c))), pres);
                if (w & kBias) y = __fadd_rn(y, __ldg(a.bias_val + sl.bias[r[u]] - 1u));
                if (out) out[static_cast<size_t>(j[u]) * a.V + v] = y;
                if constexpr (kKeys) {
                    nan |= y != y;
                    atomicMax(reinterpret_cast<unsigned long long*>(keys + static_cast<size_t>(j[u]) * nslab + (v >> 7)),
                              static_cast<unsigned long long>(argmax_key(argmax_okey(y), v)));
                }
            }
        }
    }
    if (nan) raise_error(a.err, SV_DEVERR_NONFINITE);
}

template <bool kVec, bool kKeys>
cudaError_t launch_logits(const LogitsArgs& a, int slice, size_t smem, cudaStream_t st) {
    static PerDeviceOnce once;
    const cudaError_t e = once.run([]() {
        return cudaFuncSetAttribute(logits_kernel<kVec, kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSlice * 10);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(logits_kernel<kVec, kKeys>, dim3(static_cast<unsigned int>((a.V + slice - 1) / slice) * a.B), dim3(kThreads), smem, st, a, slice);
}

}  // namespace

cudaError_t launch_logits_process(const LogitsArgs& a, cudaStream_t st) {
    // slices of whole chunks, about eight CTAs an SM where there is as much
    const int64_t want = (static_cast<int64_t>(a.V) * a.B / (8 * kSmCount) + kChunk - 1) / kChunk * kChunk;
    const int slice = static_cast<int>(want < kChunk ? kChunk : want > kMaxSlice ? kMaxSlice : want);
    const bool counted = a.hist || a.tok || a.bias_off;
    const size_t smem = counted ? static_cast<size_t>(slice) * (a.bias_off ? 10 : 6) : 0;
    if (a.V % 4 == 0)
        return a.argmax ? launch_logits<true, true>(a, slice, smem, st) : launch_logits<true, false>(a, slice, smem, st);
    return a.argmax ? launch_logits<false, true>(a, slice, smem, st) : launch_logits<false, false>(a, slice, smem, st);
}

}  // namespace sv
