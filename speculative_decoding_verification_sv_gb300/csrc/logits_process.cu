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
// the same in any order).  The rest is movement, bound by HBM (4 bytes read and 4
// written an element; keys alone need no write): a warp takes 512 columns of a
// row at a time, and where a control touches some of them lays the row into shared
// memory, does the arithmetic above for the listed ones and takes the row back.
// 64 x 9 rows of 151936 with keys take 122 us (5.8 TB/s; the same movement without
// any control 108 us), 16 x 9 rows of 152064 with masks 41 us (29 us without any
// control: the history of each slice's CTA is not hidden in its first wave).
// What was slower there: the arithmetic in place for every group of 128 columns with a
// touched token (147 and 62 us, bound by instructions), the touched tokens done again
// after the pass (159 and 70 us: scattered words of rows that had left L2).
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 3;         // per SM
constexpr int kWarps = kThreads / 32;
constexpr int kMaxR = 128;
constexpr int kChunk = 512;      // columns a warp takes at a time: four slabs, eight lanes each
constexpr int kMaxSlice = 4096;

// A token's word: times generated in the low bits, and
constexpr uint32_t kPrompt = 1u << 31;   // it is in the prompt
constexpr uint32_t kBias = 1u << 30;     // it has a bias
constexpr uint32_t kBlock = 1u << 29;    // it is a token of the block
constexpr uint32_t kCount = kBlock - 1u;

// What the CTA knows of its slice, in dynamic shared memory: [slice] words,
// [slice] bias entries + 1 (with biases), each warp's row of a chunk, [slice]
// 16-bit places: the touched columns of every chunk, listed.
struct Slice {
    uint32_t* word;
    uint32_t* bias;
    int v0, width;
};

// Lane l holds columns 4 (l % 8) + 32 k + e, e < 4, of slab l / 8 of a chunk as
// x[4 k + e], k < 4: four loads of a lane lie 128 bytes apart, its mask bits are
// bits 4 (l % 8) + e of the slab's word k, and its columns ascend.

// Key of each slab over the columns in `take`, in its eight lanes; the general
// form.  c0: the lane's first column.
__device__ __forceinline__ uint64_t slab_key(const float (&x)[16], uint32_t take, int c0) {
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

// The same where no counted value is NaN: the slab's largest, then the lowest
// column of it.  Columns that do not count are -infinity.  Returns whether there
// was no NaN in the whole warp.
__device__ __forceinline__ bool slab_key_fast(const float (&x)[16], uint32_t take, int c0, uint64_t& key) {
    constexpr uint32_t kNone = 0x7fffffffu;
    float m = x[15];
#pragma unroll
    for (int i = 0; i < 14; i += 2) m = fmax3_nan(m, x[i], x[i + 1]);
    m = fmax3_nan(m, x[14], x[14]);
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, m, off);
        m = fmax3_nan(m, o, o);
    }
    uint32_t at = kNone;
#pragma unroll
    for (int i = 15; i >= 0; --i) at = x[i] == m ? static_cast<uint32_t>(c0 + 32 * (i >> 2) + (i & 3)) : at;
    if (!__all_sync(0xffffffffu, m > -INFINITY)) {
        if (__any_sync(0xffffffffu, m != m)) return false;
        // a slab of -infinity alone: its first column that counts
        if (m == -INFINITY) {
            const int i = __ffs(take) - 1;
            at = take ? static_cast<uint32_t>(c0 + 32 * (i >> 2) + (i & 3)) : kNone;
        }
    }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) at = min(at, __shfl_xor_sync(0xffffffffu, at, off));
    key = at == kNone ? 0ull : argmax_key(argmax_okey(m), static_cast<int>(at));
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
__global__ void __launch_bounds__(kThreads, kCtas) logits_kernel(LogitsArgs a, int slice) {
    extern __shared__ __align__(16) uint32_t words[];
    __shared__ int tok_s[kMaxR];
    __shared__ uint64_t anc_s[kMaxR][2];         // tree: the row's path as a bit mask
    __shared__ int touched_s[kMaxSlice / kChunk];
    pdl_wait();
    pdl_launch_dependents();
    // the sequences' first slices start first: token ids are numbered by how often
    // they occur, so those slices have the most to do
    const int b = blockIdx.x % a.B, si = blockIdx.x / a.B;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Slice sl;
    sl.v0 = si * slice;
    sl.width = min(a.V - sl.v0, slice);
    sl.word = words;
    sl.bias = words + slice;
    float* stage = reinterpret_cast<float*>(words + (a.bias_off ? 2 : 1) * slice) + warp * kChunk;
    uint16_t* lists = reinterpret_cast<uint16_t*>(words + (a.bias_off ? 2 : 1) * slice + kWarps * kChunk);
    const bool report = si == 0;         // one slice reports what every slice sees
    const bool counted = a.hist || a.tok || a.bias_off;

    const float* in = a.logits + static_cast<size_t>(b) * a.R * a.V;
    float* out = a.out ? a.out + static_cast<size_t>(b) * a.R * a.V : nullptr;
    const int nslab = (a.V + kArgmaxSlab - 1) / kArgmaxSlab, mwords = (a.V + 31) / 32;
    const uint32_t* mask = a.mask ? a.mask + static_cast<size_t>(b) * a.R * mwords : nullptr;
    uint64_t* keys = kKeys ? a.argmax + static_cast<size_t>(b) * a.R * nslab : nullptr;
    bool nan = false;

    // What the controls are is sent for at once: first the lengths and offsets ...
    float rep = 1.0f, freq = 0.0f, pres = 0.0f;
    int hl = 0, pl = 0, o0 = 0, o1 = 0, my_tok = -1;
    if (counted) {
        if (a.hist) hl = __ldg(a.hist_len + b);
        if (a.hist && a.prompt_len) pl = __ldg(a.prompt_len + b);
        if (a.bias_off) o0 = __ldg(a.bias_off + b), o1 = __ldg(a.bias_off + b + 1);
        if (a.tok && tid < a.R) my_tok = __ldg(a.tok + static_cast<size_t>(b) * a.R + tid);
    }
    if (a.rep) rep = __ldg(a.rep + b);
    if (a.freq) freq = __ldg(a.freq + b);
    if (a.pres) pres = __ldg(a.pres + b);

    // Warp items of the pass over the slice: a chunk of columns of a row, a chunk's
    // rows one after the other, so that the warps share the rows of a chunk with many
    // touched columns.  The next item's loads are on their way while one is worked on;
    // the first item's are sent for before the history.
    const int chunks = (sl.width + kChunk - 1) / kChunk;
    const int place = (lane >> 3) * kArgmaxSlab + 4 * (lane & 7);
    float x[16];
    uint32_t ok[4];
    auto load = [&](int item) {
        const int chunk = item / a.R, j = item - chunk * a.R, c0 = sl.v0 + chunk * kChunk + place;
        load_row<kVec>(in + static_cast<size_t>(j) * a.V + c0, c0, a.V, x);
        if (mask) {
            const uint32_t* m = mask + static_cast<size_t>(j) * mwords + (c0 >> 5);
#pragma unroll
            for (int k = 0; k < 4; ++k) ok[k] = c0 + 32 * k < a.V ? __ldg(m + k) >> (c0 & 31) : 0u;
        }
    };
    if (warp < chunks * a.R) load(warp);

    if (counted) {
        const int32_t* hist = a.hist + static_cast<size_t>(b) * a.hist_cap;
        const bool vec = (a.hist_cap & 3) == 0;   // rows start on 16 bytes
        constexpr int kSpan = 16 * kThreads;
        if (hl < 0 || hl > a.hist_cap) {
            if (report && tid == 0) raise_error(a.err, SV_DEVERR_LENGTH);
            hl = hl < 0 ? 0 : a.hist_cap;
        }
        if (o0 < 0 || o1 < o0 || o1 > a.n_bias) {
            if (report && tid == 0) raise_error(a.err, SV_DEVERR_ROWS);
            o0 = o1 = 0;
        }
        // ... then 16 history tokens of each thread and a bias, on their way while the
        // words are cleared
        int4 ahead[4];
        auto fetch = [&](int base) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = base + 4 * (tid + u * kThreads);
                ahead[u] = make_int4(-1, -1, -1, -1);
                if (i + 4 <= hl) ahead[u] = __ldg(reinterpret_cast<const int4*>(hist + i));
            }
        };
        if (vec) fetch(0);
        const int my_bias = o0 + tid < o1 ? __ldg(a.bias_tok + o0 + tid) : 0;
        const int clear = (a.bias_off ? 2 : 1) * slice / 4;
        for (int i = tid; i < clear; i += kThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        auto place_of = [&](int t) { return static_cast<uint32_t>(t) - static_cast<uint32_t>(sl.v0); };
        bool bad_tok = false;
        // token t of the block or of a bias
        auto mark = [&](int t, uint32_t bit) {
            bad_tok |= t < 0 || t >= a.V;
            if (place_of(t) < static_cast<uint32_t>(sl.width)) atomicOr(&sl.word[place_of(t)], bit);
        };
        if (a.tok && tid < a.R) {   // (R <= kThreads)
            tok_s[tid] = my_tok;
            mark(my_tok, kBlock);
            if (a.parent) {
                const int32_t* par = a.parent + static_cast<size_t>(b) * a.R;
                uint64_t m[2] = {0ull, 0ull};
                int i = tid;
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
                    m[0] = tid < 64 ? 1ull << tid : 0ull;
                    m[1] = tid >= 64 ? 1ull << (tid - 64) : 0ull;
                }
                anc_s[tid][0] = m[0];
                anc_s[tid][1] = m[1];
            }
        }
        auto said = [&](int i, int t) {
            const uint32_t r = place_of(t);
            if (r >= static_cast<uint32_t>(sl.width)) return;
            if (i < pl) atomicOr(&sl.word[r], kPrompt);
            else atomicAdd(&sl.word[r], 1u);
        };
        int done = 0;
        if (vec) {
            done = hl & ~3;
            for (int base = 0; base < done; base += kSpan) {
                // few of a thread's 16 are of this slice: found first, then taken one by one
                uint32_t here = 0u;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int t[4] = {ahead[u].x, ahead[u].y, ahead[u].z, ahead[u].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        here |= place_of(t[e]) < static_cast<uint32_t>(sl.width) ? 1u << (4 * u + e) : 0u;
                }
                if (__any_sync(0xffffffffu, __popc(here) > 4)) {   // (a slice of frequent tokens: most are)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int t[4] = {ahead[u].x, ahead[u].y, ahead[u].z, ahead[u].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (here >> (4 * u + e) & 1u) said(base + 4 * (tid + u * kThreads) + e, t[e]);
                    }
                    here = 0u;
                }
                if (report) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t last = max(max(static_cast<uint32_t>(ahead[u].x), static_cast<uint32_t>(ahead[u].y)),
                                                  max(static_cast<uint32_t>(ahead[u].z), static_cast<uint32_t>(ahead[u].w)));
                        if (base + 4 * (tid + u * kThreads) < done) bad_tok |= last >= static_cast<uint32_t>(a.V);
                    }
                }
                if (base + kSpan < done) fetch(base + kSpan);
                // (what was not fetched reads as -1, which is of no slice)
                for (; here != 0u; here &= here - 1u) {
                    const int k = __ffs(here) - 1, i = base + 4 * (tid + (k >> 2) * kThreads) + (k & 3);
                    said(i, __ldg(hist + i));
                }
            }
        }
        for (int i = done + tid; i < hl; i += kThreads) {
            const int t = __ldg(hist + i);
            bad_tok |= static_cast<uint32_t>(t) >= static_cast<uint32_t>(a.V);
            said(i, t);
        }
        for (int i = o0 + tid; i < o1; i += kThreads) {
            const int t = i == o0 + tid ? my_bias : __ldg(a.bias_tok + i);
            mark(t, kBias);
            // of a token named twice the later entry holds
            if (place_of(t) < static_cast<uint32_t>(sl.width)) atomicMax(&sl.bias[place_of(t)], static_cast<uint32_t>(i) + 1u);
        }
        if (bad_tok && report) raise_error(a.err, SV_DEVERR_TOKEN);
        __syncthreads();
        for (int chunk = warp; chunk < chunks; chunk += kWarps) {
            uint32_t hit = 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint4 w = *reinterpret_cast<const uint4*>(sl.word + chunk * kChunk + place + 32 * k);
                hit |= ((w.x ? 1u : 0u) | (w.y ? 2u : 0u) | (w.z ? 4u : 0u) | (w.w ? 8u : 0u)) << (4 * k);
            }
            int upto = __popc(hit);   // over this lane and those before it
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, upto, off);
                upto += lane >= off ? o : 0;
            }
            if (lane == 31) touched_s[chunk] = upto;
            uint16_t* list = lists + chunk * kChunk + (upto - __popc(hit));
            for (; hit != 0u; hit &= hit - 1u) {
                const int i = __ffs(hit) - 1;
                *list++ = static_cast<uint16_t>(place + 32 * (i >> 2) + (i & 3));
            }
        }
        __syncthreads();
    }

    bool bad_param = false;
    if (!(rep > 0.0f) || !isfinite(rep)) rep = 1.0f, bad_param = true;
    if (!isfinite(freq)) freq = 0.0f, bad_param = true;
    if (!isfinite(pres)) pres = 0.0f, bad_param = true;
    if (bad_param && report && tid == 0) raise_error(a.err, SV_DEVERR_PARAM);

    // column r of the slice in row j
    auto control = [&](float y, int j, int r) {
        const uint32_t w = sl.word[r];
        uint32_t c = w & kCount;
        if (w & kBlock) {   // times on row j's path
            for (int i = 0; i <= j; ++i) {
                const bool on = !a.parent || (anc_s[j][i >> 6] >> (i & 63) & 1ull) != 0ull;
                c += on && tok_s[i] == sl.v0 + r;
            }
        }
        if (c > 0u || (w & kPrompt)) y = y > 0.0f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
        if (c > 0u) y = __fsub_rn(__fsub_rn(y, __fmul_rn(freq, static_cast<float>(c))), pres);
        if (w & kBias) y = __fadd_rn(y, __ldg(a.bias_val + sl.bias[r] - 1u));
        return y;
    };

#pragma unroll 1
    for (int item = warp; item < chunks * a.R; item += kWarps) {
        const int chunk = item / a.R, j = item - chunk * a.R, r0 = chunk * kChunk, c0 = sl.v0 + r0 + place;
        const int touched = counted ? touched_s[chunk] : 0;
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = x[i];
        uint32_t allow[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) allow[k] = mask ? ok[k] : 0xFu;
        if (item + kWarps < chunks * a.R) load(item + kWarps);
        if (touched) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(stage + place + 32 * k) =
                    make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
            __syncwarp();
            const uint16_t* list = lists + r0;
            int i = lane;
            for (int whole = touched / 128; whole > 0; --whole, i += 128) {   // several at a time
                int c[4];
                float v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) c[u] = list[i + 32 * u];
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] = control(stage[c[u]], j, r0 + c[u]);
#pragma unroll
                for (int u = 0; u < 4; ++u) stage[c[u]] = v[u];
            }
            for (; i < touched; i += 32) {
                const int c = list[i];
                stage[c] = control(stage[c], j, r0 + c);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(stage + place + 32 * k);
                y[4 * k] = v.x, y[4 * k + 1] = v.y, y[4 * k + 2] = v.z, y[4 * k + 3] = v.w;
            }
        }
        if (mask) {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = allow[i >> 2] >> (i & 3) & 1u ? y[i] : a.mask_value;
        }
        if (out) store_row<kVec>(out + static_cast<size_t>(j) * a.V + c0, c0, a.V, y);
        if constexpr (kKeys) {
            uint64_t key = 0ull;
            uint32_t take = 0xFFFFu;   // columns that exist
            if (sl.v0 + r0 + kChunk > a.V) {
                take = 0u;
#pragma unroll
                for (int i = 0; i < 16; ++i) take |= c0 + 32 * (i >> 2) + (i & 3) < a.V ? 1u << i : 0u;
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = take >> i & 1u ? y[i] : -INFINITY;
            }
            if (!slab_key_fast(y, take, c0, key)) {
                key = slab_key(y, take, c0);
#pragma unroll
                for (int i = 0; i < 16; ++i) nan |= y[i] != y[i];
            }
            if ((lane & 7) == 0 && c0 < a.V) keys[static_cast<size_t>(j) * nslab + (c0 >> 7)] = key;
        }
    }
    if (nan) raise_error(a.err, SV_DEVERR_NONFINITE);
}

template <bool kVec, bool kKeys>
cudaError_t launch_logits(const LogitsArgs& a, int slice, size_t smem, cudaStream_t st) {
    static PerDeviceOnce once;
    const cudaError_t e = once.run([]() {
        return cudaFuncSetAttribute(logits_kernel<kVec, kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kMaxSlice * 10 + kWarps * kChunk * 4);
    });
    if (e != cudaSuccess) return e;
    const unsigned int ctas = static_cast<unsigned int>((a.V + slice - 1) / slice) * a.B;
    return launch_pdl(logits_kernel<kVec, kKeys>, dim3(ctas), dim3(kThreads), smem, st, a, slice);
}

}  // namespace

cudaError_t launch_logits_process(const LogitsArgs& a, cudaStream_t st) {
    // Slices of one to eight chunks.  A CTA spends on its controls about what a chunk
    // and a half take it, and the grid runs in waves of kCtas an SM: the slice with the
    // least whole waves x (chunks + 1.5).  (16 x 9 rows of 152064 under all controls:
    // 6 chunks, two waves, 41 us; 4 chunks, 2.6 waves, 44 us; 8 chunks, 1.3 waves, 47 us.)
    const int chunks = (a.V + kChunk - 1) / kChunk;
    int slice = kChunk;
    int64_t best = INT64_MAX;
    const int wave = kCtas * device_sm_count();
    for (int k = 1; k <= kMaxSlice / kChunk; ++k) {
        const int64_t ctas = static_cast<int64_t>((chunks + k - 1) / k) * a.B;
        const int64_t cost = (ctas + wave - 1) / wave * (2 * k + 3);
        if (cost < best) best = cost, slice = k * kChunk;
    }
    const bool counted = a.hist || a.tok || a.bias_off;
    const size_t smem = counted ? static_cast<size_t>(slice) * (a.bias_off ? 10 : 6) + kWarps * kChunk * 4 : 0;
    if (a.V % 4 == 0)
        return a.argmax ? launch_logits<true, true>(a, slice, smem, st) : launch_logits<true, false>(a, slice, smem, st);
    return a.argmax ? launch_logits<false, true>(a, slice, smem, st) : launch_logits<false, false>(a, slice, smem, st);
}

}  // namespace sv
