// kv_q4.cuh -- the 4-bit paged KV cache: format and its conversions.
//
// A row (one position of one KV head, D = 128 dims) is four groups of 32
// consecutive dims; a group holds a bf16 scale s and 32 codes c in 0..15 for
// the values (c - 8) s.  4.5 bits an element, 72 bytes a row against 256 in
// bf16.  What the library writes has
//     s = amax / 7 rounded up to 4 significant bits, within [2^-100, 2^118]
//         (0 when amax = 0, NaN when the group holds NaN or infinity),
//     c = 8 + clamp(rint(x / s), -7, 7).
// Four significant bits, because then (c - 8) s has at most 8 and 136 s = 17 * 8 s
// at most 8 too: both are exactly bf16, so reading a value back never rounds
// and takes one bf16 fused multiply-add, (128 + c) s - 136 s, on a code that
// was or-ed into the low bits of bf16 128.  Rounding up keeps |x| <= 7 s, so
// |x - (c - 8) s| <= s / 2 (for amax up to 7 * 2^118).
//
// One (page, head) is a block of 4608 bytes, so a 64-key tile of K or V is one
// bulk copy.  Element e of the eight in a little-endian 32-bit word sits at
// bit 4 (e >> 1) + 16 (e & 1): shifts by 0, 4, 8 and 12 leave elements (0, 1),
// (2, 3), (4, 5), (6, 7) in the low nibbles of the word's halves.
//   K: codes [4 groups][64 positions][16 bytes: the group's 32 dims]; scales
//      [64 positions][4 groups].  A thread that holds a position reads 16 bytes
//      a group, neighbours next to it.
//   V: codes [8 octets of positions][128 dims][4 bytes: 8 positions of the
//      dim]; scales [4 groups][64 positions].  A thread that holds a dim reads
//      8 positions a word: V arrives transposed, as the P V product wants it.
#pragma once

#include <stdint.h>

#include "sv_device.cuh"

namespace sv {

constexpr int kQ4D = 128;             // head dim
constexpr int kQ4Page = 64;           // positions per page
constexpr int kQ4Bytes = 4608;        // one (page, head)
constexpr int kQ4ScaleOff = 4096;     // scales follow the codes
constexpr float kQ4MinScale = 0x1p-100f, kQ4MaxScale = 0x1p118f;

__host__ __device__ constexpr int q4_k_code_off(int group, int pos) { return group * 1024 + pos * 16; }
__host__ __device__ constexpr int q4_k_scale_off(int group, int pos) { return kQ4ScaleOff + pos * 8 + group * 2; }
__host__ __device__ constexpr int q4_v_code_off(int octet, int dim) { return octet * 512 + dim * 4; }
__host__ __device__ constexpr int q4_v_scale_off(int group, int pos) { return kQ4ScaleOff + group * 128 + pos * 2; }
__host__ __device__ constexpr int q4_shift(int e) { return 4 * (e >> 1) + 16 * (e & 1); }

// max(|a|, |b|) that is NaN if either is
__device__ __forceinline__ float q4_amax(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// scale of a group from its largest magnitude (NaN for NaN and infinity)
__device__ __forceinline__ float q4_scale(float amax) {
    if (!(amax < INFINITY)) return __int_as_float(0x7fc00000);
    if (amax == 0.0f) return 0.0f;
    const uint32_t up = (__float_as_uint(__fdiv_rn(amax, 7.0f)) + 0x000FFFFFu) & 0xFFF00000u;
    return fminf(fmaxf(__uint_as_float(up), kQ4MinScale), kQ4MaxScale);
}

// code of x given the group's scale s and rs = 1 / s rounded to nearest
// (0 when s is 0 or NaN: the code is then 8, the value 0 or NaN), on top of
// kQ4CodeBase.  x / s is Markstein's correction of x rs, which rounds as the
// division does wherever the quotient is not negligible; the clamped quotient
// plus 1.5 * 2^23 + 8 leaves 8 + rint above the bits of 1.5 * 2^23 (8 is even:
// ties still go to even). 
constexpr uint32_t kQ4CodeBase = 0x4B400000u;
__device__ __forceinline__ uint32_t q4_code(float x, float s, float rs) {
    const float q = __fmul_rn(x, rs);
    const float d = __fmaf_rn(__fmaf_rn(-q, s, x), rs, q);
    const float c = __fadd_rn(fminf(fmaxf(d, -7.0f), 7.0f), 12582920.0f);
    return rs == 0.0f ? kQ4CodeBase + 8u : __float_as_uint(c);
}
__device__ __forceinline__ float bf16_bits_f32(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ uint16_t f32_bf16_bits(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// Eight rows, four consecutive dims of each in a lane (dims 4 lane ..), eight
// lanes a group.  Every lane ends up with the scale of row lane & 7 of its
// group, so that the division and the reciprocal are done once a lane: a
// reduction that halves the rows a lane holds with every step.
__device__ __forceinline__ void q4_scales8(const float (&x)[8][4], float& s, float& rs) {
    const int lane = threadIdx.x & 31;
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = q4_amax(q4_amax(x[i][0], x[i][1]), q4_amax(x[i][2], x[i][3]));
#pragma unroll
    for (int half = 4; half > 0; half >>= 1) {
        const bool up = (lane & half) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + half], half);
            a[i] = q4_amax(up ? a[i + half] : a[i], other);
        }
    }
    s = q4_scale(a[0]);
    rs = s > 0.0f ? __frcp_rn(s) : 0.0f;
}

}  // namespace sv
