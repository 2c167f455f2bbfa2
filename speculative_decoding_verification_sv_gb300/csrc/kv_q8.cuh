// kv_q8.cuh -- the 8-bit paged KV cache: format and its conversions.
//
// Sixteen consecutive positions of one KV head (a run; D = 128 dims) share a scale
// s = 2^e; an element is an e4m3 code c (4 significant bits, steps of 2^-9 at least,
// at most 448) for the value c s.  128.25 bytes a row against 256 in bf16.  What the
// library writes has
//     e  the smallest in [-120, 119] with |x| <= 448 * 2^e for every finite row written
//        to the run since its first position last was;
//     c  x / s rounded to nearest even (past 448 s: 448).
// A scale is a power of two, so that a run whose later rows need a larger one has its
// earlier codes multiplied by a power of two, which is exact down to e4m3's smallest
// steps, and so that c s is exactly a bf16.  e4m3, because the tensor core multiplies it
// as it is: K goes from memory to the product without passing a register.
// A row that holds NaN or infinity is held as NaN throughout (all of its codes 0x7f)
// and has no part in the scale.
//
// One (page, head) is a block of 8320 bytes: 64 positions' codes, then four fp32
// scales, then 112 bytes that keep every block on a 128-byte line.
//   K: codes [64 positions][8 places][16 dims]; dims 16 c .. of position p lie at
//      place c ^ (p % 8): 8192 bytes that are, byte for byte, the 128-byte-swizzled
//      K-major tile that tcgen05.mma reads from shared memory.
//   V: codes [8 octets of positions][128 dims][8 positions]: a thread that holds a
//      dim reads eight positions at once, V transposed as the P V product wants it.
#pragma once

#include <stdint.h>

#include "sv_device.cuh"

namespace sv {

constexpr int kQ8D = 128;            // head dim
constexpr int kQ8Page = 64;          // positions per page
constexpr int kQ8Run = 16;           // positions per scale
constexpr int kQ8Bytes = 8320;       // one (page, head)
constexpr int kQ8Codes = 8192;       // its codes; the scales follow
constexpr int kQ8MinExp = -120, kQ8MaxExp = 119;

__host__ __device__ constexpr int q8_k_off(int pos, int chunk) { return pos * 128 + ((chunk ^ (pos & 7)) << 4); }
__host__ __device__ constexpr int q8_v_off(int octet, int dim) { return octet * 1024 + dim * 8; }
__host__ __device__ constexpr int q8_scale_off(int run) { return kQ8Codes + 4 * run; }

__device__ __forceinline__ float q8_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Exponent of the scale that holds magnitudes up to amax (finite, >= 0): 448 is 1.75 * 2^8.
__device__ __forceinline__ int q8_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x007fffffu) > 0x00600000u ? 1 : 0);
    return min(max(e, kQ8MinExp), kQ8MaxExp);
}

// Exponent of a stored scale; anything that this library does not write counts as
// the least (a pool of zeros holds zeros).
__device__ __forceinline__ int q8_stored_exponent(float s) {
    const uint32_t b = __float_as_uint(s);
    const int e = static_cast<int>(b >> 23) - 127;
    return (b & 0x007fffffu) == 0u && e >= kQ8MinExp && e <= kQ8MaxExp ? e : kQ8MinExp;
}

// codes of two values in units of the scale (lo in the low byte), rounded to nearest
// even, +-448 past that, NaN for NaN
__device__ __forceinline__ uint32_t q8_codes2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t q8_codes4(float a, float b, float c, float d) {
    return q8_codes2(a, b) | q8_codes2(c, d) << 16;
}

__device__ __forceinline__ void q8_values4(uint32_t w, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> 16 * i)));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
            : "r"(h));
    }
}

// four codes in units of 1 / f of theirs
__device__ __forceinline__ uint32_t q8_rescale4(uint32_t w, float f) {
    float x[4];
    q8_values4(w, x);
    return q8_codes4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}

// Two codes, the bytes kLo and kHi of the eight of (a, b), as a bf16 pair that is
// 2^-120 times their values (finite codes only): sign, exponent and fraction moved to
// where bf16 has them, whose exponent counts from 127 in place of 7.  A byte permute
// that also spreads the signs, a shift and a mask.
template <int kLo, int kHi>
__device__ __forceinline__ uint32_t q8_pair(uint32_t a, uint32_t b) {
    constexpr uint32_t sel = kLo | (kLo | 8) << 4 | kHi << 8 | (kHi | 8) << 12;
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "n"(sel));
    return (r << 4) & 0x87f087f0u;
}

__device__ __forceinline__ uint32_t q8_mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 2^e as a bf16 pair, -126 <= e <= 127
__device__ __forceinline__ uint32_t q8_pow2_pair(int e) { return static_cast<uint32_t>(e + 127) * 0x00800080u; }

// y, NaN where the code of pair p was NaN (0x7f: the pair holds 480 * 2^-120 there)
__device__ __forceinline__ uint32_t q8_nan_pair(uint32_t p, uint32_t y) {
    if ((p & 0x00007fffu) == 0x000007f0u) y |= 0x00007fc0u;
    if ((p & 0x7fff0000u) == 0x07f00000u) y |= 0x7fc00000u;
    return y;
}

}  // namespace sv
