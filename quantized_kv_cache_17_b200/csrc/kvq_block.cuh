// The fp8b pool format: E4M3 codes with one power-of-two scale for K and one
// for V per tile of 64 tokens of one KV head, and the device helpers that its
// append and its attention kernels share.
//
// Page block of one (layer, slot, KV head), 131,200 bytes: four tiles of 32,768
// bytes, then 32 bytes of scales, fp32 (K, V) of tile 0, of tile 1, ..., padded
// to 128.  A tile is [K codes 16,384 | V codes 16,384].  Both halves are what a
// kind::f8f6f4 tensor-core instruction takes as a K-major shared-memory operand,
// so a bulk copy of the bytes is all the staging they need:
//  K: rows = tokens, 128 dims a row, two dim halves; 8-row atoms of 1,024 bytes
//     with the 128-byte swizzle (16-byte chunk index XOR row in the atom).
//     token t, dim d at (d >> 7) * 8192 + (t >> 3) * 1024 + (t & 7) * 128 +
//     ((((d >> 4) & 7) ^ (t & 7)) << 4) + (d & 15)
//  V: rows = dims, 64 tokens a row; 8-row atoms of 512 bytes with the 64-byte
//     swizzle (chunk index XOR (row >> 1) & 3).
//     token t, dim d at (d >> 3) * 512 + (d & 7) * 64 +
//     (((t >> 4) ^ ((d >> 1) & 3)) << 4) + (t & 15)
//
// Why E4M3 with powers of two: one scale serves 64 x 256 values, so it sets the
// range only and the codes carry the relative precision; and when a later token
// raises a tile's scale, the codes already there are divided by a power of two,
// which is exact for every code that stays normal.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

constexpr int BT = 64;                        // tokens of a tile (one scale each for K and V)
constexpr int BT_PER_PAGE = PAGE / BT;
constexpr int BT_K_BYTES = BT * D;            // 16,384
constexpr int BT_BYTES = 2 * BT_K_BYTES;
constexpr int B_SCALES_OFF = BT_PER_PAGE * BT_BYTES;   // 131,072
constexpr int B_PAGE_BYTES = B_SCALES_OFF + 128;

// The smallest power of two d with amax <= 448 d, its exponent kept in
// [-120, 118] so that d and 448 d are normal fp32 numbers; 0 for amax = 0.
// 448 = 0.875 * 2^9, so with amax = m 2^x, m in [0.5, 1), the exponent is x - 9
// where m <= 0.875 and x - 8 above: read off the bits, exact.
__device__ __forceinline__ float block_scale(float amax) {
    if (!(amax > 0.0f)) return 0.0f;
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 126 - ((u & 0x7FFFFFu) <= 0x600000u ? 9 : 8);   // a subnormal amax ends at -120 all the same
    e = e < -120 ? -120 : (e > 118 ? 118 : e);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two values to two E4M3 bytes (lo in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four E4M3 bytes to two fp16 pairs, exact.  The halves of the word go to the
// conversions as they are: masked and shifted out one by one (e4m3x2_to_h2) they
// cost as many instructions as the conversions.
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ int block_k_off(int t, int d) {
    return (d >> 7) * 8192 + (t >> 3) * 1024 + (t & 7) * 128 + ((((d >> 4) & 7) ^ (t & 7)) << 4) + (d & 15);
}
__device__ __forceinline__ int block_v_off(int t, int d) {
    return (d >> 3) * 512 + (d & 7) * 64 + (((t >> 4) ^ ((d >> 1) & 3)) << 4) + (t & 15);
}

// The largest s in [0, n) with key(s) <= x, found by the whole warp, 32
// candidates a round; -1 when there is none.  Keys do not decrease over valid
// data; over any other data the result is still in range.
template <typename KEY> __device__ __forceinline__ int warp_find_last(int n, int64_t x, int lane, KEY key) {
    int lo = 0;
    bool first = true;
    while (n > 1 || first) {
        first = false;
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const bool in = i < n && key(lo + i) <= x;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (m == 0) return -1;
        const int top = 31 - __clz(m);
        lo += top * step;
        n = min(step, n - top * step);
    }
    return lo;
}

}  // namespace kvq
