// Device-side building blocks of the 4-bit key/value cache kernels.
//
// A tile is 32 slots of one key/value head, one contiguous block of
// 32 * (D + 8 * D / g) bytes (D channels, groups of g):
//   key codes    D/64 x [64 lanes][4 words]
//   value codes  D/64 x [64 lanes][4 words]
//   key parameters    [D/g][32 slots] (step | offset << 16, the activation type)
//   value parameters  [D/g][32 slots]
// The words are laid out so that one 16-byte load of lane l hands it matrix
// operands that need no data from another lane: with r = l % 16, b = l / 16,
// word w of a tile holds
//   keys:   channels 32 (w mod D/32) + 8b + 0..7 of slot 16 (w / (D/32)) + r
//           (the A operand of a 16x16x32 product over channels; channel
//           2 (n mod 4) + n / 4 in nibble n, so that the pairs of nibbles
//           (n, n + 4) which one mask extracts are neighbouring channels),
//   values: channel 16 w + r of the slots 4b + 0..3 and 16 + 4b + 0..3 (the A
//           operand of a product over slots whose B operand, the weights, then
//           is what the first product leaves in the same lane; slot
//           4b + n mod 4 + 16 (n / 4) in nibble n).
#pragma once

#include "kv4_launch.h"
#include "w4a16_device.hpp"

namespace w4a16 {

template <int D, int NG>
struct Tile {
    static constexpr int kCodes = 16 * D;               // bytes of the key (or value) codes
    static constexpr int kParams = 128 * NG;            // bytes of the key (or value) parameters
    static constexpr int kBytes = 2 * (kCodes + kParams);
    static constexpr int kGroup = D / NG;
};

// The tile of head h that holds slots 32 t .. 32 t + 31 of sequence b, or null.
template <int D, int NG>
__device__ __forceinline__ uint8_t *tile_at(const Kv4Cache &c, const int32_t *table, int stride, int b,
                                            int h, int t) {
    const int page = t / c.tiles_per_page;
    if (t < 0 || page >= stride) return nullptr;
    const int id = table[(int64_t)b * stride + page];
    if ((unsigned)id >= (unsigned)c.num_pages) return nullptr;
    const int in = t - page * c.tiles_per_page;
    return c.pages + (((int64_t)id * c.kv_heads + h) * c.tiles_per_page + in) * Tile<D, NG>::kBytes;
}

// A parameter word: step in the low half, offset in the high half.
template <bool BF>
__device__ __forceinline__ float par_step(uint32_t p) { return lo_f32<BF>(p); }
template <bool BF>
__device__ __forceinline__ float par_offset(uint32_t p) { return hi_f32<BF>(p); }

// Word index of a key word: channels 8 i .. 8 i + 7 of slot r32.
template <int D>
__device__ __forceinline__ int key_word(int r32, int i) {
    const int w = (r32 >> 4) * (D / 32) + (i >> 2);
    return (w >> 2) * 256 + 4 * (16 * (i & 3) + (r32 & 15)) + (w & 3);
}

// Word index and shift of one value code.
__device__ __forceinline__ int value_word(int r32, int d) {
    return (d >> 6) * 256 + 4 * (16 * ((r32 & 15) >> 2) + (d & 15)) + ((d >> 4) & 3);
}
__device__ __forceinline__ int value_shift(int r32) { return 4 * ((r32 & 3) + 4 * (r32 >> 4)); }

// Masks of the nibble unpack, opaque to the compiler so that each pair of
// codes is at most one shift and one v_and_or_b32.
struct CodeConsts { uint32_t mask, one; };
template <bool BF>
__device__ __forceinline__ CodeConsts code_consts() {
    CodeConsts c = BF ? CodeConsts{0x000F000Fu, 0x43004300u} : CodeConsts{0x00F000F0u, 0x54005400u};
    asm volatile("" : "+v"(c.mask), "+v"(c.one));
    return c;
}

// The eight codes of a word as kCodeBase + c in the activation type, exactly:
// the four bits become mantissa bits of 64.0 (fp16) or 128.0 (bfloat16), the
// places that one of the four pairs of nibbles already has.  Dword i holds
// nibbles i and i + 4.
template <bool BF>
constexpr float kCodeBase = BF ? 128.0f : 64.0f;
template <bool BF>
__device__ __forceinline__ u4 based_codes(uint32_t w, const CodeConsts &c) {
    u4 r;
    if constexpr (BF) {
        r[0] = (w & c.mask) | c.one;
        r[1] = ((w >> 4) & c.mask) | c.one;
        r[2] = ((w >> 8) & c.mask) | c.one;
        r[3] = ((w >> 12) & c.mask) | c.one;
    } else {
        r[0] = ((w << 4) & c.mask) | c.one;
        r[1] = (w & c.mask) | c.one;
        r[2] = ((w >> 4) & c.mask) | c.one;
        r[3] = ((w >> 8) & c.mask) | c.one;
    }
    return r;
}

// v as three bfloat16 parts, v = part 0 + part 1 + part 2 to fp32's precision.
__device__ __forceinline__ float bf16_part(float v, int part) {
    const float a = round_act<true>(v);
    if (part == 0) return a;
    const float b = round_act<true>(v - a);
    return part == 1 ? b : round_act<true>(v - a - b);
}

// The slots that new token `i` of a sequence sees, [lo, hi): `start` is the slot of the first
// new one, and those from `len` on are not seen.
__device__ __forceinline__ int row_hi(int i, int start, int len, bool causal) {
    return causal ? min(len, start + i + 1) : len;
}
__device__ __forceinline__ int row_lo(int i, int start, int window) {
    return window > 0 ? max(0, start + i + 1 - window) : 0;
}

}  // namespace w4a16
