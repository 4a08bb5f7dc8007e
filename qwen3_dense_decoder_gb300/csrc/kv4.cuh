// kv4.cuh -- the 4-bit K/V cache: its tiles and the packing of head rows.
//
// A head row (128 values) is packed by the weights' AFFINE4_GS32 rule ("Kipp
// Model Support", section "Quantization (AFFINE4_GS32)": 32 values a group,
// 4-bit codes, an fp16 scale and an fp16 bias) straight from FP32: bias =
// fp16(min), scale = fp16((max - min) / 15), code = round-half-even((x - bias)
// / scale) against the stored scale and bias, clamped to [0, 15]; a zero scale
// gives zero codes.  80 bytes a row against 256 in BF16 and 136 in Q8_0.  A
// stored value is fp16(scale * code + bias), rounded once.
//
// A pool tile is 32 positions of K or V of one KV head, KV4_TILE bytes: codes,
// then parameters.  The orders are those in which the decode attention's
// matrix fragments want them, so that every lane reads 16-byte words and one
// mask of a word gives an fp16 pair:
//  K  codes [position][group] 16 bytes: dimension i of a group in bits 4 i of
//     its 128 (the canonical order); (scale, bias) pairs [position][group].
//     A lane of K's fragment holds one group of a position.
//  V  codes [position pair][g < 8][group] words: the four dimensions 32 group
//     + 4 g + i of the even position in bits 4 i, of the odd one in bits
//     16 + 4 i, so a mask pairs two positions of one dimension, the order of
//     V's fragment; parameters [position pair][group] (scale even, scale odd,
//     bias even, bias odd).  A row still owns whole 16-bit words, so appending
//     a position is plain stores.
#pragma once

#include "common.cuh"

namespace q3 {

// Softmax weights enter the second product in fp16 as 2^(s - b), s the score in base 2
// and b a reference that lies KV4_BELOW under the largest score it was set from.  A
// score KV4_HIGH above b resets it, so weights stay under 2^15, and what rounds to
// nothing (under 2^-25) is 2^-32 of the largest weight: of n positions' sum at most n
// 2^-32 is lost, 2^-12 for a million.  (With b at the maximum 2^-25 was lost: 32,768
// positions 18 nats below one other, 2^-11 of the sum.)  b cancels in the quotient, and
// pieces with different b join as with different maxima.  Resetting costs prefill most:
// with b 11 below and so every growth by 2^4 instead of 2^8, scores four times as wide
// as unit rows give took 102.0 us instead of 96.9 (512 rows after 10,240 positions).
constexpr float KV4_BELOW = 7.0f, KV4_HIGH = 15.0f;

// |x| a packed row may hold: up to here no stored value passes the fp16 range
constexpr float KV4_MAX = 65000.0f;

// Eight values x of a group whose least and largest are lo and hi: their codes
// (value i in bits 4 i), the group's scale and bias, and the values the cache
// then holds, as fp16 pairs.  The rule divides by the scale and rounds; a
// product with the reciprocal is within 2^-18 of that quotient (below 16), so
// only where it lies within 2^-12 of a half does the division decide.
Q3_DEV uint32_t kv4_codes(const float (&x)[8], float lo, float hi, __half& scale, __half& bias, uint32_t (&val)[4]) {
    scale = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    bias = __float2half_rn(lo);
    const float s = __half2float(scale), b = __half2float(bias);
    const float inv = s != 0.0f ? __frcp_rn(s) : 0.0f;   // a zero scale gives zero codes
    float q[8];
    bool close = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float u = __fsub_rn(x[i], b) * inv;
        q[i] = rintf(u);
        close = close || fabsf(u - q[i]) > 0.5f - 0x1p-12f;
    }
    if (close && s != 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = rintf(__fdiv_rn(__fsub_rn(x[i], b), s));
    }
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = fminf(fmaxf(q[i], 0.0f), 15.0f);
        codes |= (uint32_t)q[i] << (4 * i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = __hfma2(__floats2half2_rn(q[2 * i], q[2 * i + 1]), __half2half2(scale), __half2half2(bias));
        val[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return codes;
}

// The fp16 pair 1024, 1024.  It reaches the kernels as an argument: known at
// compile time it costs kv4_pair a second logic operation (73 against 49 of the
// half-rate pipe's instructions for eight words).
constexpr uint32_t KV4_MAGIC = 0x64006400u;

// Nibble pair i of a code word (bits 4 i and 16 + 4 i) as fp16(scale * code +
// bias): an odd i keeps its place as 1024 + 16 code, so a word needs one shift.
// 1024 + code is exact in fp16, so are the code left by one exact operation and
// the fused multiply-add's argument; the last rounds once.  (Integers turned into
// fp16 by an exponent put over their bits: Kim, Henry, Fahim and Awadalla, "Who Says
// Elephants Can't Run", 2022.)
template <int I>
Q3_DEV uint32_t kv4_pair(uint32_t w, __half2 scale, __half2 bias, uint32_t magic) {
    const uint32_t x = I >= 2 ? w >> 8 : w;
    uint32_t v;                                          // x & mask | magic
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(x), "n"((I & 1) ? 0x00f000f0 : 0x000f000f), "r"(magic));
    const __half2 h = *reinterpret_cast<const __half2*>(&v);
    const __half2 c = (I & 1) ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-64.0f))
                              : __hsub2(h, __float2half2_rn(1024.0f));
    const __half2 r = __hfma2(c, scale, bias);
    return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace q3
