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

// |x| a packed row may hold: up to here no stored value passes the fp16 range
constexpr float KV4_MAX = 65000.0f;

// One head row held by a warp, lane l values [4l, 4l + 4): group b is lanes
// 8b .. 8b + 7.  Returns the lane's four codes (value 4l + i in bits 4 i), its
// group's scale and bias, and the values the cache then holds.  false in a
// lane whose values leave the range (or are not numbers).
Q3_DEV bool kv4_pack(const float (&y)[4], uint32_t& codes, __half& scale, __half& bias, __half (&val)[4]) {
    float lo = fminf(fminf(y[0], y[1]), fminf(y[2], y[3]));
    float hi = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
#pragma unroll
    for (int o = 1; o <= 4; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    scale = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    bias = __float2half_rn(lo);
    const float s = __half2float(scale), b = __half2float(bias);
    bool ok = true;
    codes = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        ok = ok && fabsf(y[e]) <= KV4_MAX;
        int q = 0;
        if (s != 0.0f) q = (int)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(y[e], b), s)), 0.0f), 15.0f);
        codes |= (uint32_t)q << (4 * e);
        val[e] = __hfma(scale, __int2half_rn(q), bias);
    }
    return ok;
}

// Store a packed row at position r of a pool tile.
Q3_DEV void kv4_store_k(uint8_t* tile, int r, uint32_t codes, __half scale, __half bias, int lane) {
    *reinterpret_cast<uint16_t*>(tile + r * 64 + lane * 2) = (uint16_t)codes;
    if ((lane & 7) == 0)
        *reinterpret_cast<__half2*>(tile + KV4_CODES + r * 16 + (lane >> 3) * 4) = __halves2half2(scale, bias);
}
Q3_DEV void kv4_store_v(uint8_t* tile, int r, uint32_t codes, __half scale, __half bias, int lane) {
    const int g = lane & 7, grp = lane >> 3;
    *reinterpret_cast<uint16_t*>(tile + (r >> 1) * 128 + g * 16 + grp * 4 + (r & 1) * 2) = (uint16_t)codes;
    if (g == 0) {
        __half* par = reinterpret_cast<__half*>(tile + KV4_CODES + (r >> 1) * 32 + grp * 8);
        par[r & 1] = scale;
        par[2 + (r & 1)] = bias;
    }
}

// The fp16 pair 1024, 1024.  It reaches the kernels as an argument: known at
// compile time it costs kv4_pair a second logic operation (73 against 49 of the
// half-rate pipe's instructions for eight words).
constexpr uint32_t KV4_MAGIC = 0x64006400u;

// Nibble pair i of a code word (bits 4 i and 16 + 4 i) as fp16(scale * code +
// bias): an odd i keeps its place as 1024 + 16 code, so a word needs one shift.
// 1024 + code is exact in fp16, so are the code left by one exact operation and
// the fused multiply-add's argument; the last rounds once.
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
