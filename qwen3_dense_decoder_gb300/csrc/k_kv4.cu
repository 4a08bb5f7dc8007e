// k_kv4.cu -- the 4-bit K/V cache's writer and attention ("Kipp Roadmap",
// status v0.0.2: 32-position block tables; status v0.0.4: a quantized cache is
// opt-in).  The tile format is in kv4.cuh.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace q3 {

namespace {

namespace cg = cooperative_groups;

constexpr int D = 128;

template <typename K, typename A>
cudaError_t launch_ex(const Launch& L, K kern, dim3 grid, dim3 block, const A& args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.counter) ++*L.counter;
    return cudaLaunchKernelEx(&cfg, kern, args);
}

Q3_DEV __half2 as_h2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
Q3_DEV uint32_t as_u32(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }

Q3_DEV void report(int* status, int bits) { if (status) set_status(status, bits); }

// lane l's values [4l, 4l + 4) of a 128-value row, in FP32
Q3_DEV void load4(const float* p, int lane, float (&y)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p + lane * 4);
    y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
}
Q3_DEV void load4(const __half* p, int lane, float (&y)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p + lane * 4);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    y[0] = a.x; y[1] = a.y; y[2] = b.x; y[3] = b.y;
}
// ---------------------------------------------------------------- append
// Eight lanes take a head, so a warp four heads of a row: q heads are normed,
// rotated and stored in fp16; k heads are normed, rotated and packed, v heads
// packed, into the position's place of the row's block table.  Lane j of a head
// holds dimensions [8j, 8j + 8) and [64 + 8j, ..): both halves of its rotation
// pairs, and eight values each of groups j / 4 and 2 + j / 4, so a head costs
// three exchange steps for the norm, none for the rotation and two for a
// group's range, and the square root, the reciprocals and the divisions serve
// four heads at once.  A head's value costs about half an instruction (q) to
// one (k); the bytes are (n_q + 2 n_kv) 128 projections in, 2 bytes a q value
// and 0.625 a k or v value out.  2,048 rows of 48 heads in f32: 18.7 us, 4.2 TB/s
// of those bytes (a warp a head took 29.7), bound by the latency of a warp's one round
// of loads (4.4 of its stalls an issue are for them, at 31 % of DRAM and 39 % of the
// warps); 32 rows: 3.0 us, that chain alone.
Q3_DEV void load8(const float* p, float* y) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    y[0] = a.x; y[1] = a.y; y[2] = a.z; y[3] = a.w; y[4] = b.x; y[5] = b.y; y[6] = b.z; y[7] = b.w;
}
Q3_DEV void load8(const __half* p, float* y) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        y[2 * i] = f.x; y[2 * i + 1] = f.y;
    }
}
Q3_DEV void load8(const __nv_bfloat16* p, float* y) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { y[2 * i] = bf16lo(w[i]); y[2 * i + 1] = bf16hi(w[i]); }
}
Q3_DEV void store8(__half* p, const uint32_t (&h)[4]) { *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]); }

template <typename Tin>
__global__ void __launch_bounds__(128) kv4_append_kernel(const Kv4AppendArgs a)
{
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, j = lane & 7;
    const int n_heads = a.n_q + 2 * a.n_kv, chunks = (n_heads + 3) / 4;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int t = (int)(w / chunks), hh = (int)(w % chunks) * 4 + (lane >> 3);
    if (t >= a.T) return;
    const bool real = hh < n_heads;                      // a warp's last heads may not exist
    const bool is_q = hh < a.n_q, is_k = !is_q && hh < a.n_q + a.n_kv;
    const int kvh = is_k ? hh - a.n_q : hh - a.n_q - a.n_kv;
    const int pos = a.row_pos[t], slot = a.row_slot[t];

    float y[16];                                         // dimensions 8 j + e, then 64 + 8 j + e
    const size_t from = (size_t)t * a.qkv_stride + (size_t)(real ? hh : 0) * D + 8 * j;
    if (sizeof(Tin) == 4 && a.n_parts > 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = 0.f;
        for (int n = 0; n < a.n_parts; ++n) {
            const float* p = a.parts + (size_t)n * a.T * a.qkv_stride + from;
            float z[16];
            load8(p, z);
            load8(p + 64, z + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] += z[e];
        }
    } else {
        const Tin* p = static_cast<const Tin*>(a.qkv) + from;
        load8(p, y);
        load8(p + 64, y + 8);
    }
    const __nv_bfloat16* gain = (is_q ? a.q_gain : a.k_gain) + 8 * j;
    const uint4 g0 = *reinterpret_cast<const uint4*>(gain), g1 = *reinterpret_cast<const uint4*>(gain + 64);
    const bool live = pos >= 0 && pos < a.rope_len;      // else a padding row, or one past the rotation table
    float cs[16];
    {
        const float* rope = reinterpret_cast<const float*>(a.rope + (size_t)(live ? pos : 0) * (D / 2) + 8 * j);
        load8(rope, cs);
        load8(rope + 8, cs + 8);
    }
    int blk = -1;
    if (live && !is_q && real && slot >= 0 && slot < a.n_slots && pos / 32 < a.max_blocks)
        blk = a.tables[(size_t)slot * a.max_blocks + pos / 32];
    const bool placed = blk >= 0 && blk < a.n_blocks;
    if (real && j == 0 && pos >= 0 && (!live || (!is_q && !placed))) report(a.status, Q3_STATUS_BLOCK_RANGE);
    __half* dst = is_q ? (a.q_out ? a.q_out + ((size_t)t * a.n_q + hh) * D : nullptr)
                       : (a.kv_out ? a.kv_out + (((size_t)t * 2 + (is_k ? 0 : 1)) * a.n_kv + kvh) * D : nullptr);
    if (!real) dst = nullptr;
    if (!live) {                                         // the same for all of the warp's heads
        const uint32_t z[4] = {0, 0, 0, 0};
        if (dst) { store8(dst + 8 * j, z); store8(dst + 64 + 8 * j, z); }
        return;
    }

    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
    for (int o = 1; o <= 4; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (is_q || is_k) {
        float g[16];
        load8(reinterpret_cast<const __nv_bfloat16*>(&g0), g);
        load8(reinterpret_cast<const __nv_bfloat16*>(&g1), g + 8);
        const float r = 1.0f / sqrtf(ss / 128.0f + a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = y[e] * r * g[e];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float lo = y[e], hi = y[8 + e], c = cs[2 * e], sn = cs[2 * e + 1];
            y[e] = lo * c - hi * sn;
            y[8 + e] = hi * c + lo * sn;
        }
    }
    // the groups' ranges: this lane's eight values, then the four lanes'
    float lo[2], hi[2];
    bool number = true;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        lo[h] = hi[h] = y[8 * h];
#pragma unroll
        for (int e = 1; e < 8; ++e) { lo[h] = fminf(lo[h], y[8 * h + e]); hi[h] = fmaxf(hi[h], y[8 * h + e]); }
#pragma unroll
        for (int e = 0; e < 8; ++e) number = number && y[8 * h + e] == y[8 * h + e];
    }
    const float most = is_q ? 65504.0f : KV4_MAX;
    const bool bad = real && (!number || fmaxf(fmaxf(hi[0], hi[1]), -fminf(lo[0], lo[1])) > most);
    if (bad) report(a.status, Q3_STATUS_F16_RANGE);
    if (__all_sync(0xffffffffu, is_q)) {
        if (!dst) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = as_u32(__floats2half2_rn(y[8 * h + 2 * i], y[8 * h + 2 * i + 1]));
            store8(dst + 64 * h + 8 * j, v);
        }
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            lo[h] = fminf(lo[h], __shfl_xor_sync(0xffffffffu, lo[h], o));
            hi[h] = fmaxf(hi[h], __shfl_xor_sync(0xffffffffu, hi[h], o));
        }
    uint8_t* tile = placed ? a.kv + (((size_t)blk * 2 + (is_k ? 0 : 1)) * a.n_kv + kvh) * KV4_TILE : nullptr;
    const int p = pos % 32;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float(&x)[8] = *reinterpret_cast<const float(*)[8]>(y + 8 * h);
        uint32_t v[4];
        if (is_q) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = as_u32(__floats2half2_rn(x[2 * i], x[2 * i + 1]));
            if (dst) store8(dst + 64 * h + 8 * j, v);
            continue;
        }
        __half scale, bias;
        const uint32_t codes = kv4_codes(x, lo[h], hi[h], scale, bias, v);
        if (dst) store8(dst + 64 * h + 8 * j, v);
        if (!tile) continue;
        const int grp = 2 * h + j / 4;
        if (is_k) {
            *reinterpret_cast<uint32_t*>(tile + p * 64 + 32 * h + 4 * j) = codes;
            if (j % 4 == 0)
                *reinterpret_cast<__half2*>(tile + KV4_CODES + p * 16 + grp * 4) = __halves2half2(scale, bias);
        } else {
            uint8_t* word = tile + (p >> 1) * 128 + (j % 4) * 32 + grp * 4 + (p & 1) * 2;
            *reinterpret_cast<uint16_t*>(word) = (uint16_t)codes;
            *reinterpret_cast<uint16_t*>(word + 16) = (uint16_t)(codes >> 16);
            if (j % 4 == 0) {
                __half* par = reinterpret_cast<__half*>(tile + KV4_CODES + (p >> 1) * 32 + grp * 8);
                par[p & 1] = scale;
                par[2 + (p & 1)] = bias;
            }
        }
    }
}

// ---------------------------------------------------------------- decode attention
// One CTA per (row, KV head, split of its context), four warps.  A warp takes
// every fourth 32-position block of the split; lane 0 keeps the next blocks'
// tiles (5,120 bytes of K and V, contiguous as stored) on their way with bulk
// copies into the warp's own ring, so no barrier is shared between warps.
//
// Both products run on mma.sync m16n8k16 with the cache as the A operand, so
// its 4-bit words become fragments in registers (kv4_pair; 1.6 instructions a
// value) and never pass through shared memory again:
//   S^T = K Q^T   rows positions, columns heads.  The order of the 16
//                 dimensions of a step is free, so a lane takes its own group's
//                 32 dimensions in the order of their nibbles.
//   O^T += V^T P^T  rows dimensions (a lane's word pairs two positions), columns
//                 heads; the weights turn from the score fragment's layout into
//                 B fragments by 8 x 8 transposes.
// q and the weights enter as fp16 high and low parts (22 bits, the weights' no finer
// than 2^-32 of the largest; kv4.cuh).  Up to four
// heads the two parts are columns 2h and 2h + 1 of one tile (c0 + c1 is the
// result of one head in one lane); from five on the columns are eight heads and
// the parts two products into the same accumulators.  An fp16 q has no low
// part, so the wide form leaves its product out.
// Softmax is online in base 2; O and the sums are rescaled only when a score passes
// its reference by KV4_HIGH, 2^8 above the maximum that set it.
//
// Splits of a (row, KV head) are one cluster; warps merge in order through
// shared memory, CTAs in order through distributed shared memory.
//
// tcgen05 would want the expanded values in shared memory, 256 bytes where 80 come
// in, for at most eight columns.  8 rows of 16,384 positions (40/8 heads): 43 us, 3.9
// TB/s.  No unit is full then (FMA pipe 42 % of its cycles, ALU 33, tensor 27, DRAM 46,
// issue 51): a block is a chain of unpacking, products and exponentials, which the four
// warps a scheduler that 128 registers allow do not hide.  32 rows of 129 to 2,239
// (32/8): 20.4 us, the longest row's CTAs; one row of 2,176: 6.4 us, latency.
constexpr int AW = 4;
constexpr int STAGES = 2;
constexpr int KV4_STAGE = 2 * KV4_TILE;

Q3_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
Q3_DEV uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// mbar_wait by a whole warp, of one mind about the outcome (the products need all of
// its lanes), with an optional status word
Q3_DEV bool wait_bar(uint64_t* bar, uint32_t parity, int* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, global_ns() - t0 > Q3_WAIT_LIMIT_NS)) {
            report(status, Q3_STATUS_TIMEOUT);
            return false;
        }
    }
}

// 32 values [32 tig, 32 tig + 32) of a head's q as the B fragments of one
// column: registers 2 s, 2 s + 1 of step s; the high halves, or the rest
template <typename Tq>
Q3_DEV void load_q(const Tq* q, bool low, uint32_t (&b)[16], bool& bad) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float f[8];
        load4(q + 8 * j, 0, *reinterpret_cast<float (*)[4]>(f));
        load4(q + 8 * j + 4, 0, *reinterpret_cast<float (*)[4]>(f + 4));
        __half h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[e] = to_f16(f[e], bad);
            if (low) h[e] = __float2half_rn(f[e] - __half2float(h[e]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) b[4 * j + i] = as_u32(__halves2half2(h[i], h[i + 4]));
    }
}

// WIDE: a lane's score columns are heads 2 tig and 2 tig + 1; else head tig.
template <bool WIDE>
struct Attend {
    static constexpr int NH = WIDE ? 2 : 1;
    float m[NH], l[NH];        // the weights' reference (kv4.cuh) and this lane's part of the sum
    float o[8][4];             // O^T: row tile 2 g + h holds dimensions 32 g + 4 (lane / 4) + 2 h, + 1
};

// One block: kt, vt its K and V tiles in shared memory, n_pos its positions
// in use (TAIL: fewer than 32).  QP parts of q.
template <bool WIDE, int QP, bool TAIL>
Q3_DEV void attend_block(const uint8_t* kt, const uint8_t* vt, const uint32_t (&q)[QP][16], int n_pos, uint32_t magic, int lane,
                         Attend<WIDE>& w)
{
    constexpr int NH = Attend<WIDE>::NH;
    const int g = lane >> 2, tig = lane & 3;
    const float scale = 1.4426950408889634f * 0.08838834764831845f;    // log2(e) / sqrt(128)
    float s[NH][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
        const int p = 16 * mt + g;
        const uint4 ka = *reinterpret_cast<const uint4*>(kt + p * 64 + tig * 16);
        const uint4 kb = *reinterpret_cast<const uint4*>(kt + (p + 8) * 64 + tig * 16);
        const __half2 sa = *reinterpret_cast<const __half2*>(kt + KV4_CODES + p * 16 + tig * 4);
        const __half2 sb = *reinterpret_cast<const __half2*>(kt + KV4_CODES + (p + 8) * 16 + tig * 4);
        const __half2 sca = __low2half2(sa), bia = __high2half2(sa), scb = __low2half2(sb), bib = __high2half2(sb);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a0[4] = {kv4_pair<0>(wa[j], sca, bia, magic), kv4_pair<0>(wb[j], scb, bib, magic),
                                    kv4_pair<1>(wa[j], sca, bia, magic), kv4_pair<1>(wb[j], scb, bib, magic)};
#pragma unroll
            for (int i = 0; i < QP; ++i) mma_f16(c, a0, q[i][4 * j], q[i][4 * j + 1]);
            const uint32_t a1[4] = {kv4_pair<2>(wa[j], sca, bia, magic), kv4_pair<2>(wb[j], scb, bib, magic),
                                    kv4_pair<3>(wa[j], sca, bia, magic), kv4_pair<3>(wb[j], scb, bib, magic)};
#pragma unroll
            for (int i = 0; i < QP; ++i) mma_f16(c, a1, q[i][4 * j + 2], q[i][4 * j + 3]);
        }
        if (WIDE) {
            s[0][2 * mt] = c[0] * scale; s[NH - 1][2 * mt] = c[1] * scale;
            s[0][2 * mt + 1] = c[2] * scale; s[NH - 1][2 * mt + 1] = c[3] * scale;
        } else {
            s[0][2 * mt] = (c[0] + c[1]) * scale;
            s[0][2 * mt + 1] = (c[2] + c[3]) * scale;
        }
    }
    if (TAIL) {
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (8 * i + g >= n_pos) s[h][i] = -INFINITY;
    }
    float mx[NH];
    bool grow = false;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        mx[h] = fmaxf(fmaxf(s[h][0], s[h][1]), fmaxf(s[h][2], s[h][3]));
        grow = grow || mx[h] > w.m[h] + KV4_HIGH;
    }
    if (__any_sync(0xffffffffu, grow)) {                 // every lane of a head takes the head's reference
        float alpha[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], o));
            const float mn = fmaxf(w.m[h], mx[h] - KV4_BELOW);
            alpha[h] = fast_ex2(w.m[h] - mn);            // 0 at first
            w.m[h] = mn;
            w.l[h] *= alpha[h];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) w.o[i][e] *= alpha[WIDE ? (e & (NH - 1)) : 0];
    }
    // the weights' B fragments, 8 positions each: (high, low) of one head side
    // by side, or the high and the low parts of two heads
    uint32_t pt[NH][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float e[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            e[h] = fast_ex2(s[h][i] - w.m[h]);
            w.l[h] += e[h];
        }
        if (WIDE) {
            const __half2 hi = __floats2half2_rn(e[0], e[NH - 1]);
            const float2 f = __half22float2(hi);
            pt[0][i] = transpose8x8(as_u32(hi));
            pt[NH - 1][i] = transpose8x8(as_u32(__floats2half2_rn(e[0] - f.x, e[NH - 1] - f.y)));
        } else {
            const __half hi = __float2half_rn(e[0]);
            pt[0][i] = transpose8x8(as_u32(__halves2half2(hi, __float2half_rn(e[0] - __half2float(hi)))));
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int pa = 8 * j + tig, pb = pa + 4;         // position pairs
        const uint4 va = *reinterpret_cast<const uint4*>(vt + pa * 128 + g * 16);
        const uint4 vb = *reinterpret_cast<const uint4*>(vt + pb * 128 + g * 16);
        const uint4* para = reinterpret_cast<const uint4*>(vt + KV4_CODES + pa * 32);
        const uint4* parb = reinterpret_cast<const uint4*>(vt + KV4_CODES + pb * 32);
        const uint4 a01 = para[0], a23 = para[1], b01 = parb[0], b23 = parb[1];
        uint32_t sba[8] = {a01.x, a01.y, a01.z, a01.w, a23.x, a23.y, a23.z, a23.w};
        uint32_t sbb[8] = {b01.x, b01.y, b01.z, b01.w, b23.x, b23.y, b23.z, b23.w};
        if (TAIL) {            // positions past the end count as zeros, whatever is there
            const uint32_t ma = (2 * pa < n_pos ? 0xffffu : 0u) | (2 * pa + 1 < n_pos ? 0xffff0000u : 0u);
            const uint32_t mb = (2 * pb < n_pos ? 0xffffu : 0u) | (2 * pb + 1 < n_pos ? 0xffff0000u : 0u);
#pragma unroll
            for (int e = 0; e < 8; ++e) { sba[e] &= ma; sbb[e] &= mb; }
        }
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
        for (int gr = 0; gr < 4; ++gr) {
            const __half2 sca = as_h2(sba[2 * gr]), bia = as_h2(sba[2 * gr + 1]);
            const __half2 scb = as_h2(sbb[2 * gr]), bib = as_h2(sbb[2 * gr + 1]);
            const uint32_t a0[4] = {kv4_pair<0>(wa[gr], sca, bia, magic), kv4_pair<1>(wa[gr], sca, bia, magic),
                                    kv4_pair<0>(wb[gr], scb, bib, magic), kv4_pair<1>(wb[gr], scb, bib, magic)};
#pragma unroll
            for (int h = 0; h < NH; ++h) mma_f16(w.o[2 * gr], a0, pt[h][2 * j], pt[h][2 * j + 1]);
            const uint32_t a1[4] = {kv4_pair<2>(wa[gr], sca, bia, magic), kv4_pair<3>(wa[gr], sca, bia, magic),
                                    kv4_pair<2>(wb[gr], scb, bib, magic), kv4_pair<3>(wb[gr], scb, bib, magic)};
#pragma unroll
            for (int h = 0; h < NH; ++h) mma_f16(w.o[2 * gr + 1], a1, pt[h][2 * j], pt[h][2 * j + 1]);
        }
    }
}

constexpr int MAX_SPLITS = 16;
struct DecodeShared {
    union {
        uint8_t ring[AW][STAGES][KV4_STAGE];
        float o[AW][8][D];                 // per warp
    };
    uint64_t full[AW][STAGES];
    float m[AW][8], l[AW][8];              // per warp
    // what the cluster's CTAs leave here of the heads this one finishes: CTA c's
    // part of its n-th head in row n C + c; ceil(8 / C) C rows at most
    float in_o[MAX_SPLITS][D], in_m[MAX_SPLITS], in_l[MAX_SPLITS];
};
static_assert(sizeof(float) * 8 * D <= (size_t)STAGES * KV4_STAGE, "merge area");

template <bool WIDE, typename Tq>
__global__ void __launch_bounds__(AW * 32, 4) kv4_decode_kernel(const Kv4DecodeArgs a, int C)
{
    constexpr int NH = Attend<WIDE>::NH;
    constexpr int QP = WIDE && sizeof(Tq) == 4 ? 2 : 1;      // narrow: the parts are columns
    extern __shared__ __align__(128) uint8_t smem_raw[];
    DecodeShared& sm = *reinterpret_cast<DecodeShared*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int rank = blockIdx.x % C, unit = blockIdx.x / C;
    const int kvh = unit % a.n_kv, t = unit / a.n_kv;
    const int G = a.n_q / a.n_kv;
    if (lane < STAGES) mbar_init(&sm.full[warp][lane], 1);
    fence_barrier_init();
    __syncwarp();
    if (C > 1) cg::this_cluster().barrier_arrive();
    grid_dep_wait();

    const int slot = a.row_slot[t];
    int ctx = min(a.row_pos[t], 0x7ffffffe) + 1;
    if (ctx > 0 && (slot < 0 || slot >= a.n_slots || ctx > a.max_blocks * 32)) {
        if (rank == 0 && threadIdx.x == 0) report(a.status, Q3_STATUS_BLOCK_RANGE);
        ctx = 0;
    }
    const int nblk = max(ctx + 31, 0) / 32, per = (nblk + C - 1) / C;
    const int b1 = min((rank + 1) * per, nblk);
    const int* table = a.tables + (size_t)(ctx > 0 ? slot : 0) * a.max_blocks;
    const uint8_t* kv = a.kv + (size_t)kvh * KV4_TILE;

    // block b's tiles into stage st; false: its table entry is outside the pool
    auto issue = [&](int phys, int st) -> bool {
        const bool in_pool = (unsigned)phys < (unsigned)a.n_blocks;
        if (lane == 0 && !in_pool) {
            report(a.status, Q3_STATUS_BLOCK_RANGE);
            mbar_arrive(&sm.full[warp][st]);
        } else if (lane == 0) {
            const uint8_t* src = kv + (size_t)phys * 2 * a.n_kv * KV4_TILE;
            uint8_t* dst = sm.ring[warp][st];
            mbar_arrive_expect_tx(&sm.full[warp][st], KV4_STAGE);
            bulk_load(dst, src, KV4_TILE, &sm.full[warp][st]);
            bulk_load(dst + KV4_TILE, src + (size_t)a.n_kv * KV4_TILE, KV4_TILE, &sm.full[warp][st]);
        }
        return in_pool;
    };
    // the blocks of this warp, first, first + AW, ...: block n's tiles pass
    // through stage n % STAGES; one outside the pool leaves its stage as it
    // is and only ends the stage's phase
    const int first = rank * per + warp;
    uint32_t held = 0;                     // bit st: stage st's block is in the pool
#pragma unroll
    for (int st = 0; st < STAGES; ++st) {
        const int b = first + st * AW;
        if (b < b1 && issue(table[b], st)) held |= 1u << st;
    }

    uint32_t q[QP][16];
    bool bad = false;
    const Tq* qrow = static_cast<const Tq*>(a.q) + (size_t)t * a.q_stride + (size_t)kvh * G * D + 32 * tig;
    const int qh = WIDE ? g : g >> 1;                        // the head of this lane's column
#pragma unroll
    for (int i = 0; i < QP; ++i) {
        if (qh < G) {
            load_q(qrow + (size_t)qh * D, WIDE ? i == 1 : (g & 1) != 0, q[i], bad);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) q[i][e] = 0u;
        }
    }
    if (bad) report(a.status, Q3_STATUS_F16_RANGE);

    Attend<WIDE> w;
#pragma unroll
    for (int h = 0; h < NH; ++h) { w.m[h] = -INFINITY; w.l[h] = 0.f; }
#pragma unroll
    for (int i = 0; i < 8; ++i) w.o[i][0] = w.o[i][1] = w.o[i][2] = w.o[i][3] = 0.f;

    bool ok = true;
    uint32_t parity = 0;
    int b = first;
    for (int st = 0; b < b1; b += AW) {
        const int bn = b + STAGES * AW;
        const int phys = bn < b1 ? table[bn] : 0;        // ahead of its use below
        ok = wait_bar(&sm.full[warp][st], parity, a.status);
        if (!ok) break;
        if (held >> st & 1) {
            const uint8_t* kt = sm.ring[warp][st];
            const int n_pos = ctx - 32 * b;
            if (n_pos >= 32) attend_block<WIDE, QP, false>(kt, kt + KV4_TILE, q, 32, a.magic, lane, w);
            else attend_block<WIDE, QP, true>(kt, kt + KV4_TILE, q, n_pos, a.magic, lane, w);
        }
        __syncwarp();                                    // every lane is done with the stage
        if (bn < b1) held = (held & ~(1u << st)) | (uint32_t)issue(phys, st) << st;
        if (++st == STAGES) { st = 0; parity ^= 1; }
    }
    if (!ok)                                             // a wait ran out: leave no copy behind
        for (int n = (b - first) / AW; first + n * AW < min(b + STAGES * AW, b1); ++n)
            wait_bar(&sm.full[warp][n % STAGES], n / STAGES & 1, a.status);
    __syncthreads();                                     // the rings become the merge area

#pragma unroll
    for (int i = 0; i < NH; ++i) {
        const int h = WIDE ? 2 * tig + i : tig;
        float l = w.l[i];
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (h >= G) continue;
        // a sum that is no number is joined under an infinite reference, so it is none in every sum
        if (g == 0) { sm.m[warp][h] = l == l ? w.m[i] : INFINITY; sm.l[warp][h] = l; }
#pragma unroll
        for (int gr = 0; gr < 4; ++gr) {
            const float(&x)[4] = w.o[2 * gr];
            const float(&y)[4] = w.o[2 * gr + 1];
            *reinterpret_cast<float4*>(&sm.o[warp][h][32 * gr + 4 * g]) =
                WIDE ? make_float4(x[i], x[2 + i], y[i], y[2 + i]) : make_float4(x[0] + x[1], x[2] + x[3], y[0] + y[1], y[2] + y[3]);
        }
    }
    __syncthreads();

    // the warps in order; thread d owns dimension d
    const int d = threadIdx.x;
    const size_t row = ((size_t)t * a.n_q + (size_t)kvh * G) * D + d;
    bad = false;
    auto put = [&](int h, float O, float L) {
        const float v = L == 0.f ? 0.f : O / L;          // nothing attended: zeros
        if (a.out_f32) static_cast<float*>(a.out)[row + (size_t)h * D] = v;
        else static_cast<__half*>(a.out)[row + (size_t)h * D] = to_f16(v, bad);
    };
    cg::cluster_group cluster = cg::this_cluster();
    if (C > 1) cluster.barrier_wait();                   // every CTA of the cluster has started
    for (int h = 0; h < G; ++h) {
        float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
        for (int i = 0; i < AW; ++i) M = fmaxf(M, sm.m[i][h]);
        if (M != -INFINITY) {
#pragma unroll
            for (int i = 0; i < AW; ++i) {
                const float e = fast_ex2(sm.m[i][h] - M);
                L = fmaf(sm.l[i][h], e, L);
                O = fmaf(sm.o[i][h][d], e, O);
            }
        }
        if (C == 1) {
            put(h, O, L);
            continue;
        }
        // CTA h % C finishes head h
        const int at = h / C * C + rank;
        *cluster.map_shared_rank(&sm.in_o[at][d], h % C) = O;
        if (d == 0) {
            *cluster.map_shared_rank(&sm.in_m[at], h % C) = M;
            *cluster.map_shared_rank(&sm.in_l[at], h % C) = L;
        }
    }
    if (C > 1) {
        cluster.sync();
        for (int h = rank; h < G; h += C) {
            const int at = h / C * C;
            float M = -INFINITY, L = 0.f, O = 0.f;
            for (int c = 0; c < C; ++c) M = fmaxf(M, sm.in_m[at + c]);
            if (M != -INFINITY)
                for (int c = 0; c < C; ++c) {
                    const float e = fast_ex2(sm.in_m[at + c] - M);
                    L = fmaf(sm.in_l[at + c], e, L);
                    O = fmaf(sm.in_o[at + c][d], e, O);
                }
            put(h, O, L);
        }
    }
    if (bad) report(a.status, Q3_STATUS_F16_RANGE);
}

// CTAs of a (row, KV head).  Four fit an SM (16 warps); the splits grow by twos
// while the grid still fits the SMs at once (608; a second wave costs more than
// idle SMs: 64 rows of 2,000 positions 38 us unsplit, 41 in two) and a CTA keeps
// two blocks (one row of 600 positions: 4.8 us in 8 splits, 5.9 in 4), four for
// 16, whose clusters leave some SMs out (4 rows of 1,000: 6.3 us in 8, 7.2 in
// 16; of 32,768: 44 in 8, 39 in 16).
int decode_splits(const Kv4DecodeArgs& a)
{
    const int64_t units = (int64_t)a.T * a.n_kv, blocks = (a.max_ctx + 31) / 32;
    int C = 1;
    while (C < MAX_SPLITS && units * 2 * C <= 4 * 152 && blocks >= (C < 8 ? 4 : 8) * C) C *= 2;
    return C;
}

template <bool WIDE, typename Tq>
cudaError_t launch_decode(const Launch& L, const Kv4DecodeArgs& a)
{
    constexpr auto kernel = kv4_decode_kernel<WIDE, Tq>;
    constexpr int smem = (int)sizeof(DecodeShared);
    const int C = decode_splits(a);
    static std::atomic<unsigned long long> attr_done{0}, wide_done{0};
    if (cudaError_t e = allow_smem_per_device(kernel, smem, attr_done)) return e;
    if (C > 8)
        if (cudaError_t e = allow_wide_clusters(kernel, wide_done)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T * a.n_kv * C);
    cfg.blockDim = dim3(AW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (L.counter) ++*L.counter;
    return cudaLaunchKernelEx(&cfg, kernel, a, C);
}

// ---------------------------------------------------------------- prefill: tile list and fp16 copy
// A prompt's attention reads every block once per query tile, so its blocks
// are expanded once, into an fp16 copy that the tcgen05 kernel (k_kv4_prefill.cu)
// fetches with TMA: 80 + 256 bytes a position and head against 512 flop a row
// and position.  A warp expands half a tile at a time, all its loads first: 4-byte
// code words in, 16-byte words out, both coalesced.  A V value that is not finite
// becomes zero, for a row's weight of a position that it does not attend is zero and the
// product with an infinity would not be; it is reported where a sequence's place holds
// it (places past a sequence's end hold whatever the pool holds).  K needs no such care:
// a score of a position that is not attended is replaced, whatever it is.
//
// CTA 0 lists the query tiles meanwhile.  Enough of them, longest context first: a
// counting sort by context in 1,024 classes (order within a class does not matter).
// Fewer stay in order, with the cost before each, for the attention kernel to cut.
// (Expansion behind the list, a quarter of a tile's loads at a time: 2,048 positions
// 4 us more, 10,752 10 us more.)
constexpr int XT = 256;
constexpr int CLASSES = 1024;

struct Seq {
    int row0, rows, skip, pos0, slot;      // rows without the skipped ones (negative positions), the first one's position
};
// Sequence i; rows 0 where it cannot be attended (then skip covers its rows)
Q3_DEV Seq seq_of(const Kv4PrefillArgs& a, int i, bool& bad) {
    Seq s;
    const int r0 = max(a.seq_rows[i], 0), n = max(min(a.seq_rows[i + 1], a.T) - r0, 0);
    const int pos = a.seq_pos[i];
    s.slot = a.seq_slot ? a.seq_slot[i] : i;
    s.skip = pos < 0 ? (int)min((int64_t)n, -(int64_t)pos) : 0;
    s.pos0 = max(pos, 0);
    bad = n > s.skip && (s.slot < 0 || s.slot >= a.n_slots || (int64_t)s.pos0 + (n - s.skip) > (int64_t)a.max_blocks * 32);
    if (bad) s.skip = n;
    s.rows = n - s.skip;
    s.row0 = r0 + s.skip;
    return s;
}

// Tiles in order and the cost before each (one warp)
Q3_DEV void plan_cuts(const Kv4PrefillArgs& a) {
    const int lane = threadIdx.x & 31;
    int n = 0, cost = 0;
    for (int i0 = 0; i0 < a.ns; i0 += 32) {
        bool b;
        Seq mine{};
        if (i0 + lane < a.ns) mine = seq_of(a, i0 + lane, b);
        for (unsigned some = __ballot_sync(0xffffffffu, mine.rows > 0); some; some &= some - 1) {
            const int from = __ffs(some) - 1;
            const int row0 = __shfl_sync(0xffffffffu, mine.row0, from), rows = __shfl_sync(0xffffffffu, mine.rows, from),
                      pos0 = __shfl_sync(0xffffffffu, mine.pos0, from), slot = __shfl_sync(0xffffffffu, mine.slot, from);
            for (int k0 = 0; k0 < rows; k0 += 32 * a.rows_per_tile) {
                const int k = k0 + lane * a.rows_per_tile, r = min(a.rows_per_tile, rows - k);
                const int own = r > 0 ? (pos0 + k + r - 1) / KV4_STEP + 1 + KV4_TILE_COST : 0;
                int x = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (r > 0) {
                    a.tiles[n + lane] = make_int4(row0 + k, slot, (pos0 + k) | ((r - 1) << 25), i0 + from);
                    a.starts[n + lane] = cost + x - own;
                }
                n += __popc(__ballot_sync(0xffffffffu, r > 0));
                cost += __shfl_sync(0xffffffffu, x, 31);
            }
        }
    }
    if (lane == 0) {
        a.n_tiles[0] = n;
        a.n_tiles[2] = cost;
    }
}

Q3_DEV void plan_tiles(const Kv4PrefillArgs& a) {
    __shared__ int s_most;
    __shared__ alignas(16) int s_at[CLASSES];
    __shared__ unsigned long long s_tiles, s_cost;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) { s_most = 0; s_tiles = 0; s_cost = 0; }
    for (int i = threadIdx.x; i < CLASSES; i += XT) s_at[i] = 0;
    for (int i = threadIdx.x; i < 8 * a.ctas; i += XT) a.come[i] = 0;
    __syncthreads();
    bool bad;
    for (int i = threadIdx.x; i < a.ns; i += XT) {
        const Seq s = seq_of(a, i, bad);
        if (bad) report(a.status, Q3_STATUS_BLOCK_RANGE);
        if (!s.rows) continue;
        atomicMax(&s_most, s.pos0 + s.rows);
        const int n = (s.rows - 1) / a.rows_per_tile + 1;
        atomicAdd(&s_tiles, (unsigned long long)n);
        atomicAdd(&s_cost, (unsigned long long)n * ((s.pos0 + (s.rows + a.rows_per_tile) / 2) / KV4_STEP + 1 + KV4_TILE_COST));
    }
    __syncthreads();
    // rows of more than one sequence: what does not fit the list is left out
    if (threadIdx.x == 0 && s_tiles > (unsigned long long)a.max_tiles) report(a.status, Q3_STATUS_BLOCK_RANGE);
    // cut where the longest CTA of whole tiles would take longer than a share and a join
    const unsigned long long items = s_tiles * a.n_kv, cost = s_cost * a.n_kv;
    const unsigned long long whole = items < KV4_CUT * a.ctas ? max((unsigned long long)(s_most - 1) / KV4_STEP + 1 + KV4_TILE_COST,
                                                                    (items + a.ctas - 1) / a.ctas * cost / max(items, 1ull))
                                                              : 0;
    if (s_tiles <= (unsigned long long)a.max_tiles && whole > max(cost / a.ctas, (unsigned long long)KV4_MIN_SHARE) + KV4_JOIN_COST) {
        if (warp == 0) plan_cuts(a);
    } else {
        const float per = (float)CLASSES / (float)(s_most + 1);
        auto each = [&](auto&& f) {                      // a warp a sequence, a lane a tile
            for (int i = warp; i < a.ns; i += XT / 32) {
                bool b;
                const Seq s = seq_of(a, i, b);
                for (int k = lane * a.rows_per_tile; k < s.rows; k += 32 * a.rows_per_tile) {
                    const int rows = min(a.rows_per_tile, s.rows - k);
                    const int last = s.pos0 + k + rows - 1;
                    f(CLASSES - 1 - min((int)((float)last * per), CLASSES - 1), make_int4(s.row0 + k, s.slot, (s.pos0 + k) | ((rows - 1) << 25), i));
                }
            }
        };
        each([&](int c, const int4&) { atomicAdd(&s_at[c], 1); });
        __syncthreads();
        // counts to first places: four classes a thread
        static_assert(CLASSES == 4 * XT, "classes");
        __shared__ int s_warp[XT / 32];
        int4 n = *reinterpret_cast<const int4*>(s_at + 4 * threadIdx.x);
        const int own = n.x + n.y + n.z + n.w;
        int x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        x -= own;
        int all = 0;
#pragma unroll
        for (int i = 0; i < XT / 32; ++i) {
            if (i < warp) x += s_warp[i];
            all += s_warp[i];
        }
        n = make_int4(x, x + n.x, x + n.x + n.y, x + n.x + n.y + n.z);
        *reinterpret_cast<int4*>(s_at + 4 * threadIdx.x) = n;
        if (threadIdx.x == 0) {
            a.n_tiles[0] = min(all, a.max_tiles);
            a.n_tiles[2] = 0;
        }
        __syncthreads();
        each([&](int c, const int4& t) {
            const int at = atomicAdd(&s_at[c], 1);
            if (at < a.max_tiles) a.tiles[at] = t;
        });
    }
    // rows that attend nothing
    for (int i = warp; i < a.ns; i += XT / 32) {
        const Seq s = seq_of(a, i, bad);
        uint4* dst = reinterpret_cast<uint4*>(a.out + (size_t)(s.row0 - s.skip) * a.n_q * D);
        for (int64_t k = lane; k < (int64_t)s.skip * a.n_q * (D / 8); k += 32) dst[k] = make_uint4(0, 0, 0, 0);
    }
}

// infinities and NaN of fp16 pairs become zeros; whether there were any
Q3_DEV bool make_finite(uint32_t& v) {
    const uint32_t was = v;
    if ((v & 0x7c00u) == 0x7c00u) v &= 0xffff0000u;
    if ((v & 0x7c000000u) == 0x7c000000u) v &= 0xffffu;
    return v != was;
}
Q3_DEV bool make_finite(uint4& v) {
    bool any = make_finite(v.x);
    any |= make_finite(v.y);
    any |= make_finite(v.z);
    return any | make_finite(v.w);
}

// 16 positions of a tile: codes and parameters at src, fp16 rows at dst
Q3_DEV void expand_k(const uint8_t* codes, const uint8_t* params, __half* dst, uint32_t magic, int lane) {
    const int c = lane & 15, p0 = lane >> 4;             // two positions a step, eight dimensions a lane
    uint32_t w[8], sb[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        w[k] = __ldg(reinterpret_cast<const uint32_t*>(codes + (2 * k + p0) * 64) + c);
        sb[k] = __ldg(reinterpret_cast<const uint32_t*>(params + (2 * k + p0) * 16) + (c >> 2));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const __half2 sc = __low2half2(as_h2(sb[k])), bi = __high2half2(as_h2(sb[k]));
        const uint32_t v0 = kv4_pair<0>(w[k], sc, bi, magic), v1 = kv4_pair<1>(w[k], sc, bi, magic), v2 = kv4_pair<2>(w[k], sc, bi, magic),
                       v3 = kv4_pair<3>(w[k], sc, bi, magic);
        const uint4 o = make_uint4(__byte_perm(v0, v1, 0x5410), __byte_perm(v2, v3, 0x5410), __byte_perm(v0, v1, 0x7632),
                                   __byte_perm(v2, v3, 0x7632));
        *reinterpret_cast<uint4*>(dst + (2 * k + p0) * D + c * 8) = o;
    }
}
// true if one of the first n_pos positions held a value that is not finite
Q3_DEV bool expand_v(const uint8_t* codes, const uint8_t* params, __half* dst, int n_pos, uint32_t magic, int lane) {
    bool lost = false;
    const int gr = (lane & 15) >> 2, m = lane & 3, pr0 = lane >> 4;      // two position pairs a step
    uint32_t w0[4], w1[4];
    uint2 sb[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int pr = 2 * k + pr0;
        w0[k] = __ldg(reinterpret_cast<const uint32_t*>(codes + pr * 128 + 2 * m * 16) + gr);
        w1[k] = __ldg(reinterpret_cast<const uint32_t*>(codes + pr * 128 + (2 * m + 1) * 16) + gr);
        sb[k] = __ldg(reinterpret_cast<const uint2*>(params + pr * 32) + gr);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int pr = 2 * k + pr0;
        const __half2 sc = as_h2(sb[k].x), bi = as_h2(sb[k].y);
        const uint32_t p0 = kv4_pair<0>(w0[k], sc, bi, magic), p1 = kv4_pair<1>(w0[k], sc, bi, magic), p2 = kv4_pair<2>(w0[k], sc, bi, magic),
                       p3 = kv4_pair<3>(w0[k], sc, bi, magic);
        const uint32_t r0 = kv4_pair<0>(w1[k], sc, bi, magic), r1 = kv4_pair<1>(w1[k], sc, bi, magic), r2 = kv4_pair<2>(w1[k], sc, bi, magic),
                       r3 = kv4_pair<3>(w1[k], sc, bi, magic);
        uint4 e = make_uint4(__byte_perm(p0, p1, 0x5410), __byte_perm(p2, p3, 0x5410), __byte_perm(r0, r1, 0x5410), __byte_perm(r2, r3, 0x5410));
        uint4 o = make_uint4(__byte_perm(p0, p1, 0x7632), __byte_perm(p2, p3, 0x7632), __byte_perm(r0, r1, 0x7632), __byte_perm(r2, r3, 0x7632));
        // a group's values lie between its bias and 15 scale + bias: where both are finite, all are
        const __half2 top = __hfma2(sc, __float2half2_rn(15.0f), bi);
        if (((as_u32(bi) & 0x7c00u) == 0x7c00u) | ((as_u32(bi) & 0x7c000000u) == 0x7c000000u) | ((as_u32(top) & 0x7c00u) == 0x7c00u) |
            ((as_u32(top) & 0x7c000000u) == 0x7c000000u)) {
            lost |= make_finite(e) & (2 * pr < n_pos);
            lost |= make_finite(o) & (2 * pr + 1 < n_pos);
        }
        uint4* to = reinterpret_cast<uint4*>(dst + 2 * pr * D + 32 * gr + 8 * m);
        to[0] = e;
        to[D / 8] = o;
    }
    return lost;
}

__global__ void __launch_bounds__(XT) kv4_expand_kernel(const Kv4PrefillArgs a)
{
    grid_dep_launch();
    grid_dep_wait();
    if (blockIdx.x == 0) {
        plan_tiles(a);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t step = (int64_t)(gridDim.x - 1) * (XT / 32);
    int64_t u = (int64_t)(blockIdx.x - 1) * (XT / 32) + warp;    // half a tile: (block, K or V, KV head, half) of the sequences in turn
    int64_t base = 0;
    const int units = 4 * a.n_kv;
    for (int i0 = 0; i0 < a.ns; i0 += 32) {
        bool bad;
        Seq mine{};
        if (i0 + lane < a.ns) mine = seq_of(a, i0 + lane, bad);
        const int64_t own = mine.rows ? (int64_t)((mine.pos0 + mine.rows + 31) / 32) * units : 0;
        int64_t upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
        for (; u < base + all; u += step) {
            const int from = __popc(__ballot_sync(0xffffffffu, upto <= u - base));
            const int64_t rel = u - base - __shfl_sync(0xffffffffu, upto - own, from);
            const int slot = __shfl_sync(0xffffffffu, mine.slot, from), end = __shfl_sync(0xffffffffu, mine.pos0 + mine.rows, from);
            const int j = (int)(rel / units), part = (int)(rel - (int64_t)j * units) >> 1, half = (int)(rel & 1);
            const int phys = a.tables[(size_t)slot * a.max_blocks + j];
            if (phys < 0 || phys >= a.n_blocks) {                // the attention kernel leaves its places zero
                if (lane == 0) report(a.status, Q3_STATUS_BLOCK_RANGE);
                continue;
            }
            const uint8_t* src = a.kv + ((size_t)phys * 2 * a.n_kv + part) * KV4_TILE;
            __half* dst = a.copy + ((size_t)(a.by_seq ? (i0 + from) * a.max_blocks + j : phys) * 2 * a.n_kv + part) * (32 * D) + half * 16 * D;
            const int n_pos = end - 32 * j - 16 * half;
            if (part < a.n_kv) expand_k(src + half * 1024, src + KV4_CODES + half * 256, dst, a.magic, lane);
            else if (expand_v(src + half * 1024, src + KV4_CODES + half * 256, dst, n_pos, a.magic, lane)) report(a.status, Q3_STATUS_F16_RANGE);
        }
        base += all;
    }
}

}  // namespace

namespace {

template <typename Tin>
cudaError_t launch_append(const Launch& L, const Kv4AppendArgs& a)
{
    const int64_t warps = (int64_t)a.T * ((a.n_q + 2 * a.n_kv + 3) / 4);
    return launch_ex(L, kv4_append_kernel<Tin>, dim3((unsigned)((warps + 3) / 4)), dim3(128), a);
}

}  // namespace

cudaError_t launch_kv4_append(const Launch& L, const Kv4AppendArgs& a, int type)
{
    switch (type) {
    case Q3_TYPE_F32: return launch_append<float>(L, a);
    case Q3_TYPE_F16: return launch_append<__half>(L, a);
    default: return launch_append<__nv_bfloat16>(L, a);
    }
}

cudaError_t launch_kv4_decode(const Launch& L, const Kv4DecodeArgs& args, int q_type, int out_type)
{
    Kv4DecodeArgs a = args;
    a.magic = KV4_MAGIC;
    a.out_f32 = out_type == Q3_TYPE_F32;
    if (a.n_q / a.n_kv <= 4)
        return q_type == Q3_TYPE_F32 ? launch_decode<false, float>(L, a) : launch_decode<false, __half>(L, a);
    return q_type == Q3_TYPE_F32 ? launch_decode<true, float>(L, a) : launch_decode<true, __half>(L, a);
}

cudaError_t launch_kv4_expand(const Launch& L, const Kv4PrefillArgs& args)
{
    Kv4PrefillArgs a = args;
    a.magic = KV4_MAGIC;
    return launch_ex(L, kv4_expand_kernel, dim3(4 * 152), dim3(XT), a);
}

}  // namespace q3
