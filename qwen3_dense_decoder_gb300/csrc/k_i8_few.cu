// k_i8_few.cu -- out[t][m] = (sum_k x[t][k] w[m][k]) xs[t] ws[m] over 8-bit codes
// for few rows of x: bound by the bytes of w.
//
// The codes of w go from memory to registers, are expanded to fp16 there (three
// byte operations and two subtractions for four codes) and meet x's in mma.sync
// m16n8k16: 16 channels by 8 tokens.  FP32 sums of products of codes are exact up to
// 2^24, 1,024 inputs; after so many they are added as 32-bit integers.  (The
// integer m16n8k32 needs no expansion but has a quarter of the rate: 260 products
// a cycle and SM against 1,030 measured: 32 tokens by 19,456 x 2,560 took 35.6 us
// with it where this takes 23.5, 7 by 5,120 x 17,408 28 and 20.)
//
// Any order of k serves as long as both operands follow it, so a lane takes 32
// consecutive bytes of one row of w (and of x), 128 of a row for a quad of lanes:
// the 8 words are 8 k-steps of 16.
#include "common.cuh"
#include "kernels.h"

namespace q3 {

namespace {

constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int STEP_K = 128, FLUSH = 8;           // inputs of a step; steps that FP32 sums exactly

struct Words { uint32_t v[8]; };                 // 32 codes of a row

// 32 codes from byte k of a row
template <bool A32>
Q3_DEV Words load32(const int8_t* row, int k)
{
    Words w;
    if (A32) {
        asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w.v[0]), "=r"(w.v[1]), "=r"(w.v[2]), "=r"(w.v[3]), "=r"(w.v[4]), "=r"(w.v[5]), "=r"(w.v[6]), "=r"(w.v[7])
                     : "l"(row + k));
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + k)), b = __ldg(reinterpret_cast<const uint4*>(row + k) + 1);
        w.v[0] = a.x; w.v[1] = a.y; w.v[2] = a.z; w.v[3] = a.w;
        w.v[4] = b.x; w.v[5] = b.y; w.v[6] = b.z; w.v[7] = b.w;
    }
    return w;
}

// The same in a row's last step: zeros past its K codes
Q3_DEV Words load32_end(const int8_t* row, int k, int K)
{
    Words w;
#pragma unroll
    for (int i = 0; i < 8; ++i) w.v[i] = k + 4 * i + 4 <= K ? *reinterpret_cast<const uint32_t*>(row + k + 4 * i) : 0u;
    const int at = K & ~3;                       // the word that K cuts
    if (at >= k && at < k + 32 && at < K) {
        uint32_t b = 0;
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (at + e < K) b |= (uint32_t)(uint8_t)row[at + e] << (8 * e);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + 4 * i == at) w.v[i] = b;
    }
    return w;
}

Q3_DEV void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

Q3_DEV void store_out(const I8MatmulArgs& a, int64_t at, float v, bool& bad)
{
    switch (a.out_type) {
    case Q3_TYPE_F32: static_cast<float*>(a.out)[at] = v; break;
    case Q3_TYPE_F16: static_cast<__half*>(a.out)[at] = to_f16(v, bad); break;
    default: static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    }
}

// A warp: 16 channels by 8 NT tokens and a part of the inputs (in one piece: every
// kw-th step took 23.4 us where this takes 20.4, 7 tokens by 5,120 x 17,408); kw warps
// of a CTA share the channels, 8 / kw groups of them.
// (registers for four, three or two CTAs an SM: with two instead of four one token's
// product with 19,456 channels of 2,560 takes 13.8 us, not 11.1)
template <int NT, bool A32>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 4 : NT == 2 ? 3 : 2) i8_few_kernel(const I8MatmulArgs a, int kw)
{
    constexpr int ROWS = 16, COLS = 8 * NT, PITCH = COLS + 1;
    __shared__ int part[WARPS * ROWS * PITCH];
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int groups = WARPS / kw, group = warp / kw, share = warp % kw;
    const int64_t m0 = ((int64_t)blockIdx.x * groups + group) * ROWS;
    const int full = a.K / STEP_K;
    const int8_t* w0 = a.w + min(m0 + g, (int64_t)a.M - 1) * a.w_stride;
    const int8_t* w1 = a.w + min(m0 + g + 8, (int64_t)a.M - 1) * a.w_stride;
    const int8_t* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = a.x + (int64_t)min(8 * n + g, a.T - 1) * a.x_stride;
    int sum[NT][4] = {};
    float c[NT][4] = {};
    int fresh = 0;
    auto flush = [&] {
        fresh = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum[n][e] += __float2int_rn(c[n][e]);
                c[n][e] = 0.f;
            }
    };
    Words u, v, xs[NT];
    auto products = [&] {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t a0, a1, a2, a3, b0, b1;
            expand4(u.v[i], a0, a2);
            expand4(v.v[i], a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                expand4(xs[n].v[i], b0, b1);
                mma_f16(c[n], a0, a1, a2, a3, b0, b1);
            }
        }
        if (++fresh == FLUSH) flush();
    };
    if (m0 < a.M) {
        // the next step's bytes are requested when this one's are used: other warps'
        // are under way meanwhile
        auto load = [&](int s) {
            const int k = s * STEP_K + q * 32;
            u = load32<A32>(w0, k);
            v = load32<A32>(w1, k);
#pragma unroll
            for (int n = 0; n < NT; ++n) xs[n] = load32<false>(x[n], k);
        };
        const int s0 = (int)((int64_t)full * share / kw), s1 = (int)((int64_t)full * (share + 1) / kw);
        if (s0 < s1) load(s0);
#pragma unroll 1
        for (int s = s0; s < s1; ++s) {
            products();
            if (s + 1 < s1) load(s + 1);
        }
        if (full * STEP_K < a.K && share == kw - 1) {
            const int k = full * STEP_K + q * 32;
            u = load32_end(w0, k, a.K);
            v = load32_end(w1, k, a.K);
#pragma unroll
            for (int n = 0; n < NT; ++n) xs[n] = load32_end(x[n], k, a.K);
            products();
        }
        flush();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[(warp * ROWS + g + 8 * (e >> 1)) * PITCH + 8 * n + 2 * q + (e & 1)] = sum[n][e];
    __syncthreads();
    bool bad = false;
    const int outs = groups * ROWS;                 // channels of the CTA
    for (int i = threadIdx.x; i < outs * COLS; i += THREADS) {
        const int r = i % outs, t = i / outs;
        const int64_t m = (int64_t)blockIdx.x * outs + r;
        if (t >= a.T) break;
        if (m >= a.M) continue;
        int s = 0;
        for (int j = 0; j < kw; ++j) s += part[((r / ROWS * kw + j) * ROWS + r % ROWS) * PITCH + t];
        store_out(a, (int64_t)t * a.out_stride + m, (float)s * a.xs[t] * a.ws[m], bad);
    }
    if (bad && a.status) set_status(a.status, Q3_STATUS_F16_RANGE);
}

template <int NT, bool A32>
cudaError_t launch_few(const Launch& L, const I8MatmulArgs& a, int kw)
{
    cudaLaunchConfig_t cfg = {};
    const int rows = WARPS / kw * 16;
    cfg.gridDim = dim3((unsigned)((a.M + (int64_t)rows - 1) / rows));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.counter) ++*L.counter;
    return cudaLaunchKernelEx(&cfg, i8_few_kernel<NT, A32>, a, kw);
}

}  // namespace

// Warps that share a channel's inputs: eight, or four where eight, at 16 channels a
// CTA, would need more than the four CTAs an SM that reside (one token, channels of
// 2,560: 9,728 of them 7.1 us with eight and 7.7 with four, 9,800 9.7 and 7.9, 19,456
// 12.6 and 10.8), and no more than there are steps.  Long inputs of many channels
// lose by it (24,576 of 5,120: 24.9 and 27.5; 16 tokens by 19,456 of 5,120: 25.6 and 30.4).  More channels a warp or more steps under way cost
// resident warps and more time (13.5 us and 11.8).
cudaError_t launch_i8_few(const Launch& L, const I8MatmulArgs& a)
{
    const bool a32 = !(reinterpret_cast<uintptr_t>(a.w) & 31) && a.w_stride % 32 == 0;
    int kw = a.M > 152 * 4 * 16 ? 4 : 8;
    while (kw > 1 && (a.K + STEP_K - 1) / STEP_K < kw) kw /= 2;
    if (a.T <= 8) return a32 ? launch_few<1, true>(L, a, kw) : launch_few<1, false>(L, a, kw);
    if (a.T <= 16) return a32 ? launch_few<2, true>(L, a, kw) : launch_few<2, false>(L, a, kw);
    return a32 ? launch_few<4, true>(L, a, kw) : launch_few<4, false>(L, a, kw);
}

}  // namespace q3
