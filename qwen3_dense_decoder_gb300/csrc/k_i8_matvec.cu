// k_i8_matvec.cu -- out[t][m] = (sum_k x[t][k] w[m][k]) xs[t] ws[m] over 8-bit
// codes, for few rows of x: bound by the bytes of w.
//
// mma.sync m16n8k32 on 16 rows of w and 8 of x sums whole numbers exactly.  Any
// order of k serves as long as both operands follow it, so a lane takes its
// fragments of two k-steps from 16 consecutive bytes of one row of w (and of x):
// 64 bytes of a row at a time for a quad of lanes.
#include "common.cuh"
#include "kernels.h"

namespace q3 {

namespace {

constexpr int WARPS = 8;

Q3_DEV void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// bytes k .. k + 15 of a row of K, zeros past its end
Q3_DEV uint4 load16(const int8_t* row, int k, int K)
{
    if (k + 16 <= K) return ldg_nc_v4(row + k);
    uint4 v = make_uint4(0, 0, 0, 0);
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (k + e < K) w[e >> 2] |= (uint32_t)(uint8_t)row[k + e] << (8 * (e & 3));
    return v;
}

Q3_DEV void store_out(const I8MatmulArgs& a, int64_t at, float v, bool& bad)
{
    switch (a.out_type) {
    case Q3_TYPE_F32: static_cast<float*>(a.out)[at] = v; break;
    case Q3_TYPE_F16: static_cast<__half*>(a.out)[at] = to_f16(v, bad); break;
    default: static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    }
}

// A CTA: WARPS / KW groups of 16 output channels, 8 rows of x; KW warps share a
// group's inputs, in steps of 64 taken in turn.
template <int KW>
__global__ void __launch_bounds__(WARPS * 32) i8_matvec_kernel(const I8MatmulArgs a)
{
    constexpr int GROUPS = WARPS / KW;
    __shared__ int part[WARPS][16][9];
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int group = warp / KW, share = warp % KW;
    const int64_t m0 = ((int64_t)blockIdx.x * GROUPS + group) * 16;
    const int t0 = blockIdx.y * 8;
    const int64_t lo = min(m0 + g, (int64_t)a.M - 1), hi = min(m0 + g + 8, (int64_t)a.M - 1);
    const int8_t* w0 = a.w + lo * a.w_stride;
    const int8_t* w1 = a.w + hi * a.w_stride;
    const bool live = t0 + g < a.T;
    const int8_t* x = a.x + (live ? t0 + g : 0) * a.x_stride;
    int c[4] = {0, 0, 0, 0};
    if (m0 < a.M) {
#pragma unroll 4
        for (int k0 = share * 64; k0 < a.K; k0 += KW * 64) {
            const int k = k0 + q * 16;
            const uint4 u = load16(w0, k, a.K), v = load16(w1, k, a.K);
            const uint4 b = live ? load16(x, k, a.K) : make_uint4(0, 0, 0, 0);
            mma_s8(c, u.x, v.x, u.y, v.y, b.x, b.y);
            mma_s8(c, u.z, v.z, u.w, v.w, b.z, b.w);
        }
    }
    part[warp][g][2 * q] = c[0];
    part[warp][g][2 * q + 1] = c[1];
    part[warp][g + 8][2 * q] = c[2];
    part[warp][g + 8][2 * q + 1] = c[3];
    __syncthreads();
    bool bad = false;
    for (int i = threadIdx.x; i < GROUPS * 128; i += WARPS * 32) {
        const int r = i & 15, gr = (i >> 4) % GROUPS, t = (i >> 4) / GROUPS;
        const int64_t m = ((int64_t)blockIdx.x * GROUPS + gr) * 16 + r;
        if (m >= a.M || t0 + t >= a.T) continue;
        int s = 0;
#pragma unroll
        for (int j = 0; j < KW; ++j) s += part[gr * KW + j][r][t];
        store_out(a, (int64_t)(t0 + t) * a.out_stride + m, (float)s * a.xs[t0 + t] * a.ws[m], bad);
    }
    if (bad && a.status) set_status(a.status, Q3_STATUS_F16_RANGE);
}

template <int KW>
cudaError_t launch_kw(const Launch& L, const I8MatmulArgs& a)
{
    cudaLaunchConfig_t cfg = {};
    const int rows = WARPS / KW * 16;
    cfg.gridDim = dim3((unsigned)((a.M + rows - 1) / rows), (unsigned)((a.T + 7) / 8));
    cfg.blockDim = dim3(WARPS * 32);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.counter) ++*L.counter;
    return cudaLaunchKernelEx(&cfg, i8_matvec_kernel<KW>, a);
}

}  // namespace

cudaError_t launch_i8_matvec(const Launch& L, const I8MatmulArgs& a) { return launch_kw<8>(L, a); }

}  // namespace q3
