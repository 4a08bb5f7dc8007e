// k_i8_rows.cu -- rows of activations or weights in 8-bit integers with one
// scale a row: as they are, after the residual's addition and the RMS norm, or
// as SwiGLU of gate and up rows.
//
//   scale = max |y| / 127,  code = round-half-even(y / scale)
//
// The code depends on y / max |y| alone, so the norm's 1 / rms, equal for the
// whole row, enters the scale only: one pass over the row gives sum s^2 and
// max |s gain| together, from registers, and one barrier joins the warps.
// Codes come from fma(y, 127 / max, 1.5 * 2^23), whose low byte is the rounded
// product of y and the FP32 reciprocal: beside y's own rounding, a code is the
// neighbour of the definition's only where y / scale is within 127 * 2^-24 of a
// half.
//
// The maximum is taken over the bits of |y|, where infinities and NaN rank
// above every number: a row with one of them has scale NaN and zero codes.
// Rows whose squares, products or reciprocals leave FP32's range take the same
// steps in 64 bits.
#include "common.cuh"
#include "kernels.h"

namespace q3 {

namespace {

constexpr int QUANT = 0, NORM = 1, SWIGLU = 2;
constexpr uint32_t INF_BITS = 0x7f800000u;
constexpr float MAGIC = 12582912.0f;             // 1.5 * 2^23

template <typename X> Q3_DEV float to_f(X v);
template <> Q3_DEV float to_f<float>(float v) { return v; }
template <> Q3_DEV float to_f<__half>(__half v) { return __half2float(v); }
template <> Q3_DEV float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename X> Q3_DEV X from_f(float v);
template <> Q3_DEV float from_f<float>(float v) { return v; }
template <> Q3_DEV __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> Q3_DEV __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename X> struct alignas(16) Eight { X v[8]; };

// Thread tid of n holds eight values of chunk i of a row: consecutive ones
// (VEC), read as vectors, or every n-th, whose addresses need no alignment.
template <bool VEC>
Q3_DEV int place(int tid, int n, int i, int e) { return VEC ? 8 * (tid + i * n) + e : tid + (i * 8 + e) * n; }

template <typename X, bool VEC>
Q3_DEV void load8(const X* p, int tid, int n, int i, int K, float (&v)[8])
{
    if (VEC && place<VEC>(tid, n, i, 7) < K) {
        const Eight<X> w = *reinterpret_cast<const Eight<X>*>(p + place<VEC>(tid, n, i, 0));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f(w.v[e]);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int k = place<VEC>(tid, n, i, e);
        v[e] = k < K ? to_f(p[k]) : 0.f;
    }
}

template <typename X, bool VEC>
Q3_DEV void store8(X* p, int tid, int n, int i, int K, const float (&v)[8], bool vec)
{
    if (VEC && vec && place<VEC>(tid, n, i, 7) < K) {
        Eight<X> w;
#pragma unroll
        for (int e = 0; e < 8; ++e) w.v[e] = from_f<X>(v[e]);
        *reinterpret_cast<Eight<X>*>(p + place<VEC>(tid, n, i, 0)) = w;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int k = place<VEC>(tid, n, i, e);
        if (k < K) p[k] = from_f<X>(v[e]);
    }
}

// z / (1 + e^-z), for z < 0 as z e^z / (1 + e^z), the power as a square of its
// root: FP32 holds every step as long as it holds the result
Q3_DEV float silu(float z)
{
    const float h = expf(-0.5f * fabsf(z));
    return (z < 0.f ? z * h * h : z) / (1.0f + h * h);
}

// The eight values of chunk i before the row's statistics: x, s = x + delta
// rounded to x's type (and stored), or silu(gate) * up
template <typename X, int OP, bool VEC>
Q3_DEV void row_values(const I8RowArgs& a, int64_t r, int tid, int n, int i, bool again, float (&y)[8])
{
    const X* x = static_cast<const X*>(a.x) + r * a.x_stride;
    if (OP == NORM && a.delta) {
        X* sum = static_cast<X*>(a.sum) + r * a.sum_stride;
        if (again) {                                       // a second pass: x may have been overwritten
            load8<X, VEC>(sum, tid, n, i, a.K, y);
            return;
        }
        float d[8];
        load8<X, VEC>(x, tid, n, i, a.K, y);
        switch (a.delta_type) {
        case Q3_TYPE_F32: load8<float, VEC>(static_cast<const float*>(a.delta) + r * a.delta_stride, tid, n, i, a.K, d); break;
        case Q3_TYPE_F16: load8<__half, VEC>(static_cast<const __half*>(a.delta) + r * a.delta_stride, tid, n, i, a.K, d); break;
        default: load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(a.delta) + r * a.delta_stride, tid, n, i, a.K, d);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = to_f(from_f<X>(y[e] + d[e]));
        store8<X, VEC>(sum, tid, n, i, a.K, y, true);
        return;
    }
    load8<X, VEC>(x, tid, n, i, a.K, y);
    if (OP == SWIGLU) {
        float u[8];
        load8<X, VEC>(x + a.K, tid, n, i, a.K, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = silu(y[e]) * u[e];
    }
}

// max over the block, by the bits of |value|, and (ss) the sum
template <bool SUM>
Q3_DEV void block_join(uint32_t& m, float& ss)
{
    __shared__ uint32_t sm_m[32];
    __shared__ float sm_s[32];
    m = __reduce_max_sync(0xffffffffu, m);
    if (SUM) ss = warp_allsum(ss);
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warps == 1) return;
    if (lane == 0) {
        sm_m[warp] = m;
        if (SUM) sm_s[warp] = ss;
    }
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, lane < warps ? sm_m[lane] : 0u);
    if (SUM) ss = warp_allsum(lane < warps ? sm_s[lane] : 0.f);
}

// the same in 64 bits; a NaN among the values stays one
__device__ __noinline__ void block_join64(double& m, double& ss)
{
    __shared__ double sm_m[32], sm_s[32];
    for (int o = 16; o > 0; o >>= 1) {
        const double v = __shfl_xor_sync(0xffffffffu, m, o);
        m = m > v || m != m ? m : v;
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warps == 1) return;
    if (lane == 0) {
        sm_m[warp] = m;
        sm_s[warp] = ss;
    }
    __syncthreads();
    m = sm_m[0];
    ss = sm_s[0];
    for (int w = 1; w < warps; ++w) {
        m = m > sm_m[w] || m != m ? m : sm_m[w];
        ss += sm_s[w];
    }
}

// codes (low bytes of bits) and the values they stand for
template <bool VEC>
Q3_DEV void store_codes(const I8RowArgs& a, int64_t r, int tid, int n, int i, const uint32_t (&bits)[8], const float (&code)[8], float scale)
{
    int8_t* codes = a.codes + r * a.code_stride;
    if (VEC && place<VEC>(tid, n, i, 7) < a.K) {
        const uint32_t lo = __byte_perm(__byte_perm(bits[0], bits[1], 0x0040), __byte_perm(bits[2], bits[3], 0x0040), 0x5410);
        const uint32_t hi = __byte_perm(__byte_perm(bits[4], bits[5], 0x0040), __byte_perm(bits[6], bits[7], 0x0040), 0x5410);
        *reinterpret_cast<uint2*>(codes + place<VEC>(tid, n, i, 0)) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int k = place<VEC>(tid, n, i, e);
            if (k < a.K) codes[k] = (int8_t)(bits[e] & 0xff);
        }
    }
    if (!a.values) return;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = code[e] * scale;
    const int64_t at = r * a.K;
    switch (a.values_type) {
    case Q3_TYPE_F32: store8<float, VEC>(static_cast<float*>(a.values) + at, tid, n, i, a.K, v, a.values_vec); break;
    case Q3_TYPE_F16: store8<__half, VEC>(static_cast<__half*>(a.values) + at, tid, n, i, a.K, v, a.values_vec); break;
    default: store8<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16*>(a.values) + at, tid, n, i, a.K, v, a.values_vec);
    }
}

// One row a CTA.  V > 0: a thread holds all its 8 V values in registers.  V ==
// 0: longer rows are read twice.
template <typename X, int OP, bool VEC, int V>
__global__ void __launch_bounds__(1024) i8_rows_kernel(const I8RowArgs a)
{
    grid_dep_wait();
    const int tid = threadIdx.x, n = blockDim.x;
    const int64_t r = blockIdx.x;
    const int chunks = V > 0 ? V : (a.K + 8 * n - 1) / (8 * n);
    float y[V > 0 ? V : 1][8];
    auto gains = [&](int i, float (&g)[8]) { load8<__nv_bfloat16, VEC>(a.gain, tid, n, i, a.K, g); };
    float g[V > 0 ? V : 1][8];

    uint32_t m = 0;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
        float (&yi)[8] = y[V > 0 ? i : 0];
        float (&gi)[8] = g[V > 0 ? i : 0];
        if (OP == NORM) gains(i, gi);
        row_values<X, OP, VEC>(a, r, tid, n, i, false, yi);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (OP == NORM) {
                ss += yi[e] * yi[e];
                m = max(m, __float_as_uint(yi[e] * gi[e]) & 0x7fffffffu);
            } else {
                m = max(m, __float_as_uint(yi[e]) & 0x7fffffffu);
            }
        }
    }
    block_join<OP == NORM>(m, ss);

    const float top = __uint_as_float(m);
    float scale = top / 127.0f;
    if (OP == NORM) scale *= 1.0f / sqrtf(ss / (float)a.K + a.eps);
    // FP32 holds every step: squares, products and the reciprocal of the maximum
    bool plain = m < INF_BITS && top > 1e-30f && scale < INFINITY;
    if (OP == NORM) plain = plain && ss > 1e-30f && ss < INFINITY;
    double top64 = 0.0;
    bool bad = false;
    if (!plain) {
        if (OP == NORM) {
            double ss64 = 0.0;
            for (int i = 0; i < chunks; ++i) {
                if (V == 0) {
                    gains(i, g[0]);
                    row_values<X, OP, VEC>(a, r, tid, n, i, true, y[0]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float ye = y[0][e], ge = g[0][e];
#pragma unroll
                    for (int j = 1; j < V; ++j) {
                        ye = i == j ? y[j][e] : ye;
                        ge = i == j ? g[j][e] : ge;
                    }
                    ss64 += (double)ye * ye;
                    const double v = fabs((double)ye * ge);
                    if (!(top64 != top64) && !(v <= top64)) top64 = v;
                }
            }
            block_join64(top64, ss64);
            scale = (float)(top64 / sqrt(ss64 / a.K + (double)a.eps) / 127.0);
            if (top64 == 0.0) scale = 0.f;
        } else {
            top64 = top;
        }
        bad = !(scale < INFINITY);
        if (bad) {
            scale = __uint_as_float(0x7fffffffu);
            if (tid == 0 && a.status) set_status(a.status, Q3_STATUS_F16_RANGE);
        }
    }
    if (tid == 0) a.scales[r] = scale;
    const bool zero = bad || scale == 0.f;
    const float inv = plain ? 127.0f / top : 0.f;
    const double inv64 = plain || zero ? 0.0 : 127.0 / top64;
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
        float (&yi)[8] = y[V > 0 ? i : 0];
        float (&gi)[8] = g[V > 0 ? i : 0];
        if (V == 0) {
            if (OP == NORM) gains(i, gi);
            row_values<X, OP, VEC>(a, r, tid, n, i, true, yi);
        }
        uint32_t bits[8];
        float code[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float c;
            if (plain) c = fmaf(OP == NORM ? yi[e] * gi[e] : yi[e], inv, MAGIC);
            else c = MAGIC + (zero ? 0.f : (float)fmin(fmax(rint((OP == NORM ? (double)yi[e] * gi[e] : (double)yi[e]) * inv64), -127.0), 127.0));
            bits[e] = __float_as_uint(c);
            code[e] = c - MAGIC;
        }
        store_codes<VEC>(a, r, tid, n, i, bits, code, scale);
    }
}

template <typename X, int OP, bool VEC, int V>
cudaError_t launch_v(const Launch& L, const I8RowArgs& a)
{
    const int per = 8 * (V > 0 ? V : 4);
    int threads = (a.K + per - 1) / per;
    threads = threads > 1024 ? 1024 : (threads + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.counter) ++*L.counter;
    return cudaLaunchKernelEx(&cfg, i8_rows_kernel<X, OP, VEC, V>, a);
}

template <typename X, int OP, bool VEC>
cudaError_t launch_k(const Launch& L, const I8RowArgs& a)
{
    if (a.K <= 8 * 1024) return launch_v<X, OP, VEC, 1>(L, a);
    if (a.K <= 16 * 1024) return launch_v<X, OP, VEC, 2>(L, a);
    return launch_v<X, OP, VEC, 0>(L, a);
}

size_t size_of(int type) { return type == Q3_TYPE_F32 ? 4 : 2; }
// whether rows `stride` elements apart from p begin on 16-byte boundaries
bool rows16(const void* p, int64_t stride, int type, int T)
{
    return !(reinterpret_cast<uintptr_t>(p) & 15) && (T == 1 || stride * size_of(type) % 16 == 0);
}

template <typename X, int OP>
cudaError_t launch_op(const Launch& L, I8RowArgs a, int type)
{
    bool vec = rows16(a.x, a.x_stride, type, a.T);
    if (OP == SWIGLU) vec = vec && a.K * size_of(type) % 16 == 0;          // where the up values begin
    if (OP == NORM) {
        vec = vec && !(reinterpret_cast<uintptr_t>(a.gain) & 15);
        if (a.delta) vec = vec && rows16(a.delta, a.delta_stride, a.delta_type, a.T) && rows16(a.sum, a.sum_stride, type, a.T);
    }
    a.values_vec = a.values && rows16(a.values, a.K, a.values_type, a.T);
    return vec ? launch_k<X, OP, true>(L, a) : launch_k<X, OP, false>(L, a);
}

template <int OP>
cudaError_t launch_type(const Launch& L, const I8RowArgs& a, int type)
{
    switch (type) {
    case Q3_TYPE_F32: return launch_op<float, OP>(L, a, type);
    case Q3_TYPE_F16: return launch_op<__half, OP>(L, a, type);
    default: return launch_op<__nv_bfloat16, OP>(L, a, type);
    }
}

}  // namespace

cudaError_t launch_i8_quantize(const Launch& L, const I8RowArgs& a, int type) { return launch_type<QUANT>(L, a, type); }
cudaError_t launch_i8_norm(const Launch& L, const I8RowArgs& a, int type) { return launch_type<NORM>(L, a, type); }
cudaError_t launch_i8_swiglu(const Launch& L, const I8RowArgs& a, int type) { return launch_type<SWIGLU>(L, a, type); }

}  // namespace q3
