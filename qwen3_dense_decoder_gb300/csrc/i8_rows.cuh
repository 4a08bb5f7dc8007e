// i8_rows.cuh -- rows of activations or weights in 8-bit integers with one
// scale a row: as they are, after the residual's addition and the RMS norm, or
// as SwiGLU of gate and up rows.
//
//   scale = max |y| / 127,  code = round-half-even(y / scale)
//
// The code depends on y / max |y| alone, so the norm's 1 / rms, equal for the
// whole row, enters the scale only: one pass over the row gives sum s^2 and
// max |s gain| together, from registers, and one barrier joins the warps.
// Codes come from the product of y and 127 / max, corrected by its remainder, so
// that a value halfway between two codes (values of 8 or 11 bits often are) is seen
// as such and goes to the even one: of fp16 or bf16 values every code is the
// definition's, of others all but those whose own rounding crosses a half.  (Without
// the correction the halves of a row all went one way, and the codes' error grew by
// up to 1.45 times.)  Adding 1.5 * 2^23 leaves the code in the low byte.
//
// The maximum is taken over the bits of |y|, where infinities and NaN rank
// above every number: a row with one of them has scale NaN and zero codes.
// Rows whose squares, products or reciprocals leave FP32's range take the same
// steps in 64 bits, and so do rows of zeros, whose maximum has no reciprocal: one
// of 2,560 values takes 10 to 12 us where another takes 2, one of 17,408 40 to 52
// where another takes 3 to 4, and 2,048 rows of 5,120 of which half are zeros 108
// to 176 us where others take 8 to 15 (a batch's padding costs as much).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace q3 {

namespace {

constexpr int QUANT = 0, NORM = 1, SWIGLU = 2;
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
    X w[8];                                     // unconditional loads, so that all eight are under way together
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = p[min(place<VEC>(tid, n, i, e), K - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = place<VEC>(tid, n, i, e) < K ? to_f(w[e]) : 0.f;
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

// z / (1 + e^-z) with e = e^-|z|: z / (1 + e), or z e / (1 + e) below zero.
// e^-b = 2^t (1 + r ln 2) with t the rounded product b log2(1/e) and r what that
// leaves: 2^-22 of the value or less, by ex2.approx.  Below -64 e^-64 is taken out
// and multiplied into z first, so that FP32 holds every step as long as it holds
// the result.  From 200 on e is 0, and b goes no further: its product with HI
// would leave FP32 (|z| above 2.35e38) and what it leaves be infinite.  IEEE expf
// and division take 35.9 us where this takes 30.9 (2,048 rows of 9,728 fp16).
Q3_DEV float silu(float z)
{
    constexpr double LOG2E = 1.44269504088896340736;
    constexpr float HI = (float)LOG2E, LO = (float)(LOG2E - (double)HI);
    const bool far = z < -64.f;
    const float b = fminf(fabsf(z) - (far ? 64.f : 0.f), 200.f), t = -HI * b;
    float e = fast_ex2(t);
    e = fmaf(e, fmaf(-LO, b, fmaf(-HI, b, -t)) * 0.69314718f, e);
    const float top = z < 0.f ? (far ? z * 1.60381089e-28f : z) * e : z;
    return __fdividef(top, 1.0f + (far ? 0.f : e));
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
// (into one of two exchanges in turn, so that a row needs one barrier)
template <bool SUM>
Q3_DEV void block_join(uint32_t& m, float& ss, int parity)
{
    __shared__ uint32_t sm_ms[2][32];
    __shared__ float sm_ss[2][32];
    uint32_t* sm_m = sm_ms[parity];
    float* sm_s = sm_ss[parity];
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

// codes (low bytes of bits) and the values they stand for; all lanes of a warp
template <bool VEC, bool TURN = false>
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
    if (TURN && !a.values_vec) {
        // rows of values begin anywhere: the warp's 256 change hands, so that its
        // lanes store consecutive ones (701 rows of 2,047 fp16: 7.9 us without)
        extern __shared__ float turned[];
        float* mine = turned + (tid & ~31) * 8;
        const int lane = tid & 31, k0 = place<VEC>(tid - lane, n, i, 0);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[lane * 8 + e] = v[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = mine[e * 32 + lane];
        const int64_t first = r * a.K + k0 + lane;
        auto put = [&](auto* p) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k0 + e * 32 + lane < a.K) p[first + e * 32] = from_f<std::remove_pointer_t<decltype(p)>>(v[e]);
        };
        if (a.values_type == Q3_TYPE_F32) put(static_cast<float*>(a.values));
        else if (a.values_type == Q3_TYPE_F16) put(static_cast<__half*>(a.values));
        else put(static_cast<__nv_bfloat16*>(a.values));
        return;
    }
    const int64_t at = r * a.K;
    switch (a.values_type) {
    case Q3_TYPE_F32: store8<float, VEC>(static_cast<float*>(a.values) + at, tid, n, i, a.K, v, a.values_vec); break;
    case Q3_TYPE_F16: store8<__half, VEC>(static_cast<__half*>(a.values) + at, tid, n, i, a.K, v, a.values_vec); break;
    default: store8<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16*>(a.values) + at, tid, n, i, a.K, v, a.values_vec);
    }
}

template <bool VEC>
Q3_DEV void gains(const I8RowArgs& a, int tid, int n, int i, float (&g)[8]) { load8<__nv_bfloat16, VEC>(a.gain, tid, n, i, a.K, g); }

// A row's scale, by one thread.  Its largest code is 127 (or the scale 0 or NaN), so
// that one comparison tells whether every value is a finite number of its type: below
// the half between that type's largest and the next power of two.
Q3_DEV void put_scale(const I8RowArgs& a, int64_t r, float scale)
{
    a.scales[r] = scale;
    if (!a.values || !a.status) return;
    const float limit = a.values_type == Q3_TYPE_F32 ? INFINITY : a.values_type == Q3_TYPE_F16 ? 65520.f : __uint_as_float(0x7f7f8000u);
    if (!(127.0f * scale < limit)) set_status(a.status, Q3_STATUS_F16_RANGE);
}

// A row whose steps leave FP32's range, in 64 bits; or one with what is no
// number, or zeros alone.  Out of line and reading the row again: the FP64 unit
// is slow, and its code beside the common path's took that one from 131 to 717 us
// (34,816 rows of 5,120).
template <typename X, int OP, bool VEC>
__device__ __noinline__ void rare_row(const I8RowArgs& a, int64_t r, int tid, int n)
{
    const int chunks = (a.K + 8 * n - 1) / (8 * n);
    float y[8], g[8];
    double top = 0.0, ss = 0.0;
    auto value = [&](int e) { return OP == NORM ? (double)y[e] * g[e] : (double)y[e]; };
    for (int i = 0; i < chunks; ++i) {
        row_values<X, OP, VEC>(a, r, tid, n, i, true, y);
        if (OP == NORM) gains<VEC>(a, tid, n, i, g);
        for (int e = 0; e < 8; ++e) {
            ss += (double)y[e] * y[e];
            const double v = fabs(value(e));
            if (!(v <= top) && top == top) top = v;
        }
    }
    block_join64(top, ss);
    float scale = top == 0.0 ? 0.f : (float)(OP == NORM ? top / sqrt(ss / a.K + (double)a.eps) / 127.0 : top / 127.0);
    const bool bad = !(scale < INFINITY);
    if (bad) scale = __uint_as_float(0x7fffffffu);
    if (tid == 0) {
        put_scale(a, r, scale);
        if (bad && a.status) set_status(a.status, Q3_STATUS_F16_RANGE);
    }
    const bool zero = bad || scale == 0.f;
    for (int i = 0; i < chunks; ++i) {
        row_values<X, OP, VEC>(a, r, tid, n, i, true, y);
        if (OP == NORM) gains<VEC>(a, tid, n, i, g);
        uint32_t bits[8];
        float code[8];
        for (int e = 0; e < 8; ++e) {
            code[e] = zero ? 0.f : (float)fmin(fmax(rint(127.0 * value(e) / top), -127.0), 127.0);
            bits[e] = (uint32_t)(int)code[e];
        }
        store_codes<VEC>(a, r, tid, n, i, bits, code, scale);
    }
}

// codes and values of eight y of a row that FP32 holds, top its maximum: the
// product with 127 / top, corrected by what 127 y leaves
template <int OP, bool VEC, bool TURN = false>
Q3_DEV void emit(const I8RowArgs& a, int64_t r, int tid, int n, int i, const float (&y)[8], float top, float scale)
{
    const float one = 1.0f / top, inv = 127.0f * one;
    uint32_t bits[8];
    float code[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = y[e] * inv;
        // (SwiGLU's y lie nowhere in particular: 30.9 us without, 32.7 with, 2,048 rows of 9,728)
        const float c = (OP == SWIGLU ? q : fmaf(fmaf(-q, top, 127.0f * y[e]), one, q)) + MAGIC;
        bits[e] = __float_as_uint(c);
        code[e] = c - MAGIC;
    }
    store_codes<VEC, TURN>(a, r, tid, n, i, bits, code, scale);
}

// the scale of a row from max |y| (by its bits) and sum s^2; false where FP32
// does not hold every step: squares, products, 127 y and the reciprocal of the maximum
template <int OP>
Q3_DEV bool row_scale(const I8RowArgs& a, uint32_t m, float ss, float& scale)
{
    const float top = __uint_as_float(m);
    scale = top / 127.0f;
    if (OP == NORM) scale *= 1.0f / sqrtf(ss / (float)a.K + a.eps);
    bool plain = top > 1e-30f && top < 1e36f && scale < INFINITY;
    if (OP == NORM) plain = plain && ss > 1e-30f && ss < INFINITY;
    return plain;
}

Q3_DEV void max_of(const float (&y)[8], uint32_t& m)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(y[e]) & 0x7fffffffu);
}

Q3_DEV void times_gain(float (&y)[8], const float (&g)[8], float& ss)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        ss += y[e] * y[e];
        y[e] *= g[e];
    }
}

// A row a CTA, at any alignment (not VEC) or of any length (V == 0: read twice;
// else its 8 V values a thread stay in registers).
template <typename X, int OP, bool VEC, int V>
__global__ void __launch_bounds__(V ? 640 : 1024) i8_rows_any_kernel(const I8RowArgs a)
{
    grid_dep_wait();
    grid_dep_launch();                           // 32 rows' SwiGLU in a row of calls: 3.9 -> 3.1 us
    const int tid = threadIdx.x, n = blockDim.x;
    const int64_t r = blockIdx.x;
    const int chunks = V ? V : (a.K + 8 * n - 1) / (8 * n);
    uint32_t m = 0;
    float ss = 0.f, y[V ? V : 1][8];
    auto values = [&](int i, bool again, float (&v)[8]) {
        float g[8];
        if (OP == NORM) gains<VEC>(a, tid, n, i, g);
        row_values<X, OP, VEC>(a, r, tid, n, i, again, v);
        if (OP == NORM) times_gain(v, g, ss);
    };
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
        values(i, false, y[V ? i : 0]);
        max_of(y[V ? i : 0], m);
    }
    block_join<OP == NORM>(m, ss, 0);
    float scale;
    if (!row_scale<OP>(a, m, ss, scale)) {
        rare_row<X, OP, VEC>(a, r, tid, n);
        return;
    }
    if (tid == 0) put_scale(a, r, scale);
    const float top = __uint_as_float(m);
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
        if (!V) values(i, true, y[0]);
        emit<OP, VEC>(a, r, tid, n, i, y[V ? i : 0], top, scale);
    }
}

// Rows that begin on 16-byte boundaries, in registers: thread tid of n holds
// eights tid, tid + n, ... of a row, V of them.  A CTA takes every gridDim.x-th
// row and requests the next one's bytes before it works on this one's.
struct Raw { uint4 v[2]; };                      // eight values, the second half used by f32

Q3_DEV Raw raw_load(const void* row, int type, int k, int K)
{
    Raw w;
    w.v[0] = w.v[1] = make_uint4(0, 0, 0, 0);
    if (k >= K) return w;
    const int size = type == Q3_TYPE_F32 ? 4 : 2;
    const uint8_t* p = static_cast<const uint8_t*>(row) + (size_t)k * size;
    if (k + 8 <= K) {
        w.v[0] = *reinterpret_cast<const uint4*>(p);
        if (size == 4) w.v[1] = *reinterpret_cast<const uint4*>(p + 16);
    } else if (size == 4) {
        uint32_t* o = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (k + e < K) o[e] = reinterpret_cast<const uint32_t*>(p)[e];
    } else {
        uint32_t* o = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (k + e < K) o[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
    }
    return w;
}

Q3_DEV void raw_values(const Raw& w, int type, float (&y)[8])
{
    const uint32_t* o = reinterpret_cast<const uint32_t*>(&w);
    if (type == Q3_TYPE_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(o[e]);
    } else if (type == Q3_TYPE_F16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[e]));
            y[2 * e] = f.x;
            y[2 * e + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[2 * e] = bf16lo(o[e]);
            y[2 * e + 1] = bf16hi(o[e]);
        }
    }
}

template <typename X> constexpr int type_code() { return sizeof(X) == 4 ? Q3_TYPE_F32 : Q3_TYPE_BF16; }
template <> constexpr int type_code<__half>() { return Q3_TYPE_F16; }

// DELTA: the type of what the norm adds, or -1
template <typename X, int OP, int V, int DELTA>
__global__ void __launch_bounds__(640) i8_rows_kernel(const I8RowArgs a)
{
    constexpr int TYPE = type_code<X>();
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, n = blockDim.x;
    constexpr bool ADD = DELTA >= 0;
    Raw x[V], z[V], gain[V];
    auto request = [&](int64_t r) {
        const X* row = static_cast<const X*>(a.x) + r * a.x_stride;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int k = 8 * (tid + i * n);
            x[i] = raw_load(row, TYPE, k, a.K);
            if (OP == SWIGLU) z[i] = raw_load(row + a.K, TYPE, k, a.K);
            if (ADD) z[i] = raw_load(static_cast<const uint8_t*>(a.delta) + r * a.delta_stride * (DELTA == Q3_TYPE_F32 ? 4 : 2), DELTA, k, a.K);
        }
    };
    int64_t r = blockIdx.x;
    request(r);
    if (OP == NORM)
#pragma unroll
        for (int i = 0; i < V; ++i) gain[i] = raw_load(a.gain, Q3_TYPE_BF16, 8 * (tid + i * n), a.K);
    int parity = 0;
    while (true) {
        float y[V][8];
        uint32_t m = 0;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            raw_values(x[i], TYPE, y[i]);
            if (OP == SWIGLU) {
                float u[8];
                raw_values(z[i], TYPE, u);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[i][e] = silu(y[i][e]) * u[e];
            }
            if (ADD) {
                float d[8];
                raw_values(z[i], DELTA, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[i][e] = to_f(from_f<X>(y[i][e] + d[e]));
                store8<X, true>(static_cast<X*>(a.sum) + r * a.sum_stride, tid, n, i, a.K, y[i], true);
            }
            if (OP == NORM) {
                float g[8];
                raw_values(gain[i], Q3_TYPE_BF16, g);
                times_gain(y[i], g, ss);
            }
            max_of(y[i], m);
        }
        const int64_t next = r + gridDim.x;
        if (next < a.T) request(next);
        block_join<OP == NORM>(m, ss, parity);
        parity ^= 1;
        float scale;
        if (row_scale<OP>(a, m, ss, scale)) {
            if (tid == 0) put_scale(a, r, scale);
            const float top = __uint_as_float(m);
#pragma unroll
            for (int i = 0; i < V; ++i) emit<OP, true, true>(a, r, tid, n, i, y[i], top, scale);
        } else {
            rare_row<X, OP, true>(a, r, tid, n);
            __syncthreads();                               // its exchange is free for the next such row
        }
        if (next >= a.T) return;
        r = next;
    }
}

template <typename K>
cudaError_t launch_one(const Launch& L, K kernel, const I8RowArgs& a, int grid, int threads, size_t smem)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.counter) ++*L.counter;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

int threads_for(int K, int V) { return ((K + 8 * V - 1) / (8 * V) + 31) / 32 * 32; }

// One wave of CTAs, 640 threads an SM: what 96 registers a thread let reside
// (two waves' worth: the norm of 2,048 rows of 5,120 20.7 us, one 19.1; SwiGLU of
// 2,048 of 9,728 32.1 and 30.9; 34,816 rows of 5,120 quantised 139 and 140).
template <typename X, int OP, int V, int DELTA>
cudaError_t launch_v(const Launch& L, const I8RowArgs& a)
{
    const int threads = threads_for(a.K, V);
    const int64_t grid = 152ll * (640 / threads);
    const size_t smem = a.values && !a.values_vec ? threads * 8 * sizeof(float) : 0;
    return launch_one(L, i8_rows_kernel<X, OP, V, DELTA>, a, a.T < grid ? a.T : (int)grid, threads, smem);
}

// Eights a thread: fewer threads a row leave more rows' bytes under way between
// barriers (34,816 bf16 rows of 5,120: 151 us with two, 141 with four), but the
// norm's two operands and gains then fill the registers (2,048 rows of 5,120: 19.1 us
// with two, 22.8 with four; one row of 2,560: 2.5 and 4.4).  SwiGLU differs less (32
// rows of 9,728: 3.2 and 3.5; 2,048: 30.9 and 30.7).
template <typename X, int OP, int DELTA>
cudaError_t launch_rows(const Launch& L, const I8RowArgs& a)
{
    if constexpr (OP != QUANT)
        if (threads_for(a.K, 2) <= 640) return launch_v<X, OP, 2, DELTA>(L, a);
    if (threads_for(a.K, 4) <= 640) return launch_v<X, OP, 4, DELTA>(L, a);
    return launch_one(L, i8_rows_any_kernel<X, OP, true, 0>, a, a.T, 1024, 0);
}

// (701 rows of 2 x 9,729 fp16 values read twice: 39 us)
template <typename X, int OP>
cudaError_t launch_unaligned(const Launch& L, const I8RowArgs& a)
{
    if (threads_for(a.K, 2) <= 640) return launch_one(L, i8_rows_any_kernel<X, OP, false, 2>, a, a.T, threads_for(a.K, 2), 0);
    if (threads_for(a.K, 4) <= 640) return launch_one(L, i8_rows_any_kernel<X, OP, false, 4>, a, a.T, threads_for(a.K, 4), 0);
    return launch_one(L, i8_rows_any_kernel<X, OP, false, 0>, a, a.T, 1024, 0);
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
    if (!vec) return launch_unaligned<X, OP>(L, a);
    if constexpr (OP == NORM) {
        if (a.delta) {
            switch (a.delta_type) {
            case Q3_TYPE_F32: return launch_rows<X, OP, Q3_TYPE_F32>(L, a);
            case Q3_TYPE_F16: return launch_rows<X, OP, Q3_TYPE_F16>(L, a);
            default: return launch_rows<X, OP, Q3_TYPE_BF16>(L, a);
            }
        }
    }
    return launch_rows<X, OP, -1>(L, a);
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

}  // namespace q3
