// k_kv4.cu -- the 4-bit K/V cache's writer and attention ("Kipp Roadmap",
// status v0.0.2: 32-position block tables; status v0.0.4: a quantized cache is
// opt-in).  The tile format is in kv4.cuh.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace q3 {

namespace {

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
Q3_DEV void load4(const __nv_bfloat16* p, int lane, float (&y)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p + lane * 4);
    y[0] = bf16lo(v.x); y[1] = bf16hi(v.x); y[2] = bf16lo(v.y); y[3] = bf16hi(v.y);
}
Q3_DEV void store4(__half* p, int lane, const __half (&h)[4]) {
    const __half2 a = __halves2half2(h[0], h[1]), b = __halves2half2(h[2], h[3]);
    *reinterpret_cast<uint2*>(p + lane * 4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// ---------------------------------------------------------------- append
// One warp per head of one row: q heads are normed, rotated and stored in
// fp16; k heads are normed, rotated and packed, v heads packed, into the
// position's place of the row's block table.
template <typename Tin>
__global__ void __launch_bounds__(128) kv4_append_kernel(const Kv4AppendArgs a)
{
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x;
    const int hh = blockIdx.y * 4 + warp;                // q heads, then k heads, then v heads
    if (hh >= a.n_q + 2 * a.n_kv) return;
    const bool is_q = hh < a.n_q, is_k = !is_q && hh < a.n_q + a.n_kv;
    const int kvh = is_k ? hh - a.n_q : hh - a.n_q - a.n_kv;
    __half* q_dst = a.q_out ? a.q_out + ((size_t)t * a.n_q + hh) * D : nullptr;
    __half* kv_dst = a.kv_out ? a.kv_out + (((size_t)t * 2 + (is_k ? 0 : 1)) * a.n_kv + kvh) * D : nullptr;
    __half* dst = is_q ? q_dst : kv_dst;
    const int pos = a.row_pos[t];
    if (pos < 0 || pos >= a.rope_len) {                  // a padding row, or one past the rotation table
        const __half z[4] = {__half(), __half(), __half(), __half()};
        if (dst) store4(dst, lane, z);
        if (pos >= 0 && lane == 0) report(a.status, Q3_STATUS_BLOCK_RANGE);
        return;
    }
    float y[4];
    load4(static_cast<const Tin*>(a.qkv) + (size_t)t * a.qkv_stride + (size_t)hh * D, lane, y);
    if (is_q || is_k)
        head_norm_rope(y, is_q ? a.q_gain : a.k_gain, a.rope + (size_t)pos * (D / 2), a.eps, lane);
    if (is_q) {
        if (!dst) return;
        bool bad = false;
        const __half h[4] = {to_f16(y[0], bad), to_f16(y[1], bad), to_f16(y[2], bad), to_f16(y[3], bad)};
        store4(dst, lane, h);
        if (bad) report(a.status, Q3_STATUS_F16_RANGE);
        return;
    }
    uint32_t codes;
    __half scale, bias, val[4];
    if (!kv4_pack(y, codes, scale, bias, val)) report(a.status, Q3_STATUS_F16_RANGE);
    if (dst) store4(dst, lane, val);
    const int slot = a.row_slot[t], at = pos / 32;
    const int blk = slot >= 0 && slot < a.n_slots && at < a.max_blocks ? a.tables[(size_t)slot * a.max_blocks + at] : -1;
    if (blk < 0 || blk >= a.n_blocks) {
        if (lane == 0) report(a.status, Q3_STATUS_BLOCK_RANGE);
        return;
    }
    uint8_t* tile = a.kv + (((size_t)blk * 2 + (is_k ? 0 : 1)) * a.n_kv + kvh) * KV4_TILE;
    if (is_k) kv4_store_k(tile, pos % 32, codes, scale, bias, lane);
    else kv4_store_v(tile, pos % 32, codes, scale, bias, lane);
}

// ---------------------------------------------------------------- attention, a row and head at a time
// Four warps take positions in turn, a lane four dimensions; each warp keeps
// the running maximum, sum and output of its positions and they are merged in
// warp order.
constexpr int AW = 4;

template <typename Tq, typename To>
Q3_DEV void attend_row(const Tq* q, To* out, int ctx, int kvh, const int* table, int n_kv, const uint8_t* kv,
                       int n_blocks, int* status)
{
    __shared__ float s_m[AW], s_l[AW], s_o[AW][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float qv[4];
    load4(q, lane, qv);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    const float scale = 1.4426950408889634f * 0.08838834764831845f;
    for (int p = warp; p < ctx; p += AW) {
        const int blk = table[p / 32];
        if (blk < 0 || blk >= n_blocks) {
            if (lane == 0) report(status, Q3_STATUS_BLOCK_RANGE);
            continue;
        }
        const uint8_t* kt = kv + ((size_t)blk * 2 * n_kv + kvh) * KV4_TILE;
        __half k[4], v[4];
        kv4_load_k(kt, p % 32, lane, k);
        kv4_load_v(kt + (size_t)n_kv * KV4_TILE, p % 32, lane, v);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fmaf(qv[e], __half2float(k[e]), s);
        s = warp_allsum(s) * scale;
        const float mn = fmaxf(m, s), alpha = exp2f(m - mn), w = exp2f(s - mn);
        m = mn;
        l = l * alpha + w;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = o[e] * alpha + w * __half2float(v[e]);
    }
    if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
    for (int e = 0; e < 4; ++e) s_o[warp][lane * 4 + e] = o[e];
    __syncthreads();
    const int d = threadIdx.x;
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int w = 0; w < AW; ++w) M = fmaxf(M, s_m[w]);
    if (M != -INFINITY)
        for (int w = 0; w < AW; ++w) {
            const float e = exp2f(s_m[w] - M);
            L = fmaf(s_l[w], e, L);
            O = fmaf(s_o[w][d], e, O);
        }
    const float v = L > 0.f ? O / L : 0.f;
    bool bad = false;
    if (sizeof(To) == 2) reinterpret_cast<__half*>(out)[d] = to_f16(v, bad);
    else reinterpret_cast<float*>(out)[d] = v;
    if (bad) report(status, Q3_STATUS_F16_RANGE);
}

template <typename Tq, typename To>
__global__ void __launch_bounds__(AW * 32) kv4_decode_kernel(const Kv4DecodeArgs a)
{
    grid_dep_wait();
    const int t = blockIdx.y, h = blockIdx.x;
    const int slot = a.row_slot[t];
    int ctx = a.row_pos[t] + 1;
    if (ctx > 0 && (slot < 0 || slot >= a.n_slots || ctx > a.max_blocks * 32)) {
        if (threadIdx.x == 0) report(a.status, Q3_STATUS_BLOCK_RANGE);
        ctx = 0;
    }
    attend_row(static_cast<const Tq*>(a.q) + (size_t)t * a.q_stride + h * D, static_cast<To*>(a.out) + ((size_t)t * a.n_q + h) * D,
               ctx, h / (a.n_q / a.n_kv), a.tables + (size_t)max(slot, 0) * a.max_blocks, a.n_kv, a.kv, a.n_blocks, a.status);
}

__global__ void __launch_bounds__(AW * 32) kv4_prefill_kernel(const Kv4PrefillArgs a)
{
    grid_dep_wait();
    const int t = blockIdx.y, h = blockIdx.x;
    int i = 0;
    while (i < a.ns && !(a.seq_rows[i] <= t && t < a.seq_rows[i + 1])) ++i;
    if (i == a.ns) return;                               // a row of no sequence
    const int slot = a.seq_slot ? a.seq_slot[i] : i;
    int ctx = a.seq_pos[i] + t - a.seq_rows[i] + 1;
    if (ctx > 0 && (slot < 0 || slot >= a.n_slots || ctx > a.max_blocks * 32)) {
        if (threadIdx.x == 0) report(a.status, Q3_STATUS_BLOCK_RANGE);
        ctx = 0;
    }
    attend_row(a.q + (size_t)t * a.q_stride + h * D, a.out + ((size_t)t * a.n_q + h) * D, ctx, h / (a.n_q / a.n_kv),
               a.tables + (size_t)max(slot, 0) * a.max_blocks, a.n_kv, a.kv, a.n_blocks, a.status);
}

}  // namespace

cudaError_t launch_kv4_append(const Launch& L, const Kv4AppendArgs& a, int type)
{
    const dim3 grid(a.T, (a.n_q + 2 * a.n_kv + 3) / 4);
    switch (type) {
    case Q3_TYPE_F32: return launch_ex(L, kv4_append_kernel<float>, grid, dim3(128), a);
    case Q3_TYPE_F16: return launch_ex(L, kv4_append_kernel<__half>, grid, dim3(128), a);
    default: return launch_ex(L, kv4_append_kernel<__nv_bfloat16>, grid, dim3(128), a);
    }
}

cudaError_t launch_kv4_decode(const Launch& L, const Kv4DecodeArgs& a, int q_type, int out_type)
{
    const dim3 grid(a.n_q, a.T), block(AW * 32);
    if (q_type == Q3_TYPE_F32)
        return out_type == Q3_TYPE_F32 ? launch_ex(L, kv4_decode_kernel<float, float>, grid, block, a)
                                       : launch_ex(L, kv4_decode_kernel<float, __half>, grid, block, a);
    return out_type == Q3_TYPE_F32 ? launch_ex(L, kv4_decode_kernel<__half, float>, grid, block, a)
                                   : launch_ex(L, kv4_decode_kernel<__half, __half>, grid, block, a);
}

cudaError_t launch_kv4_prefill(const Launch& L, const Kv4PrefillArgs& a)
{
    return launch_ex(L, kv4_prefill_kernel, dim3(a.n_q, a.T), dim3(AW * 32), a);
}

}  // namespace q3
