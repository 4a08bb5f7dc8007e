// k_logprobs.cu -- log probabilities of given tokens from logits rows, with
// the distribution's entropy and its most probable tokens.
//
// Row x of V logits, m its maximum, s = sum exp(x_i - m):
//   log p_i = x_i - m - log s,   H = log s - (sum (x_i - m) exp(x_i - m)) / s
// (a logit of -inf has probability 0 and adds nothing to H).
#include "common.cuh"
#include "kernels.h"

namespace q3 {

namespace {

constexpr int LPT = 256;

Q3_DEV float value(const float* p, int i) { return p[i]; }
Q3_DEV float value(const __half* p, int i) { return __half2float(p[i]); }
Q3_DEV float value(const __nv_bfloat16* p, int i) { return __bfloat162float(p[i]); }

// (a, i) before (b, j): the larger value, the lower index among equals; what
// is not a number comes after every number
Q3_DEV bool before(float a, int i, float b, int j) {
    const bool na = isnan(a), nb = isnan(b);
    if (na || nb) return na == nb ? i < j : nb;
    return a > b || (a == b && i < j);
}

Q3_DEV float block_sum(float v, float* red) {
    v = warp_allsum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < LPT / 32; ++w) t += red[w];
    return t;
}

template <typename T>
__global__ void __launch_bounds__(LPT) logprobs_kernel(const LogprobArgs a)
{
    __shared__ float red[LPT / 32], s_v[LPT / 32];
    __shared__ int s_i[LPT / 32];
    grid_dep_wait();
    const int r = blockIdx.x;
    const T* x = static_cast<const T*>(a.logits) + (size_t)r * a.stride;
    // top-k by passes: the first of those after the last one taken
    float pv = INFINITY, m = -INFINITY;
    int pi = -1;
    bool first = true;
    auto next = [&](float& bv, int& bi) {
        bv = 0.f; bi = -1;
        for (int i = threadIdx.x; i < a.V; i += LPT) {
            const float v = value(x, i);
            if (!first && !before(pv, pi, v, i)) continue;
            if (bi < 0 || before(v, i, bv, bi)) { bv = v; bi = i; }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
            if (oi >= 0 && (bi < 0 || before(ov, oi, bv, bi))) { bv = ov; bi = oi; }
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) { s_v[threadIdx.x >> 5] = bv; s_i[threadIdx.x >> 5] = bi; }
        __syncthreads();
        bv = s_v[0]; bi = s_i[0];
        for (int w = 1; w < LPT / 32; ++w)
            if (s_i[w] >= 0 && (bi < 0 || before(s_v[w], s_i[w], bv, bi))) { bv = s_v[w]; bi = s_i[w]; }
    };
    float bv;
    int bi;
    next(bv, bi);
    m = bv;
    float s = 0.f, xs = 0.f, nan = 0.f;
    for (int i = threadIdx.x; i < a.V; i += LPT) {
        const float v = value(x, i), d = v - m, e = expf(d);
        if (isnan(v)) nan = 1.f;
        s += e;
        if (e > 0.f) xs = fmaf(d, e, xs);
    }
    s = block_sum(s, red);
    xs = block_sum(xs, red);
    nan = block_sum(nan, red);
    float lse = m + logf(s), H = logf(s) - xs / s;
    if (m == -INFINITY) { lse = -INFINITY; H = 0.f; }        // every token ruled out
    if (nan > 0.f || m == INFINITY) lse = H = NAN;
    auto lp = [&](float v) { return m == -INFINITY && nan == 0.f ? -INFINITY : v - lse; };
    if (threadIdx.x == 0) {
        if (a.logprob) {
            const int tok = a.targets[r];
            float v = 0.f;
            if (tok >= a.V || tok < -1) {
                v = NAN;
                if (a.status) set_status(a.status, Q3_STATUS_TOKEN_RANGE);
            } else if (tok >= 0) {
                v = lp(value(x, tok));
            }
            a.logprob[r] = v;
        }
        if (a.entropy) a.entropy[r] = H;
    }
    for (int k = 0; k < a.top; ++k) {
        if (k) next(bv, bi);
        if (threadIdx.x == 0) {
            if (a.top_ids) a.top_ids[(size_t)r * a.top + k] = bi;
            if (a.top_logprob) a.top_logprob[(size_t)r * a.top + k] = lp(bv);
        }
        pv = bv; pi = bi; first = false;
    }
}

}  // namespace

cudaError_t launch_logprobs(const Launch& L, const LogprobArgs& a, int type)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.N);
    cfg.blockDim = dim3(LPT);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.counter) ++*L.counter;
    switch (type) {
    case Q3_TYPE_F32: return cudaLaunchKernelEx(&cfg, logprobs_kernel<float>, a);
    case Q3_TYPE_F16: return cudaLaunchKernelEx(&cfg, logprobs_kernel<__half>, a);
    default: return cudaLaunchKernelEx(&cfg, logprobs_kernel<__nv_bfloat16>, a);
    }
}

}  // namespace q3
