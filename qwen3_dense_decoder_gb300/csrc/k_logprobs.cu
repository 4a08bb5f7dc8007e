// k_logprobs.cu -- log probabilities of given tokens from logits rows, with
// the distribution's entropy and its most probable tokens, in one pass.
//
// Row x of V logits, m its maximum, s = sum exp(x_i - m):
//   log p_i = x_i - m - log s,   H = log s - (sum (x_i - m) exp(x_i - m)) / s
// (a logit of -inf has probability 0 and adds nothing to H).  Every lane keeps
// m, s and t = sum (x_i - m) exp(x_i - m) of the values it has read; raising m
// to m' turns (s, t) into exp(m - m') (s, t + (m - m') s).  Lanes, warps and
// CTAs merge by the same rule in a fixed order.
//
// Alternatives: a warp keeps the best 32 it has seen as a list sorted over its
// lanes.  A lane compares the maximum of 16 new values with the list's
// k-th; only when one passes does the warp offer candidates, singly (an
// insertion) or, when many lanes have one, as a sorted batch merged with the
// list.  On data in no special order that is about k ln(n / 512) insertions a
// warp.  Lists merge pairwise: element i against 31 - i, then five exchange
// steps.  Whole keys order (value, then index), so ranks do not depend on the
// schedule.
//
// Rows of few are split over the CTAs of a cluster, merged through
// distributed shared memory: no workspace, no second launch.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace q3 {

namespace {

namespace cg = cooperative_groups;

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int NL = 4;                                    // 16-byte loads a lane has in flight
constexpr float LOG2E = 1.4426950408889634f;

Q3_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- candidates
// key: a number that orders as the value does, 1 for a NaN, 0 for no candidate
struct Cand {
    uint32_t key;
    int idx;
};
Q3_DEV uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);        // -0 ranks as 0
    if (isnan(v)) return 1u;
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
Q3_DEV float value_of(uint32_t key) {
    if (key <= 1u) return NAN;
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
Q3_DEV bool before(const Cand& a, const Cand& b) { return a.key > b.key || (a.key == b.key && a.idx < b.idx); }
Q3_DEV Cand none() { return Cand{0u, 0x7fffffff}; }
Q3_DEV Cand shfl(const Cand& c, int src) {
    return Cand{__shfl_sync(0xffffffffu, c.key, src), __shfl_sync(0xffffffffu, c.idx, src)};
}
// lanes l and l ^ j exchange: the one whose bit says so keeps the better
Q3_DEV void exchange(Cand& c, int j, bool better) {
    const Cand o{__shfl_xor_sync(0xffffffffu, c.key, j), __shfl_xor_sync(0xffffffffu, c.idx, j)};
    if (before(o, c) == better) c = o;
}
// 32 candidates, one a lane, best first
Q3_DEV void sort32(Cand& c, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int j = size >> 1; j > 0; j >>= 1) exchange(c, j, ((lane & j) == 0) == ((lane & size) == 0));
}
// list and other both sorted: list becomes the best 32 of both
Q3_DEV void merge32(Cand& list, const Cand& other, int lane) {
    const Cand r = shfl(other, 31 - lane);
    if (before(r, list)) list = r;
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) exchange(list, j, (lane & j) == 0);
}
// one candidate, the same in every lane
Q3_DEV void insert(Cand& list, const Cand& c, int lane) {
    const int at = __popc(__ballot_sync(0xffffffffu, before(list, c)));
    const Cand up{__shfl_up_sync(0xffffffffu, list.key, 1), __shfl_up_sync(0xffffffffu, list.idx, 1)};
    if (lane == at) list = c;
    else if (lane > at) list = up;
}

// ---------------------------------------------------------------- sums
struct Sums {
    float m, s, t;
};
// (s, t) moved to the maximum M >= a.m
Q3_DEV void raise(Sums& a, float M) {
    const float sc = a.m == M ? 1.f : a.m == -INFINITY ? 0.f : ex2((a.m - M) * LOG2E);
    a.t = sc == 0.f ? 0.f : a.m == M ? a.t : (a.t + (a.m - M) * a.s) * sc;
    a.s *= sc;
    a.m = M;
}
Q3_DEV void join(Sums& a, Sums b) {
    const float M = fmaxf(a.m, b.m);
    raise(a, M);
    raise(b, M);
    a.s += b.s;
    a.t += b.t;
}

// values of one lane, padded with -inf
template <int N>
Q3_DEV void add_values(Sums& a, const float (&v)[N], float cm) {
    if (cm > a.m) raise(a, cm);
    const float m = a.m == -INFINITY ? 0.f : a.m;        // -inf - -inf is not a number
    float s[2] = {0.f, 0.f}, t[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = v[i] - m, e = ex2(d * LOG2E);
        s[i & 1] += e;
        t[i & 1] = fmaf(fmaxf(d, -1000.f), e, t[i & 1]); // e is 0 from -127 on; -inf * 0 would not be
    }
    a.s += s[0] + s[1];
    a.t += t[0] + t[1];
}

// the candidates among a chunk's values (index(i) of value i, or -1: none) join the list
template <int N, typename Index>
Q3_DEV void add_candidates(Cand& list, Cand& kth, int k, const float (&v)[N], Index index, int lane) {
    uint32_t left = 0;                                   // values that may still pass
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = index(i);
        if (at >= 0 && before(Cand{key_of(v[i]), at}, kth)) left |= 1u << i;
    }
    for (;;) {
        Cand best = none();
        int bi = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (left >> i & 1) {
                const Cand c{key_of(v[i]), index(i)};
                if (before(c, best)) { best = c; bi = i; }
            }
        if (!before(best, kth)) { best = none(); left = 0; }
        const uint32_t who = __ballot_sync(0xffffffffu, best.idx != 0x7fffffff);
        if (!who) return;
        if (__popc(who) >= 6) {
            left &= ~(1u << bi);
            sort32(best, lane);
            merge32(list, best, lane);
        } else {
            const int src = __ffs(who) - 1;
            insert(list, shfl(best, src), lane);
            if (lane == src) left &= ~(1u << bi);
        }
        kth = shfl(list, k - 1);
    }
}

template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static Q3_DEV void get(const uint4& w, float* v) {
        v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
    }
    static Q3_DEV float one(const float* p) { return *p; }
};
template <> struct Vec<__half> {
    static constexpr int N = 8;
    static Q3_DEV void get(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            v[2 * i] = f.x; v[2 * i + 1] = f.y;
        }
    }
    static Q3_DEV float one(const __half* p) { return __half2float(*p); }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static Q3_DEV void get(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[2 * i] = bf16lo(u[i]); v[2 * i + 1] = bf16hi(u[i]); }
    }
    static Q3_DEV float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};

struct Shared {
    Cand list[WARPS][32];
    Sums sums[WARPS];
};

// the lists of n warps (a power of two), warp w holding its own, into warp 0's
Q3_DEV void merge_lists(Shared& sm, Cand& list, int warp, int lane, int n) {
    for (int half = n >> 1; half > 0; half >>= 1) {
        if (warp >= half && warp < 2 * half) sm.list[warp][lane] = list;
        __syncthreads();
        if (warp < half) merge32(list, sm.list[warp + half][lane], lane);
        __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 3) logprobs_kernel(const LogprobArgs a, int C)
{
    constexpr int EPL = Vec<T>::N, GL = 16 / EPL;        // words of a group of 16 values
    __shared__ Shared sm;
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % C;
    const int64_t r = blockIdx.x / C;
    const T* x = static_cast<const T*>(a.logits) + r * a.stride;

    // the target's logit is fetched while the row streams
    float xt = 0.f;
    int tok = -1;
    if (rank == 0 && threadIdx.x == 0 && a.logprob) {
        tok = a.targets[r];
        if (tok >= 0 && tok < a.V) xt = Vec<T>::one(x + tok);
    }

    // [0, head) single values, then whole 16-byte words, then single values
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)), a.V);
    const int words = (a.V - head) / EPL, tail = head + words * EPL;
    const uint4* xw = reinterpret_cast<const uint4*>(x + head);

    const int k = a.top;
    Sums sums{-INFINITY, 0.f, 0.f};
    Cand list = none(), kth = none();
    // the filter on values: kth's, or nothing passes it without a list
    auto single = [&](int from, int n) {
        const int i = from + lane;
        const float v[1] = {lane < n ? Vec<T>::one(x + i) : -INFINITY};
        if (lane < n) add_values(sums, v, v[0]);
        if (k) add_candidates(list, kth, k, v, [&](int) { return lane < n ? i : -1; }, lane);
    };
    if (rank == 0 && warp == 0 && head) single(0, head);

    // this warp's share of the words, a multiple of a full load each
    const int shares = C * WARPS, share = rank * WARPS + warp;
    const int per = ((words + shares - 1) / shares + 31) / 32 * 32;
    const int w0 = min(share * per, words), w1 = min(w0 + per, words);
    uint4 next[NL];
    auto fetch = [&](int at) {
#pragma unroll
        for (int l = 0; l < NL; ++l) {
            const int w = at + l * 32 + lane;
            if (w < w1) next[l] = ldg_nc_v4(xw + w);
        }
    };
    if (w0 < w1) fetch(w0);
    for (int at = w0; at < w1; at += NL * 32) {
        uint4 cur[NL];
#pragma unroll
        for (int l = 0; l < NL; ++l) cur[l] = next[l];
        if (at + NL * 32 < w1) fetch(at + NL * 32);
#pragma unroll
        for (int g = 0; g < NL / GL; ++g) {
            const int ag = at + g * GL * 32 + lane;
            float v[16];
#pragma unroll
            for (int l = 0; l < GL; ++l) {
                Vec<T>::get(cur[g * GL + l], v + l * EPL);
                if (ag + l * 32 >= w1)
#pragma unroll
                    for (int e = 0; e < EPL; ++e) v[l * EPL + e] = -INFINITY;
            }
            float cm = v[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) cm = fmaxf(cm, v[i]);
            if (k) {
                // past the list's k-th by value, or not comparable with it
                const bool pass = kth.key <= 1u || !(cm <= value_of(kth.key));
                if (__any_sync(0xffffffffu, pass))
                    add_candidates(list, kth, k, v, [&](int i) {
                        const int w = ag + i / EPL * 32;
                        return w < w1 ? head + w * EPL + i % EPL : -1;
                    }, lane);
            }
            add_values(sums, v, cm);
        }
    }
    if (rank == C - 1 && warp == WARPS - 1 && tail < a.V) single(tail, a.V - tail);

    // lanes, then warps, then CTAs
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums b{__shfl_xor_sync(0xffffffffu, sums.m, o), __shfl_xor_sync(0xffffffffu, sums.s, o),
                     __shfl_xor_sync(0xffffffffu, sums.t, o)};
        // both lanes join in the same order, so all lanes end with one value
        Sums lo = (lane & o) ? b : sums;
        join(lo, (lane & o) ? sums : b);
        sums = lo;
    }
    if (lane == 0) sm.sums[warp] = sums;
    if (k) merge_lists(sm, list, warp, lane, WARPS);
    else __syncthreads();
    if (warp == 0) {
        sums = sm.sums[0];
        for (int w = 1; w < WARPS; ++w) join(sums, sm.sums[w]);
    }
    if (C > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        __syncthreads();
        if (warp == 0) {
            sm.list[0][lane] = list;
            if (lane == 0) sm.sums[0] = sums;
        }
        cluster.sync();
        Sums all = sums;
        if (rank == 0) {
            list = none();
            if (k && warp < C) {
                const Cand* o = cluster.map_shared_rank(&sm.list[0][lane], warp);
                list = *o;
            }
            if (warp == 0)
                for (int c = 1; c < C; ++c) join(all, *cluster.map_shared_rank(&sm.sums[0], c));
        }
        cluster.sync();                                  // nobody's shared memory is read past here
        if (rank) return;
        if (k) merge_lists(sm, list, warp, lane, C);
        sums = all;
    }
    if (warp) return;

    const float logs = logf(sums.s);
    const bool empty = sums.m == -INFINITY && sums.s == 0.f;         // every token ruled out
    const float lse = empty ? -INFINITY : sums.m + logs;
    auto lp = [&](float v) { return empty ? -INFINITY : v - lse; };
    if (lane == 0) {
        if (a.entropy) a.entropy[r] = empty ? 0.f : logs - sums.t / sums.s;
        if (a.logprob) {
            if (tok >= a.V || tok < -1) {
                if (a.status) set_status(a.status, Q3_STATUS_TOKEN_RANGE);
                a.logprob[r] = NAN;
            } else {
                a.logprob[r] = tok < 0 ? 0.f : lp(xt);
            }
        }
    }
    if (lane < k) {
        if (a.top_ids) a.top_ids[r * k + lane] = list.idx;
        if (a.top_logprob) a.top_logprob[r * k + lane] = lp(value_of(list.key));
    }
}

template <typename T>
cudaError_t launch_t(const Launch& L, const LogprobArgs& a, int C)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.N * C);
    cfg.blockDim = dim3(THREADS);
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
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a, C);
}

}  // namespace

// CTAs of a row: 1, or as many of 2, 4, 8 as it takes to give every SM a few
// (four of 256 threads are resident) while a warp still has a full round of
// loads.
cudaError_t launch_logprobs(const Launch& L, const LogprobArgs& a, int type)
{
    const int64_t round = (int64_t)WARPS * 32 * NL * (type == Q3_TYPE_F32 ? 4 : 8);
    int C = 1;
    while (C < 8 && (int64_t)a.N * C < 4 * 152 && a.V > round * C) C *= 2;
    switch (type) {
    case Q3_TYPE_F32: return launch_t<float>(L, a, C);
    case Q3_TYPE_F16: return launch_t<__half>(L, a, C);
    default: return launch_t<__nv_bfloat16>(L, a, C);
    }
}

}  // namespace q3
