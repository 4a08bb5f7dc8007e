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
// Alternatives: the pass keeps only the maximum of each lane's values of a
// round of loads (a slot: 16 values, 32 of the 16-bit types).  The k-th largest
// of the CTA's 256 lane maxima bounds the row's k-th from below, so at most the
// slots that reach it, about k of 10,000, are read again and ranked: a warp
// keeps the best 32 it has seen as a list sorted over its lanes, takes single
// candidates by insertion and many at once as a sorted batch, and lists merge
// pairwise (element i against 31 - i, then five exchange steps).  Whole keys
// order (value, then index), so ranks do not depend on the schedule, and rows in
// rising order or of one value cost what others do.
//
// Rows of few are split over the CTAs of a cluster, merged through
// distributed shared memory: no workspace, no second launch.
//
// 2,048 rows of 151,936 f32 with 5 alternatives: 214 us, 5.8 TB/s of the logits
// (lists kept in the pass took 337); in bf16 130 us, 4.8 TB/s, where the values'
// instructions count for as much as their bytes; one row with 20: 10.9 us, a chain of
// load, merge and exchange latencies (24).
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace q3 {

namespace {

namespace cg = cooperative_groups;

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int NL = 4;                                    // 16-byte loads a lane has in flight
constexpr int SLOTS = 40;                                // a lane's slots: V = 151,936 in f32 has 38 rounds
constexpr float LOG2E = 1.4426950408889634f;

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
// the same of plain values
Q3_DEV void exchange(float& c, int j, bool larger) {
    const float o = __shfl_xor_sync(0xffffffffu, c, j);
    c = larger ? fmaxf(c, o) : fminf(c, o);
}
Q3_DEV void sort32(float& c, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int j = size >> 1; j > 0; j >>= 1) exchange(c, j, ((lane & j) == 0) == ((lane & size) == 0));
}
Q3_DEV void merge32(float& list, float other, int lane) {
    list = fmaxf(list, __shfl_sync(0xffffffffu, other, 31 - lane));
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) exchange(list, j, (lane & j) == 0);
}
// eight lists into the first, pairwise
template <typename C>
Q3_DEV void merge8(C (&c)[8], int lane) {
#pragma unroll
    for (int half = 4; half > 0; half >>= 1)
#pragma unroll
        for (int i = 0; i < half; ++i) merge32(c[i], c[i + half], lane);
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
    const float sc = a.m == M ? 1.f : a.m == -INFINITY ? 0.f : fast_ex2((a.m - M) * LOG2E);
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
    if (N == 1) {
        const float d = v[0] - m, e = fast_ex2(d * LOG2E);
        a.s += e;
        a.t = fmaf(fmaxf(d, -1000.f), e, a.t);
        return;
    }
    const uint64_t nm = pair_of(-m, -m), l2e = pair_of(LOG2E, LOG2E);
    uint64_t s = pair_of(0.f, 0.f), t = s;
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        const uint64_t d = add2(pair_of(v[i], v[i + 1]), nm);
        const float2 u = halves_of(mul2(d, l2e)), dd = halves_of(d);
        const uint64_t e = pair_of(fast_ex2(u.x), fast_ex2(u.y));
        s = add2(s, e);
        // e is 0 from -127 on; -inf * 0 would not be
        t = fma2(pair_of(fmaxf(dd.x, -1000.f), fmaxf(dd.y, -1000.f)), e, t);
    }
    const float2 ss = halves_of(s), tt = halves_of(t);
    a.s += ss.x + ss.y;
    a.t += tt.x + tt.y;
}

// The candidates among 16 values, none below `bound`, join the warp's list;
// index(i): the place of this lane's value i in the row, or -1.
// kth: the list's k-th entry.
template <int N, typename Index>
Q3_DEV void add_candidates(Cand& list, Cand& kth, int k, float bound, const float (&v)[N], Index index, int lane) {
    uint32_t left = 0;                                   // values that may still pass
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = index(i);
        const Cand c{key_of(v[i]), at};
        if (at >= 0 && !(v[i] < bound) && before(c, kth)) left |= 1u << i;
    }
    for (;;) {
        const uint32_t who = __ballot_sync(0xffffffffu, left != 0);
        if (!who) return;
        Cand c = none();
        int ci = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)                      // the lane's best
            if (left >> i & 1) {
                const Cand o{key_of(v[i]), index(i)};
                if (before(o, c)) { c = o; ci = i; }
            }
        if (!before(c, kth)) { c = none(); left = 0; }
        if (__popc(who) >= 2) {
            left &= ~(1u << ci);
            sort32(c, lane);
            merge32(list, c, lane);
        } else {
            const int src = __ffs(who) - 1;
            if (lane == src) left &= ~(1u << ci);
            c = shfl(c, src);
            if (!before(c, kth)) continue;
            insert(list, c, lane);
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
    Cand list[8][32];          // of the warps; in CTA 0 then of the cluster's CTAs
    Sums sums[8];
    float maxima[WARPS][32];   // the lanes' maxima, sorted in each warp
    float slot[SLOTS][THREADS];
};
static_assert(WARPS == 8, "merge8");

template <typename T>
__global__ void __launch_bounds__(THREADS, 4) logprobs_kernel(const LogprobArgs a, int C)
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
    // what a row has before its first and after its last whole word: a value a lane
    const bool ends = rank == 0 && warp == 0;
    const int rest = a.V - tail, end_at = lane < head ? lane : lane - head < rest ? tail + lane - head : -1;
    float end_v[1] = {-INFINITY};
    if (ends && end_at >= 0) {
        end_v[0] = Vec<T>::one(x + end_at);
        add_values(sums, end_v, end_v[0]);
    }

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
    // round n of loads belongs to slot n / per_slot
    const int rounds = (w1 - w0 + NL * 32 - 1) / (NL * 32), per_slot = (rounds + SLOTS - 1) / SLOTS;
    float most = -INFINITY, slot_max = -INFINITY;        // of the lane, of its current slot
    int in_slot = 0, slot = 0;
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
            slot_max = fmaxf(slot_max, cm);
            add_values(sums, v, cm);
        }
        if (k && (++in_slot == per_slot || at + NL * 32 >= w1)) {
            sm.slot[slot++][threadIdx.x] = slot_max;
            most = fmaxf(most, slot_max);
            slot_max = -INFINITY;
            in_slot = 0;
        }
    }
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
    Cand list = none();
    if (k) {
        // the bound: the k-th largest of the lanes' maxima (-inf where fewer
        // lanes hold a number: all may be among the k)
        const float lane_max = most;
        sort32(most, lane);
        sm.maxima[warp][lane] = most;
        __syncthreads();
        float lists[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) lists[i] = sm.maxima[i][lane];
        merge8(lists, lane);
        const float bound = __shfl_sync(0xffffffffu, lists[0], k - 1);
        Cand kth = none();
        if (ends) add_candidates(list, kth, k, bound, end_v, [&](int) { return end_at; }, lane);
        // every lane walks its slots; those that may hold a candidate are read again
        const int end = lane_max < bound ? 0 : slot;         // a lane below the bound has none
        for (int n = 0;; ++n) {
            for (; n < end; ++n) {
                const float v = sm.slot[n][threadIdx.x];
                if (v < bound) continue;
                const int first = w0 + n * per_slot * NL * 32 + lane;
                if (first < w1 && before(Cand{key_of(v), head + first * EPL}, kth)) break;
            }
            if (!__any_sync(0xffffffffu, n < end)) break;
            for (int p = 0; p < per_slot; ++p) {
                const int at = w0 + (n * per_slot + p) * NL * 32 + lane;
#pragma unroll
                for (int g = 0; g < NL / GL; ++g) {
                    float v[16];
                    auto word = [&](int l) { return at + (g * GL + l) * 32; };
#pragma unroll
                    for (int l = 0; l < GL; ++l) {
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (n < end && word(l) < w1) w = __ldg(xw + word(l));
                        Vec<T>::get(w, v + l * EPL);
                    }
                    add_candidates(list, kth, k, bound, v, [&](int i) {
                        const int w = word(i / EPL);
                        return n < end && w < w1 ? head + w * EPL + i % EPL : -1;
                    }, lane);
                }
            }
        }
        sm.list[warp][lane] = list;
    }
    __syncthreads();
    // the warps' in warp 0, then the CTAs' in CTA 0's
    auto merged = [&](int n) {
        if (!k) return;
        Cand c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = i < n ? sm.list[i][lane] : none();
        merge8(c, lane);
        list = c[0];
    };
    if (warp == 0) {
        sums = sm.sums[0];
        for (int w = 1; w < WARPS; ++w) join(sums, sm.sums[w]);
        merged(WARPS);
    }
    if (C > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();                                  // CTA 0 is done with its warps' lists
        if (warp == 0) {
            *cluster.map_shared_rank(&sm.list[rank][lane], 0) = list;
            if (lane == 0) *cluster.map_shared_rank(&sm.sums[rank], 0) = sums;
        }
        cluster.sync();
        if (rank || warp) return;
        sums = sm.sums[0];
        for (int c = 1; c < C; ++c) join(sums, sm.sums[c]);
        merged(C);
    }
    if (warp) return;

    const float logs = logf(sums.s);
    const bool empty = sums.m == -INFINITY && sums.s == 0.f;         // every token ruled out
    // m + log s would round at the size of m: 4e-3 where logits lie near 60,000
    auto lp = [&](float v) { return empty ? -INFINITY : (v - sums.m) - logs; };
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

// CTAs of a row: twice as many, up to 8, while SMs are left out and a warp keeps
// a full round of loads (64 rows of 151,936 f32 with 20 alternatives: 18.7 us
// in 4, 20.4 in 8; one row: 10.9 in 8, 12.5 in 4).
cudaError_t launch_logprobs(const Launch& L, const LogprobArgs& a, int type)
{
    const int64_t round = (int64_t)WARPS * 32 * NL * (type == Q3_TYPE_F32 ? 4 : 8);
    int C = 1;
    while (C < 8 && (int64_t)a.N * C < 152 && a.V > round * C) C *= 2;
    switch (type) {
    case Q3_TYPE_F32: return launch_t<float>(L, a, C);
    case Q3_TYPE_F16: return launch_t<__half>(L, a, C);
    default: return launch_t<__nv_bfloat16>(L, a, C);
    }
}

}  // namespace q3
