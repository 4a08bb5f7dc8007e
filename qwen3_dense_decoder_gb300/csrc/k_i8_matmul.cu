// k_i8_matmul.cu -- out[t][m] = (sum_k x[t][k] w[m][k]) xs[t] ws[m] over 8-bit
// codes on tcgen05, for more than a few rows of x.
//
// sm_103a has no integer kind of tcgen05.mma.  An int8 code is an fp16 number,
// and FP32 sums of products of two are exact up to 2^24: 1,024 products of 128 x
// 128.  So kind::f16 sums chunks of 1,024 inputs in tensor memory, and the
// epilogue's warps add the chunks as 32-bit integers in registers: the exact
// whole number, at the 16-bit rate, from 8-bit operands in memory.  Reading a chunk
// slows the products beside it (2,048 rows by 19,456 x 2,560: 134 us with codes
// spread evenly over their range, which take two chunks a tile, 118 with those of
// normal values, which take one), so pairs sum longer ones where the tokens allow it:
// no partial sum exceeds 128 sum |x|, known for every token and 1,024 inputs.
//
// A CTA (or with CG == 2 a pair of CTAs, each with its own 128 channels and half
// of the tokens) takes a tile of 128 CG channels by bn tokens:
//   TMA      int8 tiles of 128 channels and of the tokens by 128 inputs into a ring
//   warps 0..3, 4..7  expand every other stage to fp16: the tokens' codes in shared
//               memory (operand B), then the channels' in tensor memory (operand A;
//               a thread owns a TMEM lane, a channel).  For pairs a kernel before
//               this one has expanded the tokens' codes, once for all channel tiles
//   one thread issues the products (of a pair, the first CTA's for both)
//   warps 8..15 add chunks, then scale and store
// Weights pass through shared memory once as bytes and never as fp16.  With
// fewer tiles than SMs a cluster of CTAs shares a tile's inputs (splits) and joins
// the whole-number sums through distributed shared memory: the same number.
#include <cooperative_groups.h>
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace q3 {

namespace {

constexpr int THREADS = 640;
constexpr int BM = 128;                          // channels of a CTA
constexpr int STAGE_K = 128;                     // inputs of a stage
constexpr int CHUNK = 8;                         // stages that FP32 sums exactly: 1,024 inputs
constexpr int MAX_NA = 4;                        // A's expanded stages
constexpr int MAX_NS = 8;                        // of either ring
constexpr int A_RAW = BM * STAGE_K;
constexpr uint32_t TMEM_COLS = 512, A_COLS = STAGE_K / 2;
constexpr int CHUNK_K = CHUNK * STAGE_K;
constexpr int TMA_WARP = 16, MMA_WARP = 17, PLAN_WARP = 18;
// registers of a thread by warpgroup; 640 threads launch with 96
constexpr int R_EXPAND = 72, R_EPILOGUE = 144, R_ISSUE = 48, R_LAUNCH = 96;
static_assert(2 * R_EXPAND + 2 * R_EPILOGUE + R_ISSUE <= 5 * R_LAUNCH, "registers");

constexpr size_t MAX_SMEM = 227 * 1024;
constexpr int I8_SMS = 152;

struct I8GemmArgs {
    I8MatmulArgs a;
    int bn, splits, ns, nb;          // tokens of a tile, CTAs that share its inputs, ring stages: codes, B in fp16
    int m_tiles, n_tiles;
    const int* l1;                   // pairs: [1,024 inputs][T] sum |x|
};

struct Bars {
    uint64_t raw_full[MAX_NS], raw_empty[MAX_NS];
    uint64_t full[MAX_NA], a_empty[MAX_NA], b_empty[MAX_NS];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint64_t plan_full[2], plan_empty[2];
    uint32_t plan[2][4];                     // bit i: a chunk ends with input 1,024 (i + 1); two units
    uint32_t tmem;
    int abort;
};

// bytes of a stage of the ring of codes and of B's in fp16; all of it with the
// barriers and what alignment may take
constexpr int raw_bytes(int cg, int bn) { return A_RAW + (cg == 1 ? bn * STAGE_K : 0); }
constexpr int half_bytes_of(int cg, int bn) { return bn / cg * STAGE_K * 2; }
constexpr size_t smem_bytes(int cg, int bn, int ns, int nb) {
    return (size_t)ns * raw_bytes(cg, bn) + (size_t)nb * half_bytes_of(cg, bn) + sizeof(Bars) + 1024;
}

// A's stages in what two accumulators leave of tensor memory: with two (bn 192) the
// expanding waits for the products, with three (160) it does not
constexpr __host__ __device__ int a_stages(int bn) { return bn > 160 ? 2 : bn > 128 ? 3 : MAX_NA; }

// Stages of the rings: as many as shared memory takes
struct Rings { int ns, nb; };
constexpr Rings rings(int cg, int bn) {
    Rings r{3, 3};
    for (bool more = true; more;) {
        more = false;
        if (cg == 2 && r.nb < MAX_NS && smem_bytes(cg, bn, r.ns, r.nb + 1) <= MAX_SMEM) ++r.nb, more = true;
        if (r.ns < MAX_NS && smem_bytes(cg, bn, r.ns + 1, r.nb) <= MAX_SMEM) ++r.ns, more = true;
    }
    return r;
}

// Whether a wait on raw_full tells a stage from the one before it in its slot, ns
// stages earlier: a parity alone does not, so that the group that waits has to know
// of the earlier one's copy.  The groups take every other stage: with an even ns it
// was the group's own.  Else the group knows by its last stage, two earlier, which
// began with a place of A (and, not for pairs, of B) free: the products that many
// stages before that were done, and so every copy up to there.
constexpr bool copies_in_order(int cg, int bn, int ns, int nb) {
    const int na = a_stages(bn), places = cg == 1 && nb < na ? nb : na;
    return ns % 2 == 0 || ns >= places + 2;
}
constexpr bool all_in_order() {
    for (int cg = 1; cg <= 2; ++cg)
        for (int bn = 16 * cg; bn <= (cg == 2 ? 192 : 128); bn += 16 * cg) {
            const Rings r = rings(cg, bn);
            if (smem_bytes(cg, bn, r.ns, r.nb) > MAX_SMEM || !copies_in_order(cg, bn, r.ns, r.nb)) return false;
        }
    return true;
}
static_assert(all_in_order(), "a width whose rings leave the order of copies open");
static_assert(!copies_in_order(1, 64, 3, 3) && !copies_in_order(2, 96, 5, 5), "rings that leave it open");

template <int R> Q3_DEV void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(R)); }
template <int R> Q3_DEV void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(R)); }

// Bounded wait (in line: a call would keep the warpgroups from registers of their own)
Q3_DEV bool wait_long(uint64_t* bar, uint32_t parity, int* abort, int* status) {
    uint64_t t0 = 0;
    for (;;) {
        for (int i = 0; i < 512; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*(volatile int*)abort) return false;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > Q3_WAIT_LIMIT_NS) {
            if (status) set_status(status, Q3_STATUS_TIMEOUT);
            *(volatile int*)abort = 1;
            return false;
        }
    }
}
// What ends a role's copies or products on its way out, bounded too
Q3_DEV void wait_last(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bar, parity) && global_ns() - t0 < Q3_WAIT_LIMIT_NS) {}
}
// By a whole warp, of one mind about the outcome
Q3_DEV bool wait_warp(uint64_t* bar, uint32_t parity, Bars& b, int* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_long(bar, parity, &b.abort, status));
}
// arrive on CTA 0's barrier of the pair
template <int CG> Q3_DEV void arrive_first(uint64_t* bar) {
    if (CG == 1) {
        mbar_arrive(bar);
    } else {
        asm volatile("{\n\t.reg .b32 a;\n\t"
                     "mapa.shared::cluster.u32 a, %0, 0;\n\t"
                     "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}"
                     :: "r"(smem_u32(bar)) : "memory");
    }
}
// D[tmem] (+)= A[tmem] B[smem], of one CTA or of a pair
template <int CG> Q3_DEV void mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    if (CG == 1) {
        tc_mma_f16_ts(d, a, b, idesc, add);
    } else {
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                     :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
    }
}
// arrive, on both CTAs' barriers of a pair, once the products issued so far are done
template <int CG> Q3_DEV void commit(uint64_t* bar) {
    if (CG == 1) {
        tc_commit(bar);
    } else {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     :: "r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
    }
}
template <int CG> Q3_DEV void alloc(uint32_t* dst) {
    if (CG == 1) {
        tmem_alloc(dst, TMEM_COLS);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(dst)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG> Q3_DEV void dealloc(uint32_t t) {
    if (CG == 1) tmem_dealloc(t, TMEM_COLS);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(t), "r"(TMEM_COLS) : "memory");
}

Q3_DEV void expand16(const uint4& w, uint32_t* r) {
    expand4(w.x, r[0], r[1]);
    expand4(w.y, r[2], r[3]);
    expand4(w.z, r[4], r[5]);
    expand4(w.w, r[6], r[7]);
}

// A place in a ring of n: the slot, the parity of its use, whether it is the first use
struct Ring {
    uint32_t n, slot = 0, phase = 0;
    bool first = true;
    Q3_DEV explicit Ring(uint32_t n) : n(n) {}
    Q3_DEV void next() {
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
            first = false;
        }
    }
};

Q3_DEV uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
Q3_DEV void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <typename O> Q3_DEV void put(O* p, float v, bool& bad);
template <> Q3_DEV void put<float>(float* p, float v, bool&) { *p = v; }
template <> Q3_DEV void put<__half>(__half* p, float v, bool& bad) { *p = to_f16(v, bad); }
template <> Q3_DEV void put<__nv_bfloat16>(__nv_bfloat16* p, float v, bool&) { *p = __float2bfloat16_rn(v); }

// A thread's sums of one channel and `n` tokens from t0 (FP32), scaled and stored
template <typename O, int ACC>
Q3_DEV void store_sums(const I8MatmulArgs& a, const int (&acc)[ACC], const float (&xs)[ACC / 32], int64_t m, int t0, int n, float ws, bool& bad)
{
    const bool live = m < a.M;
    O* p = static_cast<O*>(a.out) + (int64_t)t0 * a.out_stride + m;
#pragma unroll
    for (int j = 0; j < ACC; ++j) {
        const float x = __shfl_sync(0xffffffffu, xs[j / 32], j % 32);
        if (j < n && live) put<O>(p, __int_as_float(acc[j]) * x * ws, bad);
        p += a.out_stride;
    }
}

// x's codes as fp16 rows, Kp apart, operand B of the pairs, and sum |x| of every
// 1,024 of a row (l1: [1,024 inputs][T]), a warp's each
__global__ void __launch_bounds__(256) i8_expand_kernel(const int8_t* x, int64_t stride, int T, int K, __half* out, int64_t Kp, int* l1)
{
    grid_dep_wait();
    grid_dep_launch();                           // the product's set-up overlaps this
    const int lane = threadIdx.x & 31, chunks = (K + CHUNK_K - 1) / CHUNK_K;
    const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), t = task / chunks;
    if (t >= T) return;
    const int c = (int)(task % chunks);
    const int8_t* row = x + t * stride;
    uint4 w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int k = c * CHUNK_K + h * 512 + lane * 16;
        w[h] = make_uint4(0, 0, 0, 0);
        if (k + 16 <= K) {
            w[h] = ldg_nc_v4(row + k);
        } else {
            uint32_t* v = reinterpret_cast<uint32_t*>(&w[h]);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (k + e < K) v[e >> 2] |= (uint32_t)(uint8_t)row[k + e] << (8 * (e & 3));
        }
    }
    __half2 sum = __float2half2_rn(0.f);         // at most 16 x 128 a half: exact
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int k = c * CHUNK_K + h * 512 + lane * 16;
        uint32_t r[8];
        expand16(w[h], r);
        if (k < K) {
            uint4* o = reinterpret_cast<uint4*>(out + t * Kp + k);
            o[0] = make_uint4(r[0], r[1], r[2], r[3]);
            o[1] = make_uint4(r[4], r[5], r[6], r[7]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __hadd2(sum, __habs2(*reinterpret_cast<const __half2*>(&r[i])));
    }
    const int whole = __reduce_add_sync(0xffffffffu, (int)(__low2float(sum) + __high2float(sum)));
    if (lane == 0) l1[(int64_t)c * T + t] = whole;
}

template <int CG>
__global__ void __launch_bounds__(THREADS, 1)
i8_gemm_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx, const I8GemmArgs p)
{
    constexpr int ACC = CG == 2 ? 96 : 64;       // tokens of an epilogue warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const I8MatmulArgs& a = p.a;
    const int rows_b = p.bn / CG;                // tokens of this CTA's B operand
    const int stage_bytes = raw_bytes(CG, p.bn), half_bytes = half_bytes_of(CG, p.bn);
    uint8_t* half = smem + p.ns * stage_bytes;   // operand B in fp16: nb stages, each 64 inputs and 64 more
    Bars& b = *reinterpret_cast<Bars*>(half + p.nb * half_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int size = CG == 2 ? 2 : p.splits;     // CTAs of a cluster
    const int rank = size > 1 ? (int)(blockIdx.x % size) : 0;
    const int na = a_stages(p.bn);
    const uint32_t t_a = TMEM_COLS - na * A_COLS;    // tensor memory: two accumulators, then A's stages
    int* status = a.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.ns; ++s) {
            mbar_init(&b.raw_full[s], 1);
            mbar_init(&b.raw_empty[s], 4);
        }
        for (int c = 0; c < MAX_NA; ++c) {
            mbar_init(&b.full[c], 4 * CG);
            mbar_init(&b.a_empty[c], 1);
        }
        for (int c = 0; c < p.nb; ++c) mbar_init(&b.b_empty[c], 1);
        for (int c = 0; c < 2; ++c) {
            mbar_init(&b.acc_full[c], 1);
            mbar_init(&b.acc_empty[c], 8 * CG);
        }
        for (int c = 0; c < 2; ++c) {
            mbar_init(&b.plan_full[c], 1);
            mbar_init(&b.plan_empty[c], rank == 0 ? 9 : 8);      // the epilogue's warps and the products'
        }
        mbar_init(&b.drain, 1);
        b.abort = 0;
        fence_barrier_init();
        prefetch_tmap(&tw);
        prefetch_tmap(&tx);
    }
    if (warp == MMA_WARP) alloc<CG>(&b.tmem);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cg::this_cluster().sync();      // both CTAs' barriers are there
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    grid_dep_wait();

    // units of work: (weight tile, token tile), token tiles first; a split cluster
    // has one and shares its stages
    const int kt = (a.K + STAGE_K - 1) / STAGE_K;
    const int split = CG == 1 && p.splits > 1 ? rank : 0, splits = CG == 1 ? p.splits : 1;
    const int s0 = (int)((int64_t)kt * split / splits), s1 = (int)((int64_t)kt * (split + 1) / splits);
    const int units = p.m_tiles * p.n_tiles, first = blockIdx.x / size, stride = gridDim.x / size;
    const int stages = s1 - s0, most = (stages + CHUNK - 1) / CHUNK;
    const bool planned = CG == 2 && most > 1;    // else chunks of CHUNK stages

    if (warp < 8) {
        // ---------------- expanding: a warpgroup takes every other stage
        reg_dec<R_EXPAND>();
        const int mine = warp >> 2, row = (warp & 3) * 32 + lane;
        const bool live = row < rows_b;
        const uint32_t swz = (uint32_t)(row & 7);
        const uint32_t src0 = smem_u32(smem) + row * 128, dst0 = smem_u32(half) + row * 128;
        const uint32_t ta0 = tmem + ((uint32_t)(warp & 3) * 32 << 16) + t_a;
        Ring raw(p.ns), a_at(na), b_at(p.nb);
        int turn = 0;
        bool ok = true;
        for (int u = first; u < units && ok; u += stride) {
            for (int s = 0; s < stages && ok; ++s, turn ^= 1, raw.next(), a_at.next(), b_at.next()) {
                if (turn != mine) continue;
                if (!(ok = wait_warp(&b.raw_full[raw.slot], raw.phase, b, status))) break;
                const uint32_t src = src0 + raw.slot * stage_bytes;
                uint4 w[2][4];
                auto load = [&](uint4 (&v)[4], uint32_t from, int h) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = lds16(from + (((h * 4 + j) ^ swz) << 4));
                };
                if (CG == 2) load(w[0], src, 0);
                else if (live) load(w[0], src + A_RAW, 0);
                if (CG == 1 && !(ok = b_at.first || wait_warp(&b.b_empty[b_at.slot], b_at.phase ^ 1, b, status))) break;
#pragma unroll
                for (int h = 0; h < (CG == 1 ? 2 : 0); ++h) {
                    if (h == 0) { if (live) load(w[1], src + A_RAW, 1); }
                    else load(w[0], src, 0);
                    if (live) {
                        const uint32_t dst = dst0 + b_at.slot * half_bytes + h * (half_bytes / 2);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t r[8];
                            expand16(w[h][j], r);
                            sts16(dst + (((2 * j) ^ swz) << 4), r[0], r[1], r[2], r[3]);
                            sts16(dst + (((2 * j + 1) ^ swz) << 4), r[4], r[5], r[6], r[7]);
                        }
                    }
                }
                if (!(ok = a_at.first || wait_warp(&b.a_empty[a_at.slot], a_at.phase ^ 1, b, status))) break;
                tc_fence_after();
                const uint32_t ta = ta0 + a_at.slot * A_COLS;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 0) load(w[1], src, 1);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t r[16];
                        expand16(w[h][2 * i], r);
                        expand16(w[h][2 * i + 1], r + 8);
                        tmem_st_32x32b_x16(ta + h * 32 + i * 16, r);
                    }
                }
                if (CG == 1) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    arrive_first<CG>(&b.full[a_at.slot]);
                    mbar_arrive(&b.raw_empty[raw.slot]);
                }
            }
        }
        // the products' last arrivals on this CTA's barriers
        for (int i = 0; i < na && ok; ++i, a_at.next())
            if (!a_at.first) wait_warp(&b.a_empty[a_at.slot], a_at.phase ^ 1, b, status);
        for (int i = 0; i < (CG == 1 ? p.nb : 0) && ok; ++i, b_at.next())
            if (!b_at.first) wait_warp(&b.b_empty[b_at.slot], b_at.phase ^ 1, b, status);
    } else if (warp < TMA_WARP) {
        // ---------------- epilogue: quadrant warp % 4 of the lanes, half the columns
        reg_inc<R_EPILOGUE>();
        const int part = (warp - 8) >> 2, cols = p.bn / 2;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) * 32 << 16);
        Ring acc_at(2), plan_at(2);
        bool ok = true, bad = false;
        for (int u = first; u < units && ok; u += stride) {
            const int nt = u % p.n_tiles, mt = u / p.n_tiles;
            const int64_t m = (int64_t)mt * (BM * CG) + (CG == 2 ? rank * BM : 0) + (warp & 3) * 32 + lane;
            const int t0 = nt * p.bn + part * cols;
            int chunks = most;
            if (planned) {
                if (!(ok = wait_warp(&b.plan_full[plan_at.slot], plan_at.phase, b, status))) break;
                chunks = 1;
                for (int i = 0; i < most; i += 32) chunks += i + 1 < most ? __popc(b.plan[plan_at.slot][i >> 5]) : 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.plan_empty[plan_at.slot]);
                plan_at.next();
            }
            // the first chunk as the FP32 that it is, whole numbers from the second on
            // (every share has a stage, so that there is a first)
            int acc[ACC];
            for (int c = 0; c < chunks && ok; ++c, acc_at.next()) {
                const uint32_t d = acc_at.slot;
                if (!(ok = wait_warp(&b.acc_full[d], acc_at.phase, b, status))) break;
                tc_fence_after();
                const uint32_t from = lanes + d * p.bn + part * cols;
                if (c == 0) {
#pragma unroll
                    for (int g = 0; g < ACC / 16; ++g)
                        if (g * 16 < cols) tmem_ld_32x32b_x16(from + g * 16, *reinterpret_cast<uint32_t(*)[16]>(acc + g * 16));
                    tmem_ld_wait();
                } else {
                    if (c == 1)
#pragma unroll
                        for (int j = 0; j < ACC; ++j) acc[j] = __float2int_rn(__int_as_float(acc[j]));
#pragma unroll
                    for (int g = 0; g < ACC / 16; ++g) {
                        if (g * 16 < cols) {
                            uint32_t r[16];
                            tmem_ld_32x32b_x16(from + g * 16, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[g * 16 + j] += __float2int_rn(__uint_as_float(r[j]));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_first<CG>(&b.acc_empty[d]);
            }
            if (!ok) break;
            if (CG == 1 && splits > 1) {
                // this CTA's share of the sums, [token][channel], where its operands were
                int* red = reinterpret_cast<int*>(smem);
#pragma unroll
                for (int j = 0; j < ACC; ++j)
                    if (j < cols) red[(part * cols + j) * BM + (warp & 3) * 32 + lane] = chunks == 1 ? __float2int_rn(__int_as_float(acc[j])) : acc[j];
                break;
            }
            if (chunks > 1)
#pragma unroll
                for (int j = 0; j < ACC; ++j) acc[j] = __float_as_int((float)acc[j]);
            float xs[ACC / 32];
#pragma unroll
            for (int i = 0; i < ACC / 32; ++i) {
                const int t = t0 + i * 32 + lane;
                xs[i] = i * 32 + lane < cols && t < a.T ? a.xs[t] : 0.f;
            }
            const float ws = m < a.M ? a.ws[m] : 0.f;
            const int n = min(cols, a.T - t0);
            switch (a.out_type) {
            case Q3_TYPE_F32: store_sums<float>(a, acc, xs, m, t0, n, ws, bad); break;
            case Q3_TYPE_F16: store_sums<__half>(a, acc, xs, m, t0, n, ws, bad); break;
            default: store_sums<__nv_bfloat16>(a, acc, xs, m, t0, n, ws, bad);
            }
        }
        if (bad && status) set_status(status, Q3_STATUS_F16_RANGE);
    } else {
        reg_dec<R_ISSUE>();
        if (warp == TMA_WARP) {
            Ring raw(p.ns), b_at(p.nb);
            bool ok = true;
            for (int u = first; u < units && ok; u += stride) {
                const int nt = u % p.n_tiles, mt = u / p.n_tiles;
                const int m0 = mt * (BM * CG) + (CG == 2 ? rank * BM : 0), n0 = nt * p.bn + (CG == 2 ? rank * rows_b : 0);
                for (int s = s0; s < s1; ++s, raw.next(), b_at.next()) {
                    if (!(ok = raw.first || wait_warp(&b.raw_empty[raw.slot], raw.phase ^ 1, b, status))) break;
                    if (CG == 2 && !(ok = b_at.first || wait_warp(&b.b_empty[b_at.slot], b_at.phase ^ 1, b, status))) break;
                    uint8_t* dst = smem + raw.slot * stage_bytes;
                    uint64_t* bar = &b.raw_full[raw.slot];
                    if (elect_one()) {
                        mbar_arrive_expect_tx(bar, CG == 1 ? stage_bytes : stage_bytes + half_bytes);
                        tma_load_2d(dst, &tw, bar, s * STAGE_K, m0);
                        if (CG == 1) {
                            tma_load_2d(dst + A_RAW, &tx, bar, s * STAGE_K, n0);
                        } else {
                            uint8_t* to = half + b_at.slot * half_bytes;
                            tma_load_2d(to, &tx, bar, s * STAGE_K, n0);
                            tma_load_2d(to + half_bytes / 2, &tx, bar, s * STAGE_K + 64, n0);
                        }
                    }
                    __syncwarp();
                }
            }
            for (int i = 0; i < (CG == 2 ? p.nb : 0) && ok; ++i, b_at.next())      // the products' last arrivals
                if (!b_at.first) wait_warp(&b.b_empty[b_at.slot], b_at.phase ^ 1, b, status);
            if (!ok)                             // copies still under way end before the CTA does
                for (int i = 0; i < p.ns; ++i, raw.next())
                    if (!raw.first) wait_last(&b.raw_full[raw.slot], raw.phase ^ 1);
        } else if (warp == MMA_WARP && (CG == 1 || rank == 0)) {
            const uint32_t idesc = idesc_f16_f32(BM * CG, 0) | ((uint32_t)(p.bn >> 3) << 17);
            Ring a_at(na), b_at(p.nb), acc_at(2), plan_at(2);
            bool ok = true;
            for (int u = first; u < units && ok; u += stride) {
                if (planned && !(ok = wait_warp(&b.plan_full[plan_at.slot], plan_at.phase, b, status))) break;
                for (int at = 0; at < stages && ok; acc_at.next()) {
                    int end = at / CHUNK;                // the chunk's last 1,024 inputs
                    if (planned)
                        while (end + 1 < most && !(b.plan[plan_at.slot][end >> 5] >> (end & 31) & 1)) ++end;
                    const int n = min((end + 1) * CHUNK, stages) - at;
                    at += n;
                    if (!(ok = acc_at.first || wait_warp(&b.acc_empty[acc_at.slot], acc_at.phase ^ 1, b, status))) break;
                    tc_fence_after();
                    const uint32_t d = tmem + acc_at.slot * p.bn;
                    for (int k = 0; k < n; ++k, a_at.next(), b_at.next()) {
                        if (!(ok = wait_warp(&b.full[a_at.slot], a_at.phase, b, status))) break;
                        tc_fence_after();
                        const uint64_t desc = smem_desc_sw128(smem_u32(half) + b_at.slot * half_bytes);
                        const uint32_t ta = tmem + t_a + a_at.slot * A_COLS, next64 = half_bytes >> 5;
                        if (elect_one()) {
#pragma unroll
                            for (int j = 0; j < STAGE_K / 16; ++j)
                                mma<CG>(d, ta + j * 8, desc + (j & 3) * 2 + (j >> 2) * next64, idesc, k > 0 || j > 0);
                            commit<CG>(&b.a_empty[a_at.slot]);
                            commit<CG>(&b.b_empty[b_at.slot]);
                            if (k + 1 == n) commit<CG>(&b.acc_full[acc_at.slot]);
                        }
                        __syncwarp();
                    }
                }
                if (planned && ok) {
                    if (lane == 0) mbar_arrive(&b.plan_empty[plan_at.slot]);
                    plan_at.next();
                }
            }
            if (!ok) {                           // as do products
                if (elect_one()) commit<CG>(&b.drain);
                __syncwarp();
                wait_last(&b.drain, 0);
            }
        }
        else if (warp == PLAN_WARP && planned) {
            // where each unit's chunks end: as late as 128 sum |x| of every token stays
            // within 2^24
            Ring plan_at(2);
            bool ok = true;
            for (int u = first; u < units && ok; u += stride, plan_at.next()) {
                if (!(ok = plan_at.first || wait_warp(&b.plan_empty[plan_at.slot], plan_at.phase ^ 1, b, status))) break;
                const int t0 = u % p.n_tiles * p.bn, t1 = min(t0 + p.bn, a.T);
                uint32_t* plan = b.plan[plan_at.slot];
                uint32_t bits = 0;
                int sum = 0;
                for (int c0 = 0; c0 < most; c0 += 4) {
                    int m[4] = {0, 0, 0, 0};
                    for (int t = t0 + lane; t < t1; t += 32)
#pragma unroll
                        for (int i = 0; i < 4; ++i) m[i] = max(m[i], p.l1[(int64_t)min(c0 + i, most - 1) * a.T + t]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = c0 + i, v = (int)__reduce_max_sync(0xffffffffu, (uint32_t)m[i]);
                        if (c >= most) break;
                        if (c > 0 && sum + v > (1 << 24) / 128) {
                            bits |= 1u << ((c - 1) & 31);      // the chunk before ends with c - 1
                            sum = 0;
                        }
                        sum += v;
                        if (c > 0 && ((c & 31) == 0 || c + 1 == most)) {
                            if (lane == 0) plan[(c - 1) >> 5] = bits;
                            bits = 0;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.plan_full[plan_at.slot]);
            }
        }
        __syncwarp();
    }
    // The roles have ended and all warps of a warpgroup are here before its registers
    // change again; what follows is for all warps alike.
    __syncthreads();
    if (CG == 1) {
        if (warp >= TMA_WARP) reg_inc<R_EXPAND>();
        else if (warp >= 8) reg_dec<R_EXPAND>();
    }
    if (CG == 1 && splits > 1) {
        // the cluster's sums, a share of the tokens each
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        if (first < units && !b.abort) {
            const int nt = first % p.n_tiles, mt = first / p.n_tiles;
            const int c0 = p.bn * rank / splits, c1 = p.bn * (rank + 1) / splits;
            bool bad = false;
            for (int i = c0 * 32 + threadIdx.x; i < c1 * 32; i += THREADS) {
                const int col = i >> 5, t = nt * p.bn + col;
                const int64_t m = (int64_t)mt * BM + (i & 31) * 4;
                if (t >= a.T || m >= a.M) continue;
                int4 v[8];                       // all shares' loads together
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < splits) v[r] = *reinterpret_cast<const int4*>(cluster.map_shared_rank(reinterpret_cast<int*>(smem), r) + i * 4);
                int4 s = v[0];
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < splits) s.x += v[r].x, s.y += v[r].y, s.z += v[r].z, s.w += v[r].w;
                const int sums[4] = {s.x, s.y, s.z, s.w};
                const float xs = a.xs[t];
                for (int e = 0; e < 4; ++e) {
                    if (m + e >= a.M) break;
                    const float v = (float)sums[e] * xs * a.ws[m + e];
                    const int64_t at = (int64_t)t * a.out_stride + m + e;
                    switch (a.out_type) {
                    case Q3_TYPE_F32: put(static_cast<float*>(a.out) + at, v, bad); break;
                    case Q3_TYPE_F16: put(static_cast<__half*>(a.out) + at, v, bad); break;
                    default: put(static_cast<__nv_bfloat16*>(a.out) + at, v, bad);
                    }
                }
            }
            if (bad && status) set_status(status, Q3_STATUS_F16_RANGE);
        }
    }
    if (size > 1) cg::this_cluster().sync();     // no CTA's memory is in use by another
    if (warp == MMA_WARP) dealloc<CG>(tmem);
}

template <int CG>
cudaError_t launch_cg(const Launch& L, const CUtensorMap& tw, const CUtensorMap& tx, const I8GemmArgs& p)
{
    // the attribute and the registers that the warpgroups' split counts on, once a device
    static std::atomic<int> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        cudaFuncAttributes at;
        if ((e = cudaFuncGetAttributes(&at, i8_gemm_kernel<CG>)) != cudaSuccess) return e;
        if (at.numRegs < R_LAUNCH) return cudaErrorLaunchOutOfResources;
        if ((e = cudaFuncSetAttribute(i8_gemm_kernel<CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MAX_SMEM)) != cudaSuccess) return e;
        ready[dev].store(1, std::memory_order_release);
    }
    const int size = CG == 2 ? 2 : p.splits, units = p.m_tiles * p.n_tiles;
    const int ctas = CG == 1 && p.splits > 1 ? units : std::min(units, I8_SMS / size);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas * size));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes(CG, p.bn, p.ns, p.nb);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 2 : 1;
    if (L.counter) ++*L.counter;
    return cudaLaunchKernelEx(&cfg, i8_gemm_kernel<CG>, tw, tx, p);
}

}  // namespace

namespace {
bool few_rows(int T, int M, int K) { return T <= 16 || (T <= I8_FEW_ROWS && (int64_t)M * K <= 16 << 20); }
// Whether pairs can be the quicker by i8_plan's times.  They are not where one wave of
// single CTAs takes at most six stages: 7.8 us and 0.64 a stage against 10 and 0.29.
// Once true it stays so for larger sizes, as a workspace's bound has to.
bool may_pair(int T, int M, int K)
{
    const int64_t kt = (K + STAGE_K - 1) / STAGE_K, tiles = (M + 127ll) / 128 * ((T + 127) / 128);
    return !few_rows(T, M, K) && (kt > 6 || tiles > I8_SMS);
}
int64_t pair_workspace(int T, int K) { return i8_copy_bytes(T, K) + (K + 1023ll) / 1024 * T * (int64_t)sizeof(int); }
}  // namespace

// What a pair keeps outside the SM: x's copy and sum |x|
int64_t i8_workspace(const I8Plan& q, int T, int K) { return q.cg == 2 ? pair_workspace(T, K) : 0; }
int64_t i8_workspace_bound(int T, int M, int K) { return may_pair(T, M, K) ? pair_workspace(T, K) : 0; }

// How a product is shared out: the quickest by a model of what was measured (us, device
// time; of 132 products, 17 to 2,048 tokens by 1,024 x 2,048 to 34,816 x 5,120, nine in
// ten lie within 15 % of it, the others between 0.79 and 1.24 times):
//  - a wave of tiles takes its stages, 0.56 us and 0.6 ns a token each for one CTA,
//    0.28 us and 0.4 ns for a pair, or 0.33 and 2 ns for the tokens beyond 128;
//  - setting up takes 6.5 us and 10 ns a token, joining a cluster's sums 1.5 us and
//    12 ns a token more; a pair 9 us, and the expansion before it 1 us and its bytes.
// Few tokens take launch_i8_few's: 2.5 us and up, but its expansion of x, a warp's own,
// grows with the tokens (32 by 19,456 x 2,560: 23.8 us, by 2,560 x 4,096 8.3 to 9.2; in
// pairs or a cluster 18 and 10).  Above 16 Mi codes the step from 16 to 17 tokens costs
// up to 11 us (7,168 x 5,120: 10.1 to 20.2; 5,120 x 17,408: 24.3 to 34.5).
I8Plan i8_plan(int T, int M, int K)
{
    I8Plan q{};
    if (few_rows(T, M, K)) return q;
    const int64_t kt = (K + STAGE_K - 1) / STAGE_K, m_tiles = (M + 127ll) / 128, m_pairs = (M + 255ll) / 256;
    double best = 1e30;
    auto take = [&](double us, int cg, int bn, int splits) {
        if (us >= best) return;
        best = us;
        q.cg = cg; q.bn = bn; q.splits = splits;
    };
    for (int bn = 32; bn <= 192 && may_pair(T, M, K); bn += 32) {
        const int64_t waves = (m_pairs * ((T + bn - 1) / bn) + I8_SMS / 2 - 1) / (I8_SMS / 2);
        const double stage = bn <= 128 ? 0.28 + 0.0004 * bn : 0.33 + 0.002 * (bn - 128);
        take(10 + 7.5e-7 * T * K + waves * kt * stage, 2, bn, 1);
    }
    // token tiles of equal width; clusters of one CTA an SM in one wave, a little under
    // cudaOccupancyMaxActiveClusters' numbers (76, 46, 36, 28, 23, 15 and 15: with 20 of
    // seven CTAs 64 by 2,560 x 9,728 took 29 us, with 20 of six 16)
    constexpr int MOST_CLUSTERS[9] = {0, I8_SMS, 74, 44, 34, 26, 22, 14, 14};
    for (int n = (T + 127) / 128; n <= (T + 127) / 128 + 2; ++n) {
        const int bn = ((T + n - 1) / n + 15) / 16 * 16;
        const int64_t tiles = m_tiles * ((T + bn - 1) / bn);
        for (int splits = 1; splits <= 8; ++splits) {
            if (splits > 1 && (tiles > MOST_CLUSTERS[splits] || kt < 2 * splits)) break;
            const int64_t waves = (tiles + I8_SMS - 1) / I8_SMS;
            take(6.5 + 0.01 * bn + waves * ((kt + splits - 1) / splits) * (0.56 + 0.0006 * bn) + (splits > 1 ? 1.5 + 0.012 * bn : 0), 1, bn, splits);
        }
    }
    const Rings r = rings(q.cg, q.bn);
    q.ns = r.ns; q.nb = r.nb;
    return q;
}

cudaError_t launch_i8_expand(const Launch& L, const I8MatmulArgs& a, void* workspace)
{
    cudaLaunchConfig_t cfg = {};
    const int64_t tasks = (int64_t)a.T * ((a.K + CHUNK_K - 1) / CHUNK_K);
    cfg.gridDim = dim3((unsigned)((tasks + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.counter) ++*L.counter;
    return cudaLaunchKernelEx(&cfg, i8_expand_kernel, a.x, a.x_stride, a.T, a.K, static_cast<__half*>(workspace), i8_copy_row(a.K),
                              i8_sums(workspace, a.T, a.K));
}

cudaError_t launch_i8_gemm(const Launch& L, const CUtensorMap& tw, const CUtensorMap& tx, const I8MatmulArgs& a, const I8Plan& q, void* workspace)
{
    // what tcgen05.mma takes: 16 k tokens for 128 channels, 32 k for a pair's 256
    if (q.bn % (16 * q.cg) || q.bn < 16 * q.cg || q.bn > (q.cg == 2 ? 192 : 128)) return cudaErrorInvalidValue;
    if (!copies_in_order(q.cg, q.bn, q.ns, q.nb)) return cudaErrorInvalidValue;
    I8GemmArgs p{};
    p.a = a;
    if (q.cg == 2) p.l1 = i8_sums(workspace, a.T, a.K);
    p.bn = q.bn; p.splits = q.splits; p.ns = q.ns; p.nb = q.nb;
    p.m_tiles = (a.M + 128 * q.cg - 1) / (128 * q.cg);
    p.n_tiles = (a.T + q.bn - 1) / q.bn;
    return q.cg == 2 ? launch_cg<2>(L, tw, tx, p) : launch_cg<1>(L, tw, tx, p);
}

}  // namespace q3
