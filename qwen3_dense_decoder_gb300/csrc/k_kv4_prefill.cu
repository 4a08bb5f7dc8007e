// k_kv4_prefill.cu -- causal GQA attention of prefill rounds over the 4-bit
// cache on the tcgen05 tensor cores.  kv4_expand_kernel (k_kv4.cu) leaves an
// fp16 copy of the sequences' blocks and a list of query tiles, longest context
// first; a stored value is an fp16 number and q arrives in fp16, so both
// products run on single fp16 operands and only the softmax weights are rounded (once,
// to fp16: 11 bits, no finer than 2^-32 of the largest).
//
// Work item: R = 128 / G consecutive positions of one sequence for the G query
// heads of one KV head, as an MMA tile of 128 rows (row r = position r / G, head
// r % G).  Its context is walked in steps of 128 positions, half h of the CTA taking
// positions 64 h .. 64 h + 64 of each, with its own reference, sum and output;
// the halves are joined at an item's end.
//   S = Q K^T       tcgen05.mma, Q and K from shared memory, FP32 in tensor memory; both
//                   halves' 64 columns at once (64 alone take the time of 128)
//   P = 2^(S c - m) one thread a row, so nothing is exchanged; written over S.  m is the
//                   weights' reference, under the row's maximum (kv4.cuh)
//   O_h += P V      P from tensor memory, V read MN-major from shared memory
// A step's scores are made while the last one's weights are, and the halves'
// exponentials overlap each other and the products.  (A row shared by two threads
// spent 480 of 2,300 cycles a step on its maximum; scores issued only after the
// product before them left the softmax waiting for 1,600; one warp issuing both
// products took 1,550 cycles for 64 positions, with its commits, against the 512 they
// run.)  References are raised lazily: O and the sum are rescaled only when a score
// passes its own by KV4_HIGH, 2^8 above the maximum that set it.
//
// Items are dealt whole, longest first, where that comes out about even.  Else they
// are cut: the items in a row, their steps are shared out evenly, a CTA's share may
// begin and end inside an item, and a cut item's pieces leave reference, sum and FP32
// output in the workspace, where the warp that finishes a row range last joins them
// in order.  Cut where fewer than three items a CTA would take the longest CTA 12 steps
// more than an even share.  (Dealt and cut: 512 rows after 10,240 positions, 40/8
// heads, 123 and 88 us; 64 rows after 4,096, 32/8 heads, 30.8 and 23.2; 16 rows after
// 32,768, 221 and 68.  The other way: 256 rows after 2,000, 21.2 and 24.0; 2,048 rows,
// 35.7 and 47.9.)
//
// A step of 128 positions reads 64 KB of K and V: 1,024 cycles of an SM's 64 bytes, as
// many as its products take; it takes 1,450 with long contexts (512 rows after 10,240:
// 88 us, 1.25 PFLOP/s over the whole call, and 95 called without a pause, when 1.36 kW
// bring the clock from 2,070 to 1,850 MHz), 1,760 where a CTA has three items of nine
// steps (2,048 rows: 35.8 us, 0.96 PFLOP/s, either way).
//
// Roles (one CTA per SM; the next item's Q, K and scores are under way while an
// item ends):
//   warps 0..3, 4..7  softmax of half 0 and of half 1 (warp w: TMEM lanes 32 (w % 4)
//                     .. + 32); half 0 writes an item's output, both write a piece's
//   warps 8, 9        issue the score products and the PV products
//   warps 10, 11      fetch K (and Q) or V with TMA (blocks past the item's last
//                     position, or outside the pool, are read at a negative row and
//                     land as zeros)
// Tensor memory: two buffers of scores at 0 and 128, O_h at 256 + 128 h.  Every wait
// is bounded; a timeout sets the status word and the CTA winds down.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace q3 {

namespace {

constexpr int D = 128;
constexpr int BN = KV4_STEP;                 // positions of a step
constexpr int Q_ATOM = 128 * 128;            // 128 rows x 64 fp16, one swizzle atom column
constexpr int KV_ATOM = BN * 128;            // 128 rows x 64 fp16
constexpr int KV_TILE = 2 * KV_ATOM;
constexpr int NS = 2;                        // slots
constexpr int S_WARP = 8, PV_WARP = 9, K_WARP = 10;        // V: K_WARP + 1
constexpr int THREADS = 12 * 32;
constexpr uint32_t T_S = 0, T_O = 256;
constexpr int PART = (int)(KV4_PART_BYTES / 16);

struct alignas(1024) Smem {
    uint8_t q[2][2 * Q_ATOM];
    uint8_t k[NS][KV_TILE];
    uint8_t v[NS][KV_TILE];
    // by slot n % 2 of step n, phase n / 2: K and V landed; scores done (K's stage is
    // free); by half: weights stored; product done (V's stage and the scores are free)
    uint64_t k_load[NS], v_load[NS], s_full[NS], p_full[2][NS], pv_done[2][NS];
    uint64_t q_full[2], q_free[2];           // by item
    uint64_t ml_done[2], o_free, drain[2];
    float2 ml[2][128];                       // the halves' references and sums
    int2 cut[2];                             // where this CTA's share begins and ends: item, step
    uint32_t tmem;
    int abort;
};
constexpr size_t SMEM_BYTES = sizeof(Smem) + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

// fp16 A and B, FP32 accumulator; PV reads V MN-major (bit 16)
constexpr uint32_t IDESC_S = idesc_f16_f32(128, BN), IDESC_PV = idesc_f16_f32(128, 128) | (1u << 16);

// Bounded wait; the slow part is out of line, so that the roles' loops stay small
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, int* abort, int* status) {
    uint64_t t0 = 0;
    for (;;) {
        for (int i = 0; i < 512; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*(volatile int*)abort) return false;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > Q3_WAIT_LIMIT_NS) {
            set_status(status, Q3_STATUS_TIMEOUT);
            *(volatile int*)abort = 1;
            return false;
        }
    }
}
// By a whole warp, of one mind about the outcome: what follows needs all of its lanes
Q3_DEV bool wait_bar(uint64_t* bar, uint32_t parity, Smem& sm, int* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_long(bar, parity, &sm.abort, status));
}

// A CTA's work: n items or pieces of items
struct Work {
    int n, first, s0, s1;                    // the first piece's first step, the last one's end (0: the item's)
    int share;                               // cost between cuts; 0: whole items
};

struct Item {
    int row0, rows, pos0, seq, slot, kvh;
    int t0, t1, steps;                       // steps t0 .. t1 of the item's
    int tile;
};

// Item k of this CTA.  Number i n_kv + h is tile i of the list for KV head h, dealt in
// rows of gridDim.x, every other row backwards; of cut items, number h n_tiles + i.
Q3_DEV Item item_of(const Kv4PrefillArgs& p, const Work& w, int k) {
    Item it;
    if (w.share) {
        const int n = w.first + k, nt = *p.n_tiles;
        it.kvh = n / nt;
        it.tile = n - it.kvh * nt;
    } else {
        const int P = gridDim.x, n = k * P + ((k & 1) ? P - 1 - (int)blockIdx.x : (int)blockIdx.x);
        it.tile = n / p.n_kv;
        it.kvh = n - it.tile * p.n_kv;
    }
    const int4 t = p.tiles[it.tile];
    it.row0 = t.x; it.slot = t.y; it.pos0 = t.z & 0x1ffffff; it.rows = (int)((unsigned)t.z >> 25) + 1; it.seq = t.w;
    it.steps = (it.pos0 + it.rows - 1) / BN + 1;
    it.t0 = w.share && k == 0 ? w.s0 : 0;
    it.t1 = w.share && k == w.n - 1 && w.s1 ? w.s1 : it.steps;
    return it;
}

// This CTA's work (all threads)
Q3_DEV Work work_of(const Kv4PrefillArgs& p, Smem& sm) {
    const int P = gridDim.x, c = blockIdx.x, nt = p.n_tiles[0], cost = p.n_tiles[2];
    Work w{};
    if (cost == 0) {
        const int n = nt * p.n_kv, full = n / P;
        w.n = full + (((full & 1) ? P - 1 - c : c) < n % P ? 1 : 0);
        return w;
    }
    const int all = cost * p.n_kv;
    w.share = max((all + P - 1) / P, KV4_MIN_SHARE);
    if (c * w.share >= all) return w;
    // cut c is at cost c share; one within KV4_MIN_PIECE steps of an item's end moves there
    const int x[2] = {c * w.share, min((c + 1) * w.share, all)};
    for (int i = threadIdx.x; i < nt; i += THREADS) {
        const int start = p.starts[i], end = i + 1 < nt ? p.starts[i + 1] : cost;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = x[e] / cost, s = x[e] - h * cost - start;
            if (s >= 0 && s < end - start) {
                const int n = h * nt + i;
                sm.cut[e] = s < KV4_MIN_PIECE ? make_int2(n, 0)
                                              : s > end - start - KV4_TILE_COST - KV4_MIN_PIECE ? make_int2(n + 1, 0) : make_int2(n, s);
            }
        }
    }
    __syncthreads();
    const int2 lo = sm.cut[0], hi = sm.cut[1];
    w.first = lo.x; w.s0 = lo.y; w.s1 = hi.y;
    w.n = hi.x - lo.x + (hi.y > 0 ? 1 : 0);
    return w;
}

// The phase of step n's slot, and the one before
Q3_DEV uint32_t phase(uint32_t n) { return (n >> 1) & 1; }
Q3_DEV uint32_t phase_before(uint32_t n) { return ((n >> 1) & 1) ^ 1; }

// ---------------------------------------------------------------- MMA issuers
// A whole warp walks the loop and one lane issues, so descriptors and addresses
// stay in uniform registers.
Q3_DEV int steps_of(const Kv4PrefillArgs& p, const Work& w, int k) {
    const Item it = item_of(p, w, k);
    return __shfl_sync(0xffffffffu, it.t1 - it.t0, 0);
}

Q3_DEV void scores_role(const Kv4PrefillArgs& p, Smem& sm, uint32_t tmem, const Work& w, int* status) {
    const bool leader = elect_one();
    const uint64_t q0 = smem_desc_sw128(smem_u32(sm.q[0])), k0 = smem_desc_sw128(smem_u32(sm.k[0]));
    uint32_t n = 0;
    bool ok = true;
    for (int k = 0; k < w.n && ok; ++k) {
        const int steps = steps_of(p, w, k);
        const uint64_t qd = q0 + (uint32_t)(k & 1) * (2 * Q_ATOM >> 4);
        if (!(ok = wait_bar(&sm.q_full[k & 1], (k >> 1) & 1, sm, status))) break;
        for (int t = 0; t < steps; ++t, ++n) {
            const uint32_t slot = n & 1;
            if (!(ok = wait_bar(&sm.k_load[slot], phase(n), sm, status))) break;
            // the slot's last products have read the weights that lie over its scores
            if (n >= NS && !(ok = wait_bar(&sm.pv_done[0][slot], phase_before(n), sm, status))) break;
            if (n >= NS && !(ok = wait_bar(&sm.pv_done[1][slot], phase_before(n), sm, status))) break;
            tc_fence_after();
            const uint64_t kd = k0 + slot * (KV_TILE >> 4);
            const uint32_t d = tmem + T_S + slot * 128;
            if (leader) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    tc_mma_f16(d, qd + (((s >> 2) * Q_ATOM + (s & 3) * 32) >> 4), kd + (((s >> 2) * KV_ATOM + (s & 3) * 32) >> 4),
                               IDESC_S, s > 0);
                tc_commit(&sm.s_full[slot]);
            }
        }
        if (leader) tc_commit(&sm.q_free[k & 1]);
    }
    // nothing of this CTA's may still run on the tensor cores at deallocation
    if (leader) tc_commit(&sm.drain[0]);
    mbar_wait(&sm.drain[0], 0, status);
}

Q3_DEV void product_role(const Kv4PrefillArgs& p, Smem& sm, uint32_t tmem, const Work& w, int* status) {
    const bool leader = elect_one();
    const uint64_t v0 = smem_desc_sw128_mn(smem_u32(sm.v[0]), KV_ATOM);
    uint32_t n = 0;
    bool ok = true;
    for (int k = 0; k < w.n && ok; ++k) {
        const int steps = steps_of(p, w, k);
        // the last item's outputs are read out before this one's first products
        if (k > 0 && !(ok = wait_bar(&sm.o_free, (k - 1) & 1, sm, status))) break;
        for (int t = 0; t < steps; ++t, ++n) {
            const uint32_t slot = n & 1;
            if (!(ok = wait_bar(&sm.v_load[slot], phase(n), sm, status))) break;
            const uint64_t vd = v0 + slot * (KV_TILE >> 4);
            const uint32_t more = t > 0 ? 1u : 0u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!(ok = wait_bar(&sm.p_full[h][slot], phase(n), sm, status))) break;
                tc_fence_after();
                const uint32_t d = tmem + T_O + h * 128, a = tmem + T_S + slot * 128 + h * 64;
                if (leader) {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        tc_mma_f16_ts(d, a + s * 8, vd + ((4 * h + s) * 2048 >> 4), IDESC_PV, s > 0 ? 1u : more);
                    tc_commit(&sm.pv_done[h][slot]);
                }
            }
            if (!ok) break;
        }
    }
    if (leader) tc_commit(&sm.drain[1]);
    mbar_wait(&sm.drain[1], 0, status);
}

// ---------------------------------------------------------------- loaders
// which = 0: Q and K, 1: V.  A box of Q is R positions x G heads x 64
// dimensions.  Rows past the sequence read another's (or zeros past T); the last
// 128 - R G rows of a tile are never written.  What they give is not stored.
// A whole warp: a lane holds the block of one of 32 table entries, the next 32 under
// way (looked up step by step they took 1,100 of a step's 1,900 cycles), and four
// lanes fetch a step's four blocks.
Q3_DEV void load_role(const Kv4PrefillArgs& p, const CUtensorMap* tkv, const CUtensorMap* tq, Smem& sm, const Work& w, int which,
                      int* status) {
    constexpr int PER = BN / 32;
    const int G = p.n_q / p.n_kv, lane = threadIdx.x & 31;
    uint64_t* ld = which ? sm.v_load : sm.k_load;
    uint32_t n = 0, nq = 0;
    bool ok = true;
    for (int k = 0; k < w.n && ok; ++k) {
        const Item it = item_of(p, w, k);
        const int* table = p.tables + (size_t)it.slot * p.max_blocks;
        const int blocks = (it.pos0 + it.rows - 1) / 32 + 1;
        auto entry = [&](int i) { return i < blocks ? __ldg(table + i) : -1; };
        int chunk = it.t0 * PER >> 5, now = entry(32 * chunk + lane), next = entry(32 * chunk + 32 + lane);
        if (!which) {
            const int b = k & 1;
            if (k > 1 && !wait_bar(&sm.q_free[b], ((k >> 1) - 1) & 1, sm, status)) break;
            ++nq;
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm.q_full[b], 2 * p.rows_per_tile * G * 128);
#pragma unroll
                for (int h = 0; h < 2; ++h) tma_load_3d(sm.q[b] + h * Q_ATOM, tq, &sm.q_full[b], 64 * h, it.kvh * G, it.row0);
            }
        }
        for (int t = it.t0; t < it.t1; ++t, ++n) {
            const uint32_t slot = n & 1;
            if ((t * PER >> 5) != chunk) {
                ++chunk;
                now = next;
                next = entry(32 * chunk + 32 + lane);
            }
            const int i = t * PER + (lane & (PER - 1)), ph = __shfl_sync(0xffffffffu, now, i & 31);
            int row = -32;                               // the expansion has reported entries outside the pool
            if (ph >= 0 && ph < p.n_blocks) row = (((p.by_seq ? it.seq * p.max_blocks + i : ph) * 2 + which) * p.n_kv + it.kvh) * 32;
            if (n >= NS) {
                if (which) ok = wait_bar(&sm.pv_done[0][slot], phase_before(n), sm, status) && wait_bar(&sm.pv_done[1][slot], phase_before(n), sm, status);
                else ok = wait_bar(&sm.s_full[slot], phase_before(n), sm, status);
                if (!ok) break;
            }
            uint8_t* dst = (which ? sm.v[slot] : sm.k[slot]) + lane * 32 * 128;
            if (lane == 0) mbar_arrive_expect_tx(&ld[slot], KV_TILE);
            __syncwarp();
            if (lane < PER) {
                tma_load_2d(dst, tkv, &ld[slot], 0, row);
                tma_load_2d(dst + KV_ATOM, tkv, &ld[slot], 64, row);
            }
        }
    }
    // no copy of this CTA's may still be under way when it ends, even if another role gave up
    for (uint32_t i = n > NS ? n - NS : 0; i < n; ++i) mbar_wait(&ld[i & 1], phase(i), status);
    for (uint32_t i = nq > 2 ? nq - 2 : 0; i < nq; ++i) mbar_wait(&sm.q_full[i & 1], (i >> 1) & 1, status);
}

// ---------------------------------------------------------------- softmax + output
Q3_DEV void store32(__half* dst, const float (&v)[32], bool& bad) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint4 w;
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            __half2 h2;
            h2.x = to_f16(v[8 * e + 2 * f], bad);
            h2.y = to_f16(v[8 * e + 2 * f + 1], bad);
            (&w.x)[f] = *reinterpret_cast<uint32_t*>(&h2);
        }
        *reinterpret_cast<uint4*>(dst + e * 8) = w;
    }
}

// A cut item's pieces lie with consecutive CTAs: the first in its CTA's second
// place, the others in the first.  This warp has stored its rows of one; the last
// to come joins its rows of all, in the pieces' order.
Q3_DEV void join_pieces(const Kv4PrefillArgs& p, const Work& w, const Item& it, int half, int quad, int row, bool valid, __half* dst, bool& bad) {
    const int start = it.kvh * p.n_tiles[2] + p.starts[it.tile];
    const int c1 = (start + KV4_MIN_PIECE + w.share - 1) / w.share, c2 = (start + it.steps - KV4_MIN_PIECE) / w.share;
    const int pieces = c2 - c1 + 2;
    __threadfence();
    __syncwarp();
    int come = 0;
    if ((threadIdx.x & 31) == 0) come = atomicAdd(p.come + 8 * (c1 - 1) + 4 * half + quad, 1);
    if (__shfl_sync(0xffffffffu, come, 0) != pieces - 1) return;
    __threadfence();
    auto piece = [&](int j) { return p.parts + (size_t)(2 * (c1 - 1 + j) + (j ? 0 : 1)) * PART; };
    auto ml = [&](int j) { return __ldcg(reinterpret_cast<const float2*>(piece(j) + 32 * 128) + 128 * half + row); };
    if (!valid) return;                                  // the others have seen their own position
    float M = -INFINITY, L = 0.f;
    for (int j = 0; j < pieces; j += 4) {
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ml(min(j + i, pieces - 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float m = fmaxf(M, x[i].x);
            if (m == -INFINITY || j + i >= pieces) continue;
            L = L * fast_ex2(M - m) + x[i].y * fast_ex2(x[i].x - m);
            M = m;
        }
    }
    const float inv = 1.f / L;
#pragma unroll 1
    for (int c = 2 * half; c < 2 * half + 2; ++c) {
        float v[32] = {};
#pragma unroll 2
        for (int j = 0; j < pieces; ++j) {               // two pieces' loads under way
            const float2 x = ml(j);
            const float4* src = piece(j) + 8 * c * 128 + row;
            float4 o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __ldcg(src + e * 128);
            const float f = fast_ex2(x.x - M) * inv;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[4 * e] += f * o[e].x; v[4 * e + 1] += f * o[e].y; v[4 * e + 2] += f * o[e].z; v[4 * e + 3] += f * o[e].w;
            }
        }
        store32(dst + 32 * c, v, bad);
    }
}

Q3_DEV void softmax_role(const Kv4PrefillArgs& p, Smem& sm, uint32_t tmem, const Work& w, int half, int* status) {
    const int quad = (threadIdx.x >> 5) & 3, row = quad * 32 + (threadIdx.x & 31);
    const int G = p.n_q / p.n_kv;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t s0 = tmem + T_S + half * 64 + lanes, to = tmem + T_O + lanes;
    const float scale = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)
    const int ir = row / G, hh = row % G;
    uint32_t n = 0;                                      // steps so far
    for (int k = 0; k < w.n; ++k) {
        const Item it = item_of(p, w, k);
        const bool valid = ir < it.rows && ir < p.rows_per_tile;     // the others' scores are anything: they decide nothing
        const int qp = it.pos0 + min(ir, it.rows - 1);
        float m = -INFINITY, l = 0.f;
        for (int t = it.t0; t < it.t1; ++t, ++n) {
            const uint32_t slot = n & 1, ts = s0 + slot * 128;
            const int p0 = t * BN + half * 64;           // this half's first position
            if (!wait_bar(&sm.s_full[slot], phase(n), sm, status)) return;
            tc_fence_after();
            uint32_t v[2][32];
            tmem_ld_32x32b_x32(ts, v[0]);
            tmem_ld_32x32b_x32(ts + 32, v[1]);
            tmem_ld_wait();
            if (p0 + 63 > it.pos0) {
                const int left = qp - p0;                // columns past it are later positions
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (e > left) v[e >> 5][e & 31] = __float_as_uint(-INFINITY);
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 64; e += 2)
                mx[(e >> 1) & 3] = fmaxf(fmaxf(mx[(e >> 1) & 3], __uint_as_float(v[e >> 5][e & 31])), __uint_as_float(v[e >> 5][(e & 31) + 1]));
            const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale - KV4_BELOW);
            if (t == it.t0) {
                m = mn;
            } else if (__any_sync(0xffffffffu, valid && mn > m + (KV4_HIGH - KV4_BELOW))) {
                // O, complete up to this half's last step, and l rescale; rows that
                // have seen nothing (all of the half's positions are later ones)
                // stay as they are
                const float alpha = m == mn ? 1.f : fast_ex2(m - mn);
                if (!wait_bar(&sm.pv_done[half][slot ^ 1], phase(n - 1), sm, status)) return;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {            // 16 columns at a time: S stays in registers
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(to + half * 128 + 16 * c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tmem_st_32x32b_x16(to + half * 128 + 16 * c, o);
                }
                tmem_st_wait();
                l *= alpha;
                m = mn;
            }
            const float sub = m == -INFINITY ? 0.f : m;  // nothing seen: every weight is 0
            const uint64_t sc = pair_of(scale, scale), nm = pair_of(-sub, -sub);
            uint64_t sum[2] = {pair_of(0.f, 0.f), pair_of(0.f, 0.f)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t ph[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 u = halves_of(fma2(pair_of(__uint_as_float(v[h][2 * e]), __uint_as_float(v[h][2 * e + 1])), sc, nm));
                    const float w0 = fast_ex2(u.x), w1 = fast_ex2(u.y);
                    sum[e & 1] = add2(sum[e & 1], pair_of(w0, w1));
                    const __half2 h2 = __floats2half2_rn(w0, w1);
                    ph[e] = *reinterpret_cast<const uint32_t*>(&h2);
                }
                tmem_st_32x32b_x16(ts + 16 * h, ph);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sm.p_full[half][slot]);
            const float2 a = halves_of(add2(sum[0], sum[1]));
            l += a.x + a.y;
        }
        // The halves tell each other their references and sums, once both have read the last
        // item's.  Half 0 writes an item's output while half 1 goes on; a piece, whose
        // join takes longer, they write 64 columns each.
        const bool whole = it.t1 - it.t0 == it.steps;
        if (k > 0 && !wait_bar(&sm.o_free, (k - 1) & 1, sm, status)) return;
        sm.ml[half][row] = make_float2(m, l);
        mbar_arrive(&sm.ml_done[half]);
        if (half && whole) {
            mbar_arrive(&sm.o_free);
            continue;
        }
        if (!wait_bar(&sm.ml_done[half ^ 1], k & 1, sm, status)) return;
        // a half's O is complete once the product of its last step is
        for (int h = 0; h < 2; ++h)
            if (!wait_bar(&sm.pv_done[h][(n - 1) & 1], phase(n - 1), sm, status)) return;
        tc_fence_after();
        const float2 a = sm.ml[0][row], b = sm.ml[1][row];
        const float M = fmaxf(a.x, b.x);
        const float w0 = a.x == -INFINITY ? 0.f : fast_ex2(a.x - M), w1 = b.x == -INFINITY ? 0.f : fast_ex2(b.x - M);
        const float sum = a.y * w0 + b.y * w1;
        const float r0 = whole ? w0 / sum : w0, r1 = whole ? w1 / sum : w1;
        bool bad = false;
        __half* dst = p.out + ((size_t)(it.row0 + min(ir, it.rows - 1)) * p.n_q + it.kvh * G + hh) * D;
        float4* part = p.parts + (size_t)(2 * blockIdx.x + (it.t0 ? 0 : 1)) * PART;
#pragma unroll 1
        for (int c = whole ? 0 : 2 * half; c < (whole ? 4 : 2 * half + 2); ++c) {
            uint32_t o[32], ob[32];
            tmem_ld_32x32b_x32(to + 32 * c, o);
            tmem_ld_32x32b_x32(to + 128 + 32 * c, ob);
            tmem_ld_wait();
            float v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * r0 + __uint_as_float(ob[e]) * r1;
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 8; ++e) part[(8 * c + e) * 128 + row] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            } else if (valid) {
                store32(dst + 32 * c, v, bad);
            }
        }
        tc_fence_before();
        mbar_arrive(&sm.o_free);
        if (!whole) {
            reinterpret_cast<float2*>(part + 32 * 128)[128 * half + row] = make_float2(M, sum);
            join_pieces(p, w, it, half, quad, row, valid, dst, bad);
        }
        if (bad) set_status(status, Q3_STATUS_F16_RANGE);
    }
}

__global__ void __launch_bounds__(THREADS, 1) kv4_prefill_kernel(const __grid_constant__ CUtensorMap tkv,
                                                                 const __grid_constant__ CUtensorMap tq, const Kv4PrefillArgs p)
{
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sm.k_load[i], 1);
            mbar_init(&sm.v_load[i], 1);
            mbar_init(&sm.s_full[i], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sm.p_full[h][i], 128);
                mbar_init(&sm.pv_done[h][i], 1);
            }
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_free[i], 1);
            mbar_init(&sm.drain[i], 1);
        }
        mbar_init(&sm.ml_done[0], 128);
        mbar_init(&sm.ml_done[1], 128);
        mbar_init(&sm.o_free, 256);
        sm.abort = 0;
        fence_barrier_init();
        prefetch_tmap(&tkv);
        prefetch_tmap(&tq);
    }
    if (warp == S_WARP) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;

    grid_dep_wait();
    const Work w = work_of(p, sm);
    if (warp < 8) softmax_role(p, sm, tmem, w, warp >> 2, p.status);
    else if (warp == S_WARP) scores_role(p, sm, tmem, w, p.status);
    else if (warp == PV_WARP) product_role(p, sm, tmem, w, p.status);
    else load_role(p, &tkv, &tq, sm, w, warp - K_WARP, p.status);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == S_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

size_t kv4_prefill_smem() { return SMEM_BYTES; }

cudaError_t launch_kv4_prefill(const Launch& L, const CUtensorMap& tkv, const CUtensorMap& tq, const Kv4PrefillArgs& a, int grid)
{
    static std::atomic<unsigned long long> attr_done{0};
    if (cudaError_t e = allow_smem_per_device(kv4_prefill_kernel, (int)SMEM_BYTES, attr_done)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (L.counter) ++*L.counter;
    return cudaLaunchKernelEx(&cfg, kv4_prefill_kernel, tkv, tq, a);
}

}  // namespace q3
