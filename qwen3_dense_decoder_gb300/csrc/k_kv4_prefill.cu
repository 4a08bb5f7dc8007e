// k_kv4_prefill.cu -- causal GQA attention of prefill rounds over the 4-bit
// cache on the tcgen05 tensor cores.  kv4_expand_kernel (k_kv4.cu) leaves an
// fp16 copy of the sequences' blocks and a list of query tiles, longest context
// first; a stored value is an fp16 number and q arrives in fp16, so both
// products run on single fp16 operands and only the softmax weights are rounded
// (once, to fp16).
//
// Work item: up to 2 R consecutive positions of one sequence (R = 128 / G) for
// the G query heads of one KV head, as two MMA tiles A and B of 128 rows (row r =
// position r / G, head r % G) that share every K/V tile of 128 positions:
//   S_X = Q_X K^T   tcgen05.mma, Q and K from shared memory, FP32 in tensor memory
//   P_X = 2^(S_X c - m)  one thread a row; written over S_X
//   O_X += P_X V    P from tensor memory, V read MN-major from shared memory
// The two tiles take turns: while the tensor cores work on one, the softmax
// warps of the other do its exponentials, and the scores of a tile's next
// position tile follow its product at once.  A 128 x 128 x 128 product takes
// 512 cycles of the tensor cores at their nominal rate; the softmax of a tile
// about as many of its warps' issue slots, so neither waits long for the other.
// The running maximum is raised lazily: O and the sum are rescaled only when a
// row maximum grows by more than 2^8.
//
// Roles (one CTA per SM):
//   warps 0..3, 4..7  softmax and output of A and of B (warp w: TMEM lanes 32 (w % 4) .. + 32)
//   warp 8            lane 0 issues every MMA and owns the tensor-memory columns
//   warps 9, 10       lane 0 fetches K or V tiles with TMA (blocks past the item's
//                     last position, or outside the pool, are read at a negative
//                     row and land as zeros)
//   warp 11           lane 0 fetches the item's Q with TMA
// Tensor memory: S_A, S_B, O_A, O_B of 128 columns each.  Every wait is bounded;
// a timeout sets the status word and the CTA winds down.
#include "common.cuh"
#include "kernels.h"

namespace q3 {

namespace {

constexpr int D = 128;
constexpr int BN = 128;                      // positions of a K/V tile
constexpr int ATOM = 128 * 128;              // 128 rows x 64 fp16, one swizzle atom column
constexpr int TILE = 2 * ATOM;               // 128 x 128 fp16
constexpr int NSK = 2, NSV = 3;              // K and V ring stages
constexpr int MMA_WARP = 8, K_WARP = 9, Q_WARP = 11;      // V: K_WARP + 1
constexpr int THREADS = 12 * 32;
constexpr uint32_t T_S = 0, T_O = 256;       // S_X at 128 X, O_X at 256 + 128 X
constexpr float LAZY = 8.0f;

struct alignas(1024) Smem {
    uint8_t q[2][TILE];
    uint8_t k[NSK][TILE];
    uint8_t v[NSV][TILE];
    uint64_t q_full, q_free, k_load[NSK], k_free[NSK], v_load[NSV], v_free[NSV];
    uint64_t s_full[2], p_full[2], pv_done[2], drain;
    uint32_t tmem;
    int abort;
};
constexpr size_t SMEM_BYTES = sizeof(Smem) + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

// fp16 A and B, FP32 accumulator, 128 x 128; PV reads V MN-major (bit 16)
constexpr uint32_t IDESC_S = idesc_f16_f32(128, 128), IDESC_PV = IDESC_S | (1u << 16);

Q3_DEV bool wait_bar(uint64_t* bar, uint32_t parity, Smem& sm, int* status) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*(volatile int*)&sm.abort) return false;
        if (global_ns() - t0 > Q3_WAIT_LIMIT_NS) {
            set_status(status, Q3_STATUS_TIMEOUT);
            *(volatile int*)&sm.abort = 1;
            return false;
        }
    }
}

struct Item {
    int row0, pos0, kvh, seq, slot;
    int rows[2];                             // of A and B
    int n_kt[2];                             // their K/V tiles (B's at least A's, or 0)
    Q3_DEV int most() const { return max(n_kt[0], n_kt[1]); }
};

// Item k of this CTA: tile i of the list for KV head h is number i n_kv + h,
// dealt in rows of gridDim.x, every other row backwards.
Q3_DEV Item item_of(const Kv4PrefillArgs& p, int k) {
    const int P = gridDim.x, n = k * P + ((k & 1) ? P - 1 - (int)blockIdx.x : (int)blockIdx.x);
    const int4 t = p.tiles[n / p.n_kv];
    const int R = p.rows_per_tile / 2;
    Item it;
    it.kvh = n % p.n_kv;
    it.row0 = t.x; it.pos0 = t.z; it.seq = t.w;
    it.slot = p.seq_slot ? p.seq_slot[t.w] : t.w;
    it.rows[0] = min(t.y, R);
    it.rows[1] = t.y - it.rows[0];
    it.n_kt[0] = (t.z + it.rows[0] - 1) / BN + 1;
    it.n_kt[1] = it.rows[1] ? (t.z + t.y - 1) / BN + 1 : 0;
    return it;
}

// ---------------------------------------------------------------- MMA issuer
Q3_DEV void mma_role(const Kv4PrefillArgs& p, Smem& sm, uint32_t tmem, int n_items, int* status) {
    uint32_t g[2] = {0, 0};                  // K/V tiles A and B have begun
    uint32_t gk = 0;                         // K/V tiles of the CTA before this item's
    bool ok = true;
    for (int k = 0; k < n_items && ok; ++k) {
        const Item it = item_of(p, k);
        const int most = it.most();
        // scores of tile t of X; the last user of the stage (or of Q) frees it
        auto scores = [&](int X, int t) -> bool {
            const uint32_t n = gk + t, st = n % NSK;
            if (!wait_bar(&sm.k_load[st], (n / NSK) & 1, sm, status)) return false;
            tc_fence_after();
            const uint32_t qa = smem_u32(sm.q[X]), ka = smem_u32(sm.k[st]);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint32_t off = (s >> 2) * ATOM + (s & 3) * 32;
                tc_mma_f16(tmem + T_S + X * 128, smem_desc_sw128(qa + off), smem_desc_sw128(ka + off), IDESC_S, s > 0);
            }
            tc_commit(&sm.s_full[X]);
            const bool last = X == 1 || t >= it.n_kt[1];
            if (last) tc_commit(&sm.k_free[st]);
            if (last && t + 1 == most) tc_commit(&sm.q_free);
            return true;
        };
        ok = wait_bar(&sm.q_full, k & 1, sm, status);
        for (int X = 0; X < 2 && ok; ++X)
            if (it.n_kt[X]) ok = scores(X, 0);
        for (int t = 0; t < most && ok; ++t) {
#pragma unroll 1
            for (int X = 0; X < 2 && ok; ++X) {
                if (t >= it.n_kt[X]) continue;
                const uint32_t n = gk + t, st = n % NSV;
                // (X's warps give their first weights of an item after they have read the last one's O)
                if (!(ok = wait_bar(&sm.p_full[X], g[X] & 1, sm, status))) break;
                if (!(ok = wait_bar(&sm.v_load[st], (n / NSV) & 1, sm, status))) break;
                tc_fence_after();
                const uint32_t va = smem_u32(sm.v[st]);
#pragma unroll
                for (int s = 0; s < BN / 16; ++s)
                    tc_mma_f16_ts(tmem + T_O + X * 128, tmem + T_S + X * 128 + s * 8, smem_desc_sw128_mn(va + s * 2048, ATOM),
                                  IDESC_PV, (t > 0 || s > 0) ? 1u : 0u);
                tc_commit(&sm.pv_done[X]);
                if (X == 1 || t >= it.n_kt[1]) tc_commit(&sm.v_free[st]);
                ++g[X];
                // P_X is read by now (the tensor cores keep issue order): its next scores go over it
                if (t + 1 < it.n_kt[X]) ok = scores(X, t + 1);
            }
        }
        gk += most;
    }
    // nothing of this CTA's may still run on the tensor cores at deallocation
    tc_commit(&sm.drain);
    mbar_wait(&sm.drain, 0, status);
}

// ---------------------------------------------------------------- loaders
Q3_DEV void load_role(const Kv4PrefillArgs& p, const CUtensorMap* tkv, Smem& sm, int n_items, int which, int* status) {
    const int NS = which ? NSV : NSK;
    uint64_t* ld = which ? sm.v_load : sm.k_load;
    uint64_t* fr = which ? sm.v_free : sm.k_free;
    uint32_t n = 0;
    for (int k = 0; k < n_items; ++k) {
        const Item it = item_of(p, k);
        const int* table = p.tables + (size_t)it.slot * p.max_blocks;
        const int last = it.pos0 + it.rows[0] + it.rows[1] - 1;
        for (int t = 0; t < it.most(); ++t, ++n) {
            const uint32_t st = n % NS;
            int row[BN / 32];
#pragma unroll
            for (int j = 0; j < BN / 32; ++j) {
                const int kp = t * BN + 32 * j;
                row[j] = -32;
                if (kp <= last) {
                    const int ph = table[kp >> 5];
                    if (ph >= 0 && ph < p.n_blocks)
                        row[j] = (((p.by_seq ? it.seq * p.max_blocks + (kp >> 5) : ph) * 2 + which) * p.n_kv + it.kvh) * 32;
                    // the expansion has reported any other
                }
            }
            if (n >= (uint32_t)NS && !wait_bar(&fr[st], (n / NS - 1) & 1, sm, status)) return;
            uint8_t* dst = which ? sm.v[st] : sm.k[st];
            mbar_arrive_expect_tx(&ld[st], TILE);
#pragma unroll
            for (int j = 0; j < BN / 32; ++j) {
                tma_load_2d(dst + j * 32 * 128, tkv, &ld[st], 0, row[j]);
                tma_load_2d(dst + ATOM + j * 32 * 128, tkv, &ld[st], 64, row[j]);
            }
        }
    }
}

// R positions x G heads x 64 dimensions a box: row r of the tile is position
// r / G, head r % G.  Rows past the sequence read another's (or zeros past T);
// the last 128 - R G rows of a tile are never written.  What they give is not
// stored.
Q3_DEV void q_role(const Kv4PrefillArgs& p, const CUtensorMap* tq, Smem& sm, int n_items, int* status) {
    const int G = p.n_q / p.n_kv, R = p.rows_per_tile / 2;
    for (int k = 0; k < n_items; ++k) {
        const Item it = item_of(p, k);
        if (k > 0 && !wait_bar(&sm.q_free, (k - 1) & 1, sm, status)) return;
        const int tiles = it.rows[1] ? 2 : 1;
        mbar_arrive_expect_tx(&sm.q_full, tiles * 2 * R * G * 128);
        for (int X = 0; X < tiles; ++X)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                tma_load_3d(sm.q[X] + h * ATOM, tq, &sm.q_full, 64 * h, it.kvh * G, it.row0 + X * R);
    }
}

// ---------------------------------------------------------------- softmax + output
Q3_DEV void softmax_role(const Kv4PrefillArgs& p, Smem& sm, uint32_t tmem, int n_items, int X, int* status) {
    const int quad = (threadIdx.x >> 5) & 3, row = quad * 32 + (threadIdx.x & 31);
    const int G = p.n_q / p.n_kv, R = p.rows_per_tile / 2;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t ts = tmem + T_S + X * 128 + lanes, to = tmem + T_O + X * 128 + lanes;
    const float scale = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)
    const int ir = row / G, hh = row % G;
    uint32_t g = 0;
    for (int k = 0; k < n_items; ++k) {
        const Item it = item_of(p, k);
        const int rows = it.rows[X], n_kt = it.n_kt[X];
        if (!n_kt) continue;                             // no tile of this item is X's
        const int pos0 = it.pos0 + X * R, qp = pos0 + min(ir, rows - 1);
        float m = -INFINITY, l = 0.f;
        for (int t = 0; t < n_kt; ++t, ++g) {
            if (!wait_bar(&sm.s_full[X], g & 1, sm, status)) return;
            tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + 32 * c, v[c]);
            tmem_ld_wait();
            const int left = qp - t * BN;                // columns past it are later positions
            if (t * BN + BN - 1 > pos0) {
#pragma unroll
                for (int e = 0; e < 128; ++e)
                    if (e > left) v[e >> 5][e & 31] = __float_as_uint(-INFINITY);
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 128; e += 2)
                mx[(e >> 1) & 3] = fmaxf(fmaxf(mx[(e >> 1) & 3], __uint_as_float(v[e >> 5][e & 31])), __uint_as_float(v[e >> 5][(e & 31) + 1]));
            const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale);
            if (t == 0) {
                m = mn;
            } else if (__any_sync(0xffffffffu, mn > m + LAZY)) {
                // O, complete up to the previous tile, and l rescale
                const float alpha = fast_ex2(m - mn);
                if (!wait_bar(&sm.pv_done[X], (g - 1) & 1, sm, status)) return;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {            // 16 columns at a time: S stays in registers
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(to + 16 * c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tmem_st_32x32b_x16(to + 16 * c, o);
                }
                tmem_st_wait();
                l *= alpha;
                m = mn;
            }
            const uint64_t sc = pair_of(scale, scale), nm = pair_of(-m, -m);
            uint64_t sum[2] = {pair_of(0.f, 0.f), pair_of(0.f, 0.f)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t ph[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const int c = 64 * h + 2 * e;
                    const float2 u = halves_of(fma2(pair_of(__uint_as_float(v[c >> 5][c & 31]), __uint_as_float(v[c >> 5][(c & 31) + 1])), sc, nm));
                    const float p0 = fast_ex2(u.x), p1 = fast_ex2(u.y);
                    sum[e & 1] = add2(sum[e & 1], pair_of(p0, p1));
                    const __half2 h2 = __floats2half2_rn(p0, p1);
                    ph[e] = *reinterpret_cast<const uint32_t*>(&h2);
                }
                tmem_st_32x32b_x32(ts + 32 * h, ph);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sm.p_full[X]);
            const float2 a = halves_of(add2(sum[0], sum[1]));
            l += a.x + a.y;
        }
        // the item's O is complete once the product of its last tile is
        if (!wait_bar(&sm.pv_done[X], (g - 1) & 1, sm, status)) return;
        tc_fence_after();
        const float inv = 1.0f / l;
        const bool valid = ir < rows && ir < R;
        bool bad = false;
        __half* dst = p.out + ((size_t)(it.row0 + X * R + min(ir, rows - 1)) * p.n_q + it.kvh * G + hh) * D;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + 32 * c, o);
            tmem_ld_wait();
            if (valid) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint4 w;
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        __half2 h2;
                        h2.x = to_f16(__uint_as_float(o[8 * e + 2 * f]) * inv, bad);
                        h2.y = to_f16(__uint_as_float(o[8 * e + 2 * f + 1]) * inv, bad);
                        (&w.x)[f] = *reinterpret_cast<uint32_t*>(&h2);
                    }
                    *reinterpret_cast<uint4*>(dst + c * 32 + e * 8) = w;
                }
            }
        }
        if (bad) set_status(status, Q3_STATUS_F16_RANGE);
        tc_fence_before();
    }
}

__global__ void __launch_bounds__(THREADS, 1) kv4_prefill_kernel(const __grid_constant__ CUtensorMap tkv,
                                                                 const __grid_constant__ CUtensorMap tq, const Kv4PrefillArgs p)
{
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_free, 1);
        for (int i = 0; i < NSK; ++i) { mbar_init(&sm.k_load[i], 1); mbar_init(&sm.k_free[i], 1); }
        for (int i = 0; i < NSV; ++i) { mbar_init(&sm.v_load[i], 1); mbar_init(&sm.v_free[i], 1); }
        for (int X = 0; X < 2; ++X) {
            mbar_init(&sm.s_full[X], 1);
            mbar_init(&sm.p_full[X], 128);
            mbar_init(&sm.pv_done[X], 1);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        fence_barrier_init();
        prefetch_tmap(&tkv);
        prefetch_tmap(&tq);
    }
    if (warp == MMA_WARP) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;

    grid_dep_wait();
    const int P = gridDim.x, n = *p.n_tiles * p.n_kv, full = n / P;
    const int n_items = full + (((full & 1) ? P - 1 - (int)blockIdx.x : (int)blockIdx.x) < n % P ? 1 : 0);
    const bool one = (threadIdx.x & 31) == 0;
    if (warp < 8) softmax_role(p, sm, tmem, n_items, warp >> 2, p.status);
    else if (one && warp == MMA_WARP) mma_role(p, sm, tmem, n_items, p.status);
    else if (one && warp == Q_WARP) q_role(p, &tq, sm, n_items, p.status);
    else if (one) load_role(p, &tkv, sm, n_items, warp - K_WARP, p.status);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
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
