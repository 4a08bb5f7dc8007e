// runtime.cu -- host runtime behind include/q3.h: model creation, the KV
// block pool and sessions, round planning, and the per-round launch sequence.
//
// The round ("Kipp Roadmap", status v0.0.2 and v0.0.4; "Kipp Model Support",
// section "The registry"):
//   x = embed[tokens]
//   per layer: QKV = W_qkv RMSNorm(x); q/k RMSNorm + RoPE, K/V -> paged pool;
//              o = attention; x += W_o o; x += W_down SwiGLU(W_gate h, W_up h)
//              with h = RMSNorm(x)
//   logits = U RMSNorm(x_last) for the last row of each session; argmax.
// One-token rounds stream weights through the GEMV kernel (FP32
// activations); wider rounds use the tcgen05 GEMM with fp16 operands (an fp16
// copy of the bf16 projection weights, fp16 activations).
// The host only plans: token positions, session slots and block tables are
// uploaded to device memory and every kernel reads them there.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdlib>
#include <cstdio>
#include <cstring>
#include <map>
#include <queue>
#include <set>
#include <unordered_map>
#include <string>
#include <tuple>
#include <vector>

#include "../../include/q3.h"
#include "kernels.h"

using bf16 = __nv_bfloat16;
using f16 = __half;
using namespace q3;

namespace {

thread_local std::string g_err;

int fail(int code, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return code;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    // resolved once, thread-safely (a function-local static)
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        return nullptr;
    }();
    return fn;
}

// 2-D fp16 tensor [rows][cols] (row-major) read in boxes of 64 columns (one
// 128-byte swizzle row) by box_rows rows.
bool tmap_f16(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint32_t box_rows)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t elem[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(ptr), dims, strides, box,
              elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A K/V pool (or one layer of it) as rows of 128 bf16, read in boxes of 32
// positions x 64 dimensions with the 128-byte swizzle (prefill attention).
bool tmap_kv(CUtensorMap* m, const void* ptr, uint64_t rows)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {128, rows};
    cuuint64_t strides[1] = {256};
    cuuint32_t box[2] = {64, 32};
    cuuint32_t elem[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The fp16 copy of the 4-bit cache, in the same boxes.
bool tmap_kv16(CUtensorMap* m, const void* ptr, uint64_t rows)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {128, rows};
    cuuint64_t strides[1] = {256};
    cuuint32_t box[2] = {64, 32};
    cuuint32_t elem[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows [T][n_q][128] fp16, stride elements apart, in boxes of R rows x G
// heads x 64 dimensions.
bool tmap_q16(CUtensorMap* m, const void* ptr, uint64_t T, uint64_t n_q, int64_t stride, uint32_t R, uint32_t G)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {128, n_q, T};
    cuuint64_t strides[2] = {256, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, G, R};
    cuuint32_t elem[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t round_up(size_t a, size_t b) { return (a + b - 1) / b * b; }

struct Q8Planes {
    int8_t* qs = nullptr;
    __half* sc = nullptr;
};

// AFFINE4_GS32 planes of the one-token matvec (k_gemv_a4.cu): lane-major
// code words and (scale, bias) words, 5.0 bits a weight as in the format
struct A4Planes {
    void* codes = nullptr;
    void* sb = nullptr;
};

enum Proj { P_Q, P_K, P_V, P_O, P_G, P_U, P_D, N_PROJ };

struct LayerMaps {
    CUtensorMap m[N_PROJ];
};

}  // namespace

struct q3_pool;

struct q3_model {
    q3_config c{};
    int max_rows = 0, rows_alloc = 0;
    int qw = 0, kvw = 0, qkvw = 0;
    cudaStream_t stream = nullptr;
    bool poisoned = false;
    bool pdl = false;
    int64_t launches = 0;
    int refs = 1;             // the caller's handle + one per live pool

    const bf16* embed = nullptr;
    const bf16* final_norm = nullptr;
    const bf16* lm_head = nullptr;
    std::vector<q3_layer_weights> layers;
    std::vector<std::vector<Q8Planes>> q8;   // [layer][proj]
    std::vector<std::vector<A4Planes>> a4;   // [layer][proj]

    // device memory owned by the model
    std::vector<void*> allocs;
    int* status = nullptr;
    unsigned long long* conv_counts = nullptr;   // fp16 copy: inexact, overflow
    int64_t inexact_f16 = 0;
    float2* rope = nullptr;
    float* x = nullptr;       // [rows][H] residual
    f16* ha = nullptr;        // [rows_alloc][H] normed rows (GEMM path)
    float* qkv = nullptr;     // [rows][qkvw]
    float* q = nullptr;       // [rows][qw]
    f16* att = nullptr;       // [rows_alloc][qw]
    float* attf = nullptr;    // [qw]
    f16* s = nullptr;         // [rows_alloc][F]
    float* sf = nullptr;      // [F]
    f16* hfin = nullptr;      // [rows_alloc][H]
    float* part_ml = nullptr;
    float* part_o = nullptr;
    size_t part_rows = 0;     // (row, split) pairs the partial buffers hold
    float* ws = nullptr;
    size_t ws_elems = 0;
    std::vector<std::vector<f16*>> w16;   // [layer][proj] fp16 copies for the tensor cores
                                          // (of the BF16 weights, or the dequantised Q8_0 planes)
    f16* lm16 = nullptr;      // fp16 copy of the lm_head for batched rows
#ifdef Q3_TEST_FAULTS
    int fault = 0;            // the planted addressing fault of a test build (Q3_FAULT)
    int* fault_pos = nullptr; // fault 2: the writers' row positions
#endif
    int* meta = nullptr;      // [6][max_rows]: row_pos, row_slot, last_row, tile_row0, tile_rows, row_order,
                              // then the tcgen05 attention schedule: [SCHED_GRID + 1] starts, items
    f16* q16 = nullptr;       // [rows_alloc][qw] fp16 q of prefill rounds
    int* attn_counters = nullptr;   // [max_rows][n_kv] split tickets, zero between rounds
    float* am_val = nullptr;        // lm_head argmax partials, one per GEMV CTA
    int* am_idx = nullptr;
    int* am_counter = nullptr;      // ticket of the argmax merge, zero between rounds
    int* pre_counter = nullptr;     // work queue of the prefill attention, zero between launches
    int n_sm = 0;
    bool kv_q8 = false;             // the opt-in Q8_0 K/V cache
    bool kv4 = false;               // the opt-in 4-bit K/V cache
    float* score_logits = nullptr;  // [SCORE_ROWS][vocab], made by the first scoring round
    bool prefill_tc_ok = false;     // the tcgen05 prefill attention supports these shapes
    bool prefill_tc = true;         // use it when prefill_tc_ok

    // fused one-kernel decode step (one-session decode rounds)
    bool step_ok = false;           // shapes and device support it
    bool fused_decode = true;       // use it when step_ok
    int step_grid = 0, step_slots = 0, step_splits = 0;
    size_t step_smem = 0;
    DecodeLayer* step_layers = nullptr;       // device [n_layers]
    unsigned long long* step_bar = nullptr;   // grid barrier counter
    unsigned long long step_epoch = 0;        // its value before the next launch
    float* step_am_val = nullptr;
    int* step_am_idx = nullptr;

    // pinned staging ring for host -> device metadata
    uint8_t* stage = nullptr;
    size_t stage_slot = 0;
    int stage_n = 0, stage_next = 0;
    std::vector<cudaEvent_t> stage_ev;
    std::vector<char> stage_used;

    std::vector<LayerMaps> maps;
    CUtensorMap lm_map{};
    std::map<std::tuple<const void*, int, int>, CUtensorMap> act_maps;

    // per-launch event timing (q3_model_profile)
    bool prof_on = false;
    struct ProfRec { cudaEvent_t a, b; int cls; };
    std::vector<ProfRec> prof_pending;
    std::vector<cudaEvent_t> prof_free;
    double prof_ms[Q3_K_CLASSES] = {};
    int64_t prof_n[Q3_K_CLASSES] = {};
    cudaEvent_t prof_event()
    {
        cudaEvent_t e = nullptr;
        if (!prof_free.empty()) { e = prof_free.back(); prof_free.pop_back(); }
        else cudaEventCreate(&e);
        return e;
    }
    void prof_begin(int cls)
    {
        if (!prof_on) return;
        ProfRec r{prof_event(), prof_event(), cls};
        cudaEventRecord(r.a, stream);
        prof_pending.push_back(r);
    }
    void prof_end()
    {
        if (prof_on && !prof_pending.empty()) cudaEventRecord(prof_pending.back().b, stream);
    }
    int prof_collect()
    {
        if (cudaStreamSynchronize(stream) != cudaSuccess) return Q3_ERR_CUDA;
        for (auto& r : prof_pending) {
            float ms = 0.f;
            if (cudaEventElapsedTime(&ms, r.a, r.b) == cudaSuccess) {
                prof_ms[r.cls] += ms;
                prof_n[r.cls] += 1;
            }
            prof_free.push_back(r.a);
            prof_free.push_back(r.b);
        }
        prof_pending.clear();
        return Q3_OK;
    }

    int check(cudaError_t e, const char* what)
    {
        if (e == cudaSuccess) return Q3_OK;
        poisoned = true;
        return fail(Q3_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    }

    void* dalloc(size_t bytes)
    {
        void* p = nullptr;
        if (cudaMalloc(&p, bytes ? bytes : 16) != cudaSuccess) return nullptr;
        allocs.push_back(p);
        return p;
    }

    // a pinned staging slot; blocks only if the slot's previous copy is pending
    uint8_t* stage_acquire(int* slot)
    {
        const int i = stage_next;
        stage_next = (stage_next + 1) % stage_n;
        if (stage_used[i]) cudaEventSynchronize(stage_ev[i]);
        *slot = i;
        return stage + (size_t)i * stage_slot;
    }
    cudaError_t stage_copy(int slot, void* dst, size_t bytes)
    {
        cudaError_t e = cudaMemcpyAsync(dst, stage + (size_t)slot * stage_slot, bytes,
                                        cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaEventRecord(stage_ev[slot], stream);
        stage_used[slot] = 1;
        return e;
    }

    const CUtensorMap* act_map(const void* ptr, int K, int bn)
    {
        auto key = std::make_tuple(ptr, K, bn);
        auto it = act_maps.find(key);
        if (it != act_maps.end()) return &it->second;
        CUtensorMap mp;
        if (!tmap_f16(&mp, ptr, rows_alloc, K, bn)) return nullptr;
        return &(act_maps[key] = mp);
    }
};

struct q3_session;

struct q3_pool {
    q3_model* m = nullptr;
    int n_blocks = 0, max_sessions = 0, max_blocks = 0;
    bf16* kv = nullptr;          // [L][n_blocks][2][n_kv][32][128] bf16, or [L][n_blocks][2][n_kv] Q8_0 tiles
    size_t block_bytes = 0;      // one block of one layer: K and V of every KV head
    CUtensorMap kv_map;          // kv as rows of 128 (tcgen05 prefill attention)
    int* tables = nullptr;       // [max_sessions][max_blocks]
    uint8_t* kv4_ws = nullptr;   // 4-bit cache: the prefill attention's tile list and fp16 copy of one layer's blocks
#ifdef Q3_TEST_FAULTS
    int* fault_tables = nullptr; // faults 1, 3 (readers) and 4 (writers): the perturbed tables
#endif
    std::set<int> free_blocks;   // blocks nobody holds
    std::vector<int> holders;    // per block: sessions holding it, +1 while published
    std::vector<char> slot_used;
    int refs = 1;                // the caller's handle + one per live session

    // content-addressed prefix index ("Kipp Roadmap", status v0.0.3): a
    // published block is found by (parent block, 32 tokens); the hash picks
    // a bucket and a candidate counts only if parent and tokens compare equal
    bool prefix_on = false;
    uint64_t bucket_mask = 0;
    std::unordered_map<uint64_t, std::vector<int>> buckets;
    std::vector<int> parent_of, successors;   // per published block
    std::vector<int64_t> last_use;            // publish or attach order, for eviction
    std::vector<int32_t> block_tokens;        // [n_blocks][32]
    std::vector<char> published;
    int64_t use_clock = 0;
};

namespace {
// most CTAs of the tcgen05 prefill attention (one per SM); sizes its schedule area
constexpr int SCHED_GRID = 1024;

// ints of the per-round metadata: rows, tiles and the attention schedule
// (tiles <= max_rows, so items <= max_rows * n_kv)
size_t meta_capacity(const q3_model* m)
{
    return 6 * (size_t)m->max_rows + SCHED_GRID + 1 + (size_t)m->max_rows * m->c.n_kv_heads;
}
}  // namespace

struct q3_session {
    q3_pool* pool = nullptr;
    int slot = 0;
    int pos = 0;
    std::vector<int> blocks;     // physical block of each 32 positions
    int n_fixed = 0;             // leading blocks fixed by set_block_table
    int uploaded = 0;            // table entries already on the device
};

namespace {

// ---------------------------------------------------------------- block ownership

uint64_t prefix_key(int parent, const int32_t* t)
{
    // 64-bit FNV-1a over the parent id and the 32 tokens, little-endian bytes
    uint64_t h = 0xcbf29ce484222325ull;
    auto mix = [&h](uint32_t w) {
        for (int b = 0; b < 4; ++b) { h ^= (w >> (8 * b)) & 0xffu; h *= 0x100000001b3ull; }
    };
    mix((uint32_t)parent);
    for (int i = 0; i < 32; ++i) mix((uint32_t)t[i]);
    return h;
}

int find_published(const q3_pool* p, int parent, const int32_t* t)
{
    auto it = p->buckets.find(prefix_key(parent, t) & p->bucket_mask);
    if (it == p->buckets.end()) return -1;
    for (int b : it->second)
        if (p->parent_of[b] == parent &&
            std::memcmp(&p->block_tokens[(size_t)b * 32], t, 32 * sizeof(int32_t)) == 0)
            return b;
    return -1;
}

void unpublish(q3_pool* p, int b)
{
    auto& v = p->buckets[prefix_key(p->parent_of[b], &p->block_tokens[(size_t)b * 32]) & p->bucket_mask];
    v.erase(std::find(v.begin(), v.end(), b));
    if (p->parent_of[b] >= 0) --p->successors[p->parent_of[b]];
    p->parent_of[b] = -1;
    p->published[b] = 0;
    if (--p->holders[b] == 0) p->free_blocks.insert(b);
}

// The lowest free block; with the prefix index on and none free, the
// published block held by the index alone, with no published successor,
// used longest ago is evicted.  -1: none.
int take_block(q3_pool* p)
{
    if (p->free_blocks.empty() && p->prefix_on) {
        int best = -1;
        for (int b = 0; b < p->n_blocks; ++b)
            if (p->published[b] && p->holders[b] == 1 && p->successors[b] == 0 &&
                (best < 0 || p->last_use[b] < p->last_use[best]))
                best = b;
        if (best >= 0) unpublish(p, best);
    }
    if (p->free_blocks.empty()) return -1;
    const int b = *p->free_blocks.begin();
    p->free_blocks.erase(p->free_blocks.begin());
    p->holders[b] = 1;
    return b;
}

void drop_block(q3_pool* p, int b)
{
    if (--p->holders[b] == 0) p->free_blocks.insert(b);
}

// a block another session may read: held twice or published
bool shared_block(const q3_pool* p, int b)
{
    return p->holders[b] > 1 || (p->prefix_on && p->published[b]);
}

int validate_config(const q3_config* c)
{
    if (!c) return fail(Q3_ERR_INVALID_ARG, "config is NULL");
    if (c->n_layers < 1 || c->hidden < 128 || c->n_q_heads < 1 || c->n_kv_heads < 1 ||
        c->ffn < 128 || c->vocab < 128 || c->max_ctx < 1)
        return fail(Q3_ERR_INVALID_ARG, "config: non-positive dimension");
    if (c->head_dim != 128) return fail(Q3_ERR_INVALID_ARG, "config: head_dim must be 128");
    if (c->n_q_heads % c->n_kv_heads || c->n_q_heads / c->n_kv_heads > 8)
        return fail(Q3_ERR_INVALID_ARG, "config: n_q_heads must be a multiple (<= 8x) of n_kv_heads");
    if (c->hidden % 128 || c->ffn % 128 || c->vocab % 128)
        return fail(Q3_ERR_INVALID_ARG, "config: hidden, ffn and vocab must be multiples of 128");
    if (c->scheme != Q3_BF16 && c->scheme != Q3_Q8_0 && c->scheme != Q3_AFFINE4)
        return fail(Q3_ERR_INVALID_ARG, "config: unknown weight scheme %d", c->scheme);
    if (c->kv_scheme != Q3_BF16 && c->kv_scheme != Q3_Q8_0 && c->kv_scheme != Q3_AFFINE4)
        return fail(Q3_ERR_INVALID_ARG, "config: unknown K/V cache scheme %d", c->kv_scheme);
    if (!(c->rms_eps > 0.f) || !(c->rope_theta > 0.f))
        return fail(Q3_ERR_INVALID_ARG, "config: rms_eps and rope_theta must be positive");
    return Q3_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// bytes of one 32-position block of one layer: K and V of every KV head
size_t kv_block_bytes(const q3_model* m)
{
    return (size_t)2 * m->c.n_kv_heads * (m->kv4 ? KV4_TILE : m->kv_q8 ? KVQ_TILE : 32 * 128 * 2);
}

// ---------------------------------------------------------------- 4-bit cache prefill

// The prefill attention's workspace: counts and a spare status word, the tile
// list, the pieces of cut tiles, the fp16 copy of the blocks (numbered as in the
// pool, or by sequence where that is fewer).
struct Kv4Workspace {
    size_t come, starts, parts, tiles, copy, bytes;
    int64_t blocks;
    bool by_seq;
};
Kv4Workspace kv4_workspace(int ns, int T, int n_q, int n_kv, int max_blocks, int n_blocks)
{
    Kv4Workspace w;
    w.by_seq = (int64_t)ns * max_blocks < n_blocks;
    w.blocks = w.by_seq ? (int64_t)ns * max_blocks : n_blocks;
    w.come = 256;
    w.starts = w.come + 8 * KV4_PREFILL_CTAS * sizeof(int);
    w.parts = round_up(w.starts + KV4_CUT * KV4_PREFILL_CTAS * sizeof(int), 1024);
    w.tiles = w.parts + 2 * KV4_PREFILL_CTAS * KV4_PART_BYTES;
    w.copy = round_up(w.tiles + sizeof(int4) * ((size_t)T / prefill_tc_rows(n_q, n_kv) + ns), 1024);
    w.bytes = w.copy + (size_t)w.blocks * 2 * n_kv * 32 * 128 * sizeof(f16);
    return w;
}

// expansion, then attention over the copy, on the workspace at ws
cudaError_t run_kv4_prefill(const Launch& L, Kv4PrefillArgs a, uint8_t* ws, int n_sm)
{
    const Kv4Workspace w = kv4_workspace(a.ns, a.T, a.n_q, a.n_kv, a.max_blocks, a.n_blocks);
    int* head = reinterpret_cast<int*>(ws);
    a.rows_per_tile = prefill_tc_rows(a.n_q, a.n_kv);
    a.n_tiles = head;
    a.ctas = std::min(n_sm, KV4_PREFILL_CTAS);
    a.come = reinterpret_cast<int*>(ws + w.come);
    a.starts = reinterpret_cast<int*>(ws + w.starts);
    a.parts = reinterpret_cast<float4*>(ws + w.parts);
    a.tiles = reinterpret_cast<int4*>(ws + w.tiles);
    a.max_tiles = a.T / a.rows_per_tile + a.ns;
    a.copy = reinterpret_cast<f16*>(ws + w.copy);
    a.by_seq = w.by_seq;
    const int G = a.n_q / a.n_kv;
    CUtensorMap tkv, tq;
    if (!tmap_kv16(&tkv, a.copy, (uint64_t)w.blocks * 2 * a.n_kv * 32) ||
        !tmap_q16(&tq, a.q, a.T, a.n_q, a.q_stride, a.rows_per_tile, G))
        return cudaErrorInvalidValue;
    if (cudaError_t e = launch_kv4_expand(L, a)) return e;
    if (!a.status) a.status = head + 1;              // a spare word nobody reads
    const Launch after{L.stream, true, L.counter};   // its setup overlaps the expansion
    return launch_kv4_prefill(after, tkv, tq, a, a.ctas);
}

// ---------------------------------------------------------------- the round

// Rows of logits a scoring round holds at a time: the lm_head is read once per
// chunk (0.8 GB at 151,936 x 2,560), which 512 rows of products cover.
constexpr int SCORE_ROWS = 512;

// What a scoring round returns of its last n_out rows instead of their logits.
struct Score {
    const int32_t* targets;
    int top;
    float* logprob;
    float* entropy;
    int32_t* top_ids;
    float* top_logprob;
};

struct Round {
    int T = 0, ns = 0;
    std::vector<int> n;              // tokens per session
    const int32_t* tokens = nullptr;
    float* logits = nullptr;
    int32_t* argmax = nullptr;
    q3_pool* pool = nullptr;
    int last_row = 0;                // host copy when ns == 1
    int n_out = 1;                   // rows with logits: one per session, or (ns == 1) the last n_out
    int max_ctx = 0;                 // largest context of the round
    bool decode = false;             // every session appends exactly one token
    int n_tiles = 0;                 // query tiles (prefill attention)
    bool attn_tc = false;            // the tiles and schedule are the tcgen05 kernel's
    int attn_grid = 0;               // its CTAs
    const Score* score = nullptr;    // scores of the logit rows, which then stay in the model's scratch
};

#ifndef Q3_ATTN_BATCH_BPW
#define Q3_ATTN_BATCH_BPW 8
#endif

// (row, split) pairs the decode attention's partial buffers hold
constexpr size_t ATTN_PART_ROWS = 2 * 8 * 152 + 64;

int attention_splits_impl(int n_kv, int T, int max_ctx, size_t part_rows)
{
    // Blocks per split CTA from the round's work: one block per warp while
    // the (row, KV head) units' split CTAs (the longest context bounds every
    // row) fit in about one wave of three CTAs per SM, doubling up to
    // Q3_ATTN_BATCH_BPW per warp until they do (fewer, longer CTAs, whose
    // fixed costs -- q prologue, warp merge, split ticket -- then weigh
    // less).  A round with many rows needs no splitting.
    const int nblk = (max_ctx + 31) / 32;
    const int rows = T * n_kv;
    if (rows >= 8 * 152) return 1;
    int bpw = 1;
    while (bpw < Q3_ATTN_BATCH_BPW &&
           (long long)rows * ((nblk + attention_blocks_per_cta() * bpw - 1) / (attention_blocks_per_cta() * bpw)) >
               3LL * 152)
        bpw *= 2;
    const int per_cta = attention_blocks_per_cta() * bpw;
    int s = (nblk + per_cta - 1) / per_cta;
    s = std::max(1, std::min({s, nblk, attention_max_splits()}));
    while (s > 1 && (size_t)T * s > part_rows) --s;
    return s;
}

int attention_splits(const q3_model* m, int T, int max_ctx)
{
    return attention_splits_impl(m->c.n_kv_heads, T, max_ctx, m->part_rows);
}

// Plan a tcgen05 GEMM: tile width and split-K count.  Per 64-deep k-block a
// 128 x BN tile costs the largest of 2 BN SM cycles (MMA issue), 128 + BN
// (shared-memory reads of the A and B tiles at 128 bytes per cycle), the L2
// time of those tiles and the HBM time of the weight tile (one read shared
// by the n tiles); units run in rounds of 152 (one persistent CTA per SM);
// split-K adds a reduction.  Tiles that fill the SMs take 1, 2 or 4 splits;
// fewer tiles (the weight-streaming GEMMs of batched decode rounds) any count
// up to 8, so that every SM streams a share of the weights.
void plan_gemm_impl(int M, int N, int K, size_t ws_elems, int* bn, int* splits)
{
    const int kb = K / 64;
    const int cand[9] = {32, 64, 96, 128, 144, 160, 176, 192, 256};
    int best_bn = gemm_block_n(N), best_s = 1;
    double best = 1e30;
    for (int b : cand) {
        if (b > gemm_block_n(N)) break;                  // wider than the rows need
        const int tiles = (M / 128) * ((N + b - 1) / b);
        const bool few = tiles < 152;
        for (int s = 1; s <= (few ? 8 : 4); s += (few || s == 1) ? 1 : s) {
            if (!few && s == 3) continue;
            if (s > 1 && (kb / s < 4 || (size_t)s * N * M > ws_elems)) break;
            const int rounds = (tiles * s + 151) / 152;
            // weight tile bytes from HBM per k-block, shared by the n tiles that
            // read it at about the same time, at ~22 bytes per SM cycle
            const int n_t = (N + b - 1) / b;
            const double hbm = 16384.0 / n_t / 22.0;
            // A and B tiles from L2 at ~58 bytes per SM cycle (measured on 2048-token tiles)
            const double l2 = (16384.0 + 128.0 * b) / 58.0;
            const double per_kb = std::max({(double)(2 * b), (double)(128 + b), hbm, l2});
            double cost = (double)rounds * ((double)kb / s * per_kb + 600.0);
            // partials written and read back plus the output pass, at ~3 TB/s (cycles at 2 GHz)
            if (s > 1) cost += ((double)s * N * M * 8.0 + (double)N * M * 8.0) / 1500.0;
            if (cost < best * 0.98) { best = cost; best_bn = b; best_s = s; }
        }
    }
    *bn = best_bn;
    *splits = best_s;
}

// the model's split-K workspace, in floats
constexpr size_t SPLITK_WS_ELEMS = (size_t)32 << 20;

void plan_gemm(const q3_model* m, int M, int N, int K, int* bn, int* splits)
{
    plan_gemm_impl(M, N, K, m->ws_elems, bn, splits);
}

// With norm_gain, a residual-add GEMM that splits K also writes the RMSNorm of
// its updated rows (gain norm_gain, fp16 into norm_out) in the split-K finish
// and sets *normed; otherwise the caller norms the rows itself.  With
// deferred, a plain-store GEMM that splits K leaves its partials in the
// workspace for its consumer to sum (*deferred = the split count, else 0).
// With rope, a QKV GEMM whose plan does not split K applies the q/k head
// norm, RoPE and the KV append in its epilogue (*roped = true); otherwise it
// stores the fp32 projections and the caller runs the separate kernel.
int gemm(q3_model* m, const CUtensorMap* a0, const CUtensorMap* a1, const CUtensorMap* a2,
         int tiles0, int tiles1, int pair, int M, int N, int K, const void* act, int epi, void* out,
         int ldo, const bf16* norm_gain = nullptr, f16* norm_out = nullptr, bool* normed = nullptr,
         int* deferred = nullptr, const RopeArgs* rope = nullptr, bool* roped = nullptr)
{
    int bn, splits;
    plan_gemm(m, M, N, K, &bn, &splits);
    const bool head_epi = rope && splits == 1 && !pair;
    if (roped) *roped = head_epi;
    if (head_epi) epi = EPI_QKV_ROPE;
    const CUtensorMap* b = m->act_map(act, K, bn);
    if (!b) return fail(Q3_ERR_CUDA, "tensor map encoding failed");
    GemmArgs g{};
    g.M = M; g.N = N; g.K = K;
    g.a_tiles0 = tiles0; g.a_tiles1 = tiles1;
    g.pair = pair;
    g.k_splits = splits;
    g.epi = epi;
    g.out = out; g.ldo = ldo;
    g.ws = m->ws;
    g.early_a = N <= 256;                    // batched decode rounds: the ring ramp overlaps the previous kernel
    g.status = m->status;
    if (head_epi) g.rope = *rope;
    Launch L{m->stream, m->pdl && !m->prof_on, &m->launches};
    m->prof_begin(Q3_K_GEMM);
    int rc = m->check(launch_gemm(L, *a0, a1 ? *a1 : *a0, a2 ? *a2 : *a0, *b, bn, g), "gemm");
    const bool fuse = norm_gain && gemm_add_norm_ok(g);
    const bool defer = deferred && splits > 1 && !pair && epi == EPI_STORE_F32;
    if (normed) *normed = fuse;
    if (deferred) *deferred = defer ? splits : 0;
    if (rc == Q3_OK && splits > 1 && !defer)
        rc = fuse ? m->check(launch_gemm_splitk_add_norm(L, g, norm_gain, m->c.rms_eps, norm_out), "gemm reduce+norm")
                  : m->check(launch_gemm_splitk_reduce(L, g), "gemm reduce");
    m->prof_end();
    return rc;
}

int gemv(q3_model* m, int n_tensors, const void* const* w, const __half* const* sc, const int* rows,
         int pair, int K, const float* x, const bf16* gain, int epi, float* out,
         int32_t* argmax = nullptr, const L2Prefetch* next = nullptr)
{
    GemvArgs a{};
    if (next) a.next = *next;
    int total = 0;
    for (int i = 0; i < n_tensors; ++i) {
        a.w[i] = w[i];
        a.scales[i] = sc ? sc[i] : nullptr;
        a.rows[i] = rows[i];
        total += rows[i];
    }
    a.n_tensors = n_tensors;
    a.pair = pair;
    a.K = K;
    const int scheme = !sc ? Q3_BF16 : m->c.scheme;     // the lm_head is bf16 in every scheme
    a.warps_per_row = scheme == Q3_AFFINE4 ? gemv_a4_warps_per_tile(total, K, pair)
                                           : gemv_warps_per_row(total, K, scheme, pair);
    a.argmax_out = argmax;
    a.am_val = m->am_val;
    a.am_idx = m->am_idx;
    a.am_counter = m->am_counter;
    a.x = x;
    a.norm_gain = gain;
    a.eps = m->c.rms_eps;
    a.epi = epi;
    a.out = out;
    a.status = m->status;
    Launch L{m->stream, m->pdl && !m->prof_on, &m->launches};
    m->prof_begin(Q3_K_GEMV);
    const int rc = m->check(scheme == Q3_AFFINE4 ? launch_gemv_a4(L, a) : launch_gemv(L, scheme, a), "gemv");
    m->prof_end();
    return rc;
}

#ifndef Q3_L2_PREFETCH_MB
#define Q3_L2_PREFETCH_MB 32
#endif

// The weight ranges of decode GEMV g of layer l (g: 0 QKV, 1 O, 2 gate/up,
// 3 down; layer n_layers: the lm_head), capped to a prefix for L2 prefetch.
L2Prefetch decode_weights(const q3_model* m, int l, int g)
{
    L2Prefetch pf{};
    const q3_config& c = m->c;
    const bool q8 = c.scheme == Q3_Q8_0;
    const uint64_t cap = (uint64_t)Q3_L2_PREFETCH_MB << 20;
    const uint64_t es = q8 ? 1 : 2;
    const int H = c.hidden, F = c.ffn;
    auto put = [&](int i, const void* p, uint64_t bytes) { pf.ptr[i] = p; pf.bytes[i] = bytes & ~uint64_t(15); };
    if (l >= c.n_layers) {
        put(0, m->lm_head, (uint64_t)c.vocab * H * 2);
    } else {
        const q3_layer_weights& W = m->layers[l];
        auto wp = [&](int proj, const void* bf) -> const void* { return q8 ? (const void*)m->q8[l][proj].qs : bf; };
        switch (g) {
        case 0:
            put(0, wp(P_Q, W.wq), (uint64_t)m->qw * H * es);
            put(1, wp(P_K, W.wk), (uint64_t)m->kvw * H * es);
            put(2, wp(P_V, W.wv), (uint64_t)m->kvw * H * es);
            break;
        case 1: put(0, wp(P_O, W.wo), (uint64_t)H * m->qw * es); break;
        case 2:
            put(0, wp(P_G, W.w_gate), (uint64_t)F * H * es);
            put(1, wp(P_U, W.w_up), (uint64_t)F * H * es);
            break;
        default: put(0, wp(P_D, W.w_down), (uint64_t)H * F * es); break;
        }
    }
    // cap the total to a prefix of each range, in proportion
    uint64_t total = pf.bytes[0] + pf.bytes[1] + pf.bytes[2];
    if (total > cap)
        for (int i = 0; i < 3; ++i) pf.bytes[i] = (pf.bytes[i] * cap / total) & ~uint64_t(15);
    if (cap == 0) pf = L2Prefetch{};
    return pf;
}

// The fused decode step: one CTA per SM, a cooperative launch.  Chooses the
// ring depth that fits the shared memory, the attention splits per KV head,
// and uploads the per-layer weight pointers.  Shapes the kernel does not
// handle leave it off (the per-operation path runs instead).
int setup_decode_step(q3_model* m, int n_sm)
{
    const q3_config& c = m->c;
    if (c.scheme == Q3_AFFINE4) return Q3_OK;   // no AFFINE4 consumer in the step
    if (m->kv_q8 || m->kv4) return Q3_OK;       // the step reads the BF16 cache only
#ifdef Q3_TEST_FAULTS
    if (m->fault) return Q3_OK;                 // planted faults reach the per-operation kernels only
#endif
    const bool q8 = c.scheme == Q3_Q8_0;
    int dev = 0, optin = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
        return fail(Q3_ERR_CUDA, "device query failed");
    const int grid = n_sm;
    int splits = grid / c.n_kv_heads;
    splits = std::min<int>(splits, (int)m->part_rows);
    if (splits < 1) return Q3_OK;
    int slots = 0;
    size_t smem = 0;
    for (int n = 8; n >= 3; --n) {
        const size_t b = decode_step_smem(c.hidden, c.ffn, c.n_q_heads, c.n_kv_heads, q8, n, splits, grid,
                                          c.n_layers);
        if (b && b <= (size_t)optin) { slots = n; smem = b; break; }
    }
    if (!slots) return Q3_OK;
    if (decode_step_prepare(smem) != cudaSuccess) {
        cudaGetLastError();
        return Q3_OK;
    }
    std::vector<DecodeLayer> h(c.n_layers);
    for (int l = 0; l < c.n_layers; ++l) {
        const q3_layer_weights& W = m->layers[l];
        DecodeLayer& d = h[l];
        d.attn_norm = static_cast<const bf16*>(W.attn_norm);
        d.q_norm = static_cast<const bf16*>(W.q_norm);
        d.k_norm = static_cast<const bf16*>(W.k_norm);
        d.ffn_norm = static_cast<const bf16*>(W.ffn_norm);
        const void* src[N_PROJ] = {W.wq, W.wk, W.wv, W.wo, W.w_gate, W.w_up, W.w_down};
        for (int p = 0; p < N_PROJ; ++p) {
            d.w[p] = q8 ? static_cast<const void*>(m->q8[l][p].qs) : src[p];
            d.sc[p] = q8 ? m->q8[l][p].sc : nullptr;
        }
    }
    m->step_layers = static_cast<DecodeLayer*>(m->dalloc(sizeof(DecodeLayer) * c.n_layers));
    m->step_bar = static_cast<unsigned long long*>(m->dalloc(sizeof(unsigned long long)));
    m->step_am_val = static_cast<float*>(m->dalloc(sizeof(float) * grid));
    m->step_am_idx = static_cast<int*>(m->dalloc(sizeof(int) * grid));
    if (!m->step_layers || !m->step_bar || !m->step_am_val || !m->step_am_idx)
        return fail(Q3_ERR_OOM, "device allocation failed");
    if (cudaMemcpy(m->step_layers, h.data(), sizeof(DecodeLayer) * c.n_layers, cudaMemcpyHostToDevice) !=
            cudaSuccess ||
        cudaMemset(m->step_bar, 0, sizeof(unsigned long long)) != cudaSuccess)
        return fail(Q3_ERR_CUDA, "fused decode setup failed");
    m->step_grid = grid;
    m->step_slots = slots;
    m->step_splits = splits;
    m->step_smem = smem;
    m->step_epoch = 0;
    m->step_ok = true;
    return Q3_OK;
}

// One-session decode round as one fused kernel.
int run_decode_step(q3_model* m, const Round& r)
{
    const q3_config& c = m->c;
    DecodeArgs a{};
    a.n_layers = c.n_layers; a.H = c.hidden; a.F = c.ffn; a.V = c.vocab;
    a.n_q = c.n_q_heads; a.n_kv = c.n_kv_heads; a.eps = c.rms_eps;
    a.q8 = c.scheme == Q3_Q8_0;
    a.layers = m->step_layers;
    a.embed = m->embed; a.final_norm = m->final_norm; a.lm_head = m->lm_head;
    a.rope = m->rope;
    a.token = r.tokens;
    a.row_pos = m->meta;
    a.row_slot = m->meta + m->max_rows;
    a.tables = r.pool->tables; a.max_blocks = r.pool->max_blocks;
    a.kv = r.pool->kv;
    a.layer_kv = (int64_t)r.pool->n_blocks * 2 * c.n_kv_heads * 32 * 128;
    a.n_blocks = r.pool->n_blocks;
    a.n_splits = m->step_splits;
    a.x = m->x; a.qkv = m->qkv; a.att = m->attf; a.ffn = m->sf;
    a.part_ml = m->part_ml; a.part_o = m->part_o;
    a.counters = m->attn_counters;
    a.logits = r.logits; a.argmax_out = r.argmax;
    a.am_val = m->step_am_val; a.am_idx = m->step_am_idx; a.am_counter = m->am_counter;
    a.bar = m->step_bar; a.bar_base = m->step_epoch;
    a.n_slots = m->step_slots;
    a.status = m->status;
    Launch L{m->stream, false, &m->launches};
    m->prof_begin(Q3_K_STEP);
    const int rc = m->check(launch_decode_step(L, a, m->step_grid, m->step_smem), "fused decode step");
    m->prof_end();
    if (rc == Q3_OK)
        m->step_epoch += (unsigned long long)decode_step_barriers(c.n_layers) * m->step_grid;
    return rc;
}

// The scores of n rows, from row `first` of the scored ones, whose logits are
// in the model's scratch.
int score_rows(q3_model* m, const Round& r, int first, int n)
{
    const Score& s = *r.score;
    LogprobArgs a{};
    a.logits = m->score_logits; a.stride = m->c.vocab;
    a.N = n; a.V = m->c.vocab; a.top = s.top;
    a.targets = s.targets ? s.targets + first : nullptr;
    a.logprob = s.logprob ? s.logprob + first : nullptr;
    a.entropy = s.entropy ? s.entropy + first : nullptr;
    a.top_ids = s.top_ids ? s.top_ids + (size_t)first * s.top : nullptr;
    a.top_logprob = s.top_logprob ? s.top_logprob + (size_t)first * s.top : nullptr;
    a.status = m->status;
    const Launch L{m->stream, m->pdl && !m->prof_on, &m->launches};
    m->prof_begin(Q3_K_OTHER);
    const int rc = m->check(launch_logprobs(L, a, Q3_TYPE_F32), "token log probabilities");
    m->prof_end();
    return rc;
}

int run_round(q3_model* m, const Round& r)
{
    const q3_config& c = m->c;
    const int H = c.hidden, F = c.ffn, T = r.T;
    const int* row_pos = m->meta;
    const int* row_slot = m->meta + m->max_rows;
    const int* last_rows = m->meta + 2 * m->max_rows;
    // one-row rounds take the matvec path, which reads BF16, Q8_0 planes or
    // AFFINE4 planes; wider rounds the tensor-core GEMM
    const bool one = (T == 1);
    const bool q8 = c.scheme == Q3_Q8_0;
    const bool a4 = c.scheme == Q3_AFFINE4;
    // a projection's matvec planes: quants / codes and scales (null for bf16)
    auto planes = [&](int l, int proj, const void* bf, const void** w, const __half** sc) {
        if (q8) { *w = m->q8[l][proj].qs; *sc = m->q8[l][proj].sc; }
        else if (a4) { *w = m->a4[l][proj].codes; *sc = static_cast<const __half*>(m->a4[l][proj].sb); }
        else { *w = bf; *sc = nullptr; }
    };
    Launch L{m->stream, m->pdl && !m->prof_on, &m->launches};
    // one launcher call, bracketed by profiling events of kernel class cls
    auto run = [m](int cls, auto&& launch) {
        m->prof_begin(cls);
        const cudaError_t e = launch();
        m->prof_end();
        return e;
    };
    if (one && r.ns == 1 && m->step_ok && m->fused_decode) {
        const int rc = run_decode_step(m, r);
        return rc || !r.score ? rc : score_rows(m, r, 0, 1);
    }
    const size_t layer_kv = (size_t)r.pool->n_blocks * 2 * c.n_kv_heads * 32 * 128;   // bf16 cache
    const size_t layer_bytes = (size_t)r.pool->n_blocks * r.pool->block_bytes;
    const int n_splits = attention_splits(m, T, r.max_ctx);
    int rc;

    if ((rc = m->check(run(Q3_K_NORM, [&] { return launch_embed(L, r.tokens, T, m->embed, H, c.vocab, m->x, m->status); }), "embed")))
        return rc;

    bool ha_ready = false;            // the previous residual GEMM already wrote this layer's normed rows
    int qkv_splits = 0;               // the QKV projection's partials are left for the attention to sum
    for (int l = 0; l < c.n_layers; ++l) {
        const q3_layer_weights& W = m->layers[l];
        const LayerMaps& Mp = m->maps[l];
        const bf16* attn_norm = static_cast<const bf16*>(W.attn_norm);
        const bf16* ffn_norm = static_cast<const bf16*>(W.ffn_norm);
        const bf16* next_attn_norm =
            l + 1 < c.n_layers ? static_cast<const bf16*>(m->layers[l + 1].attn_norm) : nullptr;

        // ---- QKV projection
        // prefill rounds: q/k head norm, RoPE and the KV append in the epilogue
        // (BF16 cache, no K split) or in their own kernel; decode rounds: the
        // attention sums the QKV partials and does all three itself
        RopeArgs ra{};
        if (!r.decode || m->kv4) {
            ra.qkv = m->qkv; ra.T = T; ra.n_q = c.n_q_heads; ra.n_kv = c.n_kv_heads;
            ra.q_gain = static_cast<const bf16*>(W.q_norm);
            ra.k_gain = static_cast<const bf16*>(W.k_norm);
            ra.eps = c.rms_eps; ra.rope = m->rope;
            ra.row_pos = row_pos; ra.row_slot = row_slot;
            ra.tables = r.pool->tables; ra.max_blocks = r.pool->max_blocks;
#ifdef Q3_TEST_FAULTS
            if (m->fault_pos) ra.row_pos = m->fault_pos;
            if (m->fault == 4) ra.tables = r.pool->fault_tables;
#endif
            ra.kv_layer = r.pool->kv + (size_t)l * layer_kv;
            ra.kvq_layer = m->kv_q8 ? reinterpret_cast<uint8_t*>(r.pool->kv) + (size_t)l * layer_bytes : nullptr;
            ra.n_blocks = r.pool->n_blocks;
            ra.q_out = nullptr; ra.q_out16 = m->q16; ra.status = m->status;
        }
        bool roped = false;
        if (one) {
            const void* w[3];
            const __half* sc[3];
            const int rows[3] = {m->qw, m->kvw, m->kvw};
            planes(l, P_Q, W.wq, &w[0], &sc[0]);
            planes(l, P_K, W.wk, &w[1], &sc[1]);
            planes(l, P_V, W.wv, &w[2], &sc[2]);
            const L2Prefetch nx = decode_weights(m, l, 1);
            if ((rc = gemv(m, 3, w, sc, rows, 0, H, m->x, attn_norm, EPI_STORE_F32, m->qkv, nullptr, &nx)))
                return rc;
        } else {
            if (!ha_ready &&
                (rc = m->check(run(Q3_K_NORM, [&] { return launch_rmsnorm_f16(L, m->x, nullptr, T, H, attn_norm, c.rms_eps, m->ha, m->status); }),
                               "rmsnorm")))
                return rc;
            ha_ready = false;
            const bool head_epi_ok = !r.decode && !m->kv_q8 && !m->kv4 && c.head_dim == 128;
            rc = gemm(m, &Mp.m[P_Q], &Mp.m[P_K], &Mp.m[P_V], m->qw / 128, (m->qw + m->kvw) / 128, 0,
                      m->qkvw, T, H, m->ha, EPI_STORE_F32, m->qkv, m->qkvw, nullptr, nullptr, nullptr,
                      r.decode ? &qkv_splits : nullptr, head_epi_ok ? &ra : nullptr, &roped);
            if (rc) return rc;
        }
        if (m->kv4) {
            Kv4AppendArgs ka{};
            ka.qkv = m->qkv; ka.qkv_stride = m->qkvw;
            if (!one && qkv_splits > 1) { ka.parts = m->ws; ka.n_parts = qkv_splits; }
            ka.q_gain = ra.q_gain; ka.k_gain = ra.k_gain; ka.eps = ra.eps;
            ka.rope = m->rope; ka.rope_len = c.max_ctx;
            ka.row_pos = ra.row_pos; ka.row_slot = ra.row_slot;
            ka.T = T; ka.n_q = c.n_q_heads; ka.n_kv = c.n_kv_heads;
            ka.tables = ra.tables; ka.n_slots = r.pool->max_sessions; ka.max_blocks = r.pool->max_blocks;
            ka.kv = reinterpret_cast<uint8_t*>(r.pool->kv) + (size_t)l * layer_bytes; ka.n_blocks = r.pool->n_blocks;
            ka.q_out = m->q16; ka.status = m->status;
            if ((rc = m->check(run(Q3_K_ROPE, [&] { return launch_kv4_append(L, ka, Q3_TYPE_F32); }), "4-bit append")))
                return rc;
        } else if (!r.decode && !roped &&
            (rc = m->check(run(Q3_K_ROPE, [&] { return launch_qk_norm_rope_append(L, ra); }),
                           "qk-norm/rope/append")))
            return rc;

        // ---- attention
        if (m->kv4 && r.decode) {
            Kv4DecodeArgs da{};
            da.q = m->q16; da.q_stride = m->qw;
            da.row_pos = row_pos; da.row_slot = row_slot;
            da.T = T; da.n_q = c.n_q_heads; da.n_kv = c.n_kv_heads;
            da.tables = r.pool->tables; da.n_slots = r.pool->max_sessions; da.max_blocks = r.pool->max_blocks;
            da.max_ctx = r.max_ctx;
            da.kv = reinterpret_cast<uint8_t*>(r.pool->kv) + (size_t)l * layer_bytes; da.n_blocks = r.pool->n_blocks;
            da.out = one ? (void*)m->attf : (void*)m->att;
            da.status = m->status;
            if ((rc = m->check(run(Q3_K_ATTN, [&] {
                     return launch_kv4_decode(L, da, Q3_TYPE_F16, one ? Q3_TYPE_F32 : Q3_TYPE_F16);
                 }), "4-bit attention")))
                return rc;
        } else if (m->kv4) {
            Kv4PrefillArgs pa{};
            pa.q = m->q16; pa.q_stride = m->qw;
            pa.seq_rows = m->meta + 3 * m->max_rows; pa.seq_pos = m->meta + 4 * m->max_rows;
            pa.seq_slot = m->meta + 6 * m->max_rows;
            pa.ns = r.ns; pa.T = T; pa.n_q = c.n_q_heads; pa.n_kv = c.n_kv_heads;
            pa.tables = r.pool->tables; pa.n_slots = r.pool->max_sessions; pa.max_blocks = r.pool->max_blocks;
            pa.kv = reinterpret_cast<uint8_t*>(r.pool->kv) + (size_t)l * layer_bytes; pa.n_blocks = r.pool->n_blocks;
            pa.out = m->att; pa.status = m->status;
            if ((rc = m->check(run(Q3_K_ATTN, [&] { return run_kv4_prefill(L, pa, r.pool->kv4_ws, m->n_sm); }), "4-bit prefill attention")))
                return rc;
        } else if (r.decode) {
            AttnArgs aa{};
            aa.q = m->q; aa.qkv = m->qkv;
            aa.qkv_ws = m->ws; aa.qkv_splits = one ? 0 : qkv_splits;
            aa.q_gain = static_cast<const bf16*>(W.q_norm);
            aa.k_gain = static_cast<const bf16*>(W.k_norm);
            aa.rope = m->rope; aa.eps = c.rms_eps;
            aa.T = T; aa.n_q = c.n_q_heads; aa.n_kv = c.n_kv_heads;
            aa.row_pos = row_pos; aa.row_slot = row_slot;
            aa.tables = r.pool->tables; aa.max_blocks = r.pool->max_blocks;
            aa.kv_layer = r.pool->kv + (size_t)l * layer_kv; aa.n_blocks = r.pool->n_blocks;
            aa.kvq_layer = m->kv_q8 ? reinterpret_cast<uint8_t*>(r.pool->kv) + (size_t)l * layer_bytes : nullptr;
            aa.n_splits = n_splits;
            aa.part_ml = m->part_ml; aa.part_o = m->part_o;
            aa.counters = m->attn_counters;
            aa.row_order = m->meta + 5 * m->max_rows;
            aa.out = one ? (void*)m->attf : (void*)m->att;
            aa.out_f16 = one ? 0 : 1;
            aa.status = m->status;
            if (one) aa.next = decode_weights(m, l, 1);
            if ((rc = m->check(run(Q3_K_ATTN, [&] { return launch_attention(L, aa, true); }), "attention")))
                return rc;
        } else {
            PrefillAttnArgs pa{};
            pa.q = m->q16; pa.T = T; pa.n_q = c.n_q_heads; pa.n_kv = c.n_kv_heads;
            pa.row_pos = row_pos; pa.row_slot = row_slot;
            pa.tile_row0 = m->meta + 3 * m->max_rows;
            pa.tile_rows = m->meta + 4 * m->max_rows;
            pa.n_tiles = r.n_tiles;
            pa.tables = r.pool->tables; pa.max_blocks = r.pool->max_blocks;
#ifdef Q3_TEST_FAULTS
            if (m->fault == 1 || m->fault == 3) pa.tables = r.pool->fault_tables;
#endif
            pa.kv_layer = r.pool->kv + (size_t)l * layer_kv; pa.n_blocks = r.pool->n_blocks;
            pa.kvq_layer = m->kv_q8 ? reinterpret_cast<uint8_t*>(r.pool->kv) + (size_t)l * layer_bytes : nullptr;
            pa.out = m->att;
            pa.work_counter = m->pre_counter;
            pa.sched_start = m->meta + 6 * m->max_rows;
            pa.sched_items = pa.sched_start + SCHED_GRID + 1;
            pa.kv_row0 = (int)((size_t)l * layer_kv / 128);
            pa.status = m->status;
            if ((rc = m->check(run(Q3_K_ATTN, [&] {
                     return r.attn_tc ? launch_prefill_attention_tc(L, r.pool->kv_map, pa, r.attn_grid)
                                      : launch_prefill_attention(L, pa);
                 }), "prefill attention")))
                return rc;
        }

        // ---- O projection + residual
        if (one) {
            const void* w[1];
            const __half* sc[1];
            planes(l, P_O, W.wo, &w[0], &sc[0]);
            const int rows[1] = {H};
            const L2Prefetch nx = decode_weights(m, l, 2);
            if ((rc = gemv(m, 1, w, sc, rows, 0, m->qw, m->attf, nullptr, EPI_ADD_F32, m->x, nullptr, &nx)))
                return rc;
        } else {
            rc = gemm(m, &Mp.m[P_O], nullptr, nullptr, H / 128, H / 128, 0, H, T, m->qw, m->att,
                      EPI_ADD_F32, m->x, H, ffn_norm, m->ha, &ha_ready);
            if (rc) return rc;
        }

        // ---- FFN: gate/up + SwiGLU, down + residual
        if (one) {
            const void* w[2];
            const __half* sc[2];
            planes(l, P_G, W.w_gate, &w[0], &sc[0]);
            planes(l, P_U, W.w_up, &w[1], &sc[1]);
            const int rows[2] = {F, F};
            const L2Prefetch nx2 = decode_weights(m, l, 3);
            if ((rc = gemv(m, 2, w, sc, rows, 1, H, m->x, ffn_norm, EPI_SWIGLU_F32, m->sf, nullptr, &nx2)))
                return rc;
            const void* wd[1];
            const __half* scd[1];
            planes(l, P_D, W.w_down, &wd[0], &scd[0]);
            const int rowsd[1] = {H};
            const L2Prefetch nx3 = decode_weights(m, l + 1, 0);
            if ((rc = gemv(m, 1, wd, scd, rowsd, 0, F, m->sf, nullptr, EPI_ADD_F32, m->x, nullptr, &nx3)))
                return rc;
        } else {
            if (!ha_ready &&
                (rc = m->check(run(Q3_K_NORM, [&] { return launch_rmsnorm_f16(L, m->x, nullptr, T, H, ffn_norm, c.rms_eps, m->ha, m->status); }),
                               "rmsnorm")))
                return rc;
            ha_ready = false;
            rc = gemm(m, &Mp.m[P_G], &Mp.m[P_U], nullptr, 0, 0, 1, 2 * F, T, H, m->ha,
                      EPI_SWIGLU_F16, m->s, F);
            if (rc) return rc;
            rc = gemm(m, &Mp.m[P_D], nullptr, nullptr, H / 128, H / 128, 0, H, T, F, m->s, EPI_ADD_F32,
                      m->x, H, next_attn_norm, m->ha, &ha_ready);
            if (rc) return rc;
        }
    }

    // ---- final norm + lm_head (+ argmax): the last row of each session, or
    // the last n_out rows of a one-session round
    const int n_out = r.ns == 1 ? r.n_out : r.ns;
    // logits of the n rows listed from `first` on
    auto logit_rows = [&](int first, int n, float* logits, int32_t* argmax) -> int {
        if (n == 1) {
            const void* w[1] = {m->lm_head};
            const int rows[1] = {c.vocab};
            return gemv(m, 1, w, nullptr, rows, 0, H, m->x + (size_t)(r.last_row - n_out + 1 + first) * H, m->final_norm, EPI_STORE_F32,
                        logits, argmax);
        }
        int e = m->check(run(Q3_K_NORM, [&] { return launch_rmsnorm_f16(L, m->x, last_rows + first, n, H, m->final_norm, c.rms_eps,
                                                                        m->hfin, m->status); }), "final norm");
        return e ? e : gemm(m, &m->lm_map, nullptr, nullptr, c.vocab / 128, c.vocab / 128, 0, c.vocab, n, H, m->hfin,
                            EPI_STORE_F32, logits, c.vocab);
    };
    if (r.score) {
        for (int i = 0; i < n_out; i += SCORE_ROWS) {
            const int n = std::min(SCORE_ROWS, n_out - i);
            if ((rc = logit_rows(i, n, m->score_logits, nullptr))) return rc;
            if ((rc = score_rows(m, r, i, n))) return rc;
        }
        return Q3_OK;
    }
    if ((rc = logit_rows(0, n_out, r.logits, n_out == 1 ? r.argmax : nullptr))) return rc;
    if (n_out > 1 && r.argmax &&
        (rc = m->check(run(Q3_K_OTHER, [&] { return launch_argmax(L, r.logits, n_out, c.vocab, r.argmax); }), "argmax")))
        return rc;
    return Q3_OK;
}

// Reserve blocks for positions [0, end) of a session.
int reserve(q3_session* s, int end, std::vector<std::pair<int, int>>* newly)
{
    q3_pool* p = s->pool;
    const int need = (end + 31) / 32;
    if (need > p->max_blocks) return fail(Q3_ERR_CTX_OVERFLOW, "context %d exceeds max_ctx", end);
    while ((int)s->blocks.size() < need) {
        const int b = take_block(p);
        if (b < 0) return fail(Q3_ERR_POOL_EXHAUSTED, "KV pool exhausted");
        s->blocks.push_back(b);
    }
    // a round writes positions [pos, end): their blocks must be the session's own
    for (int i = s->pos / 32; i < need; ++i)
        if (shared_block(p, s->blocks[i]))
            return fail(Q3_ERR_INVALID_ARG, "round would write shared KV block %d", s->blocks[i]);
    (void)newly;
    return Q3_OK;
}

// Upload the table entries a session gained since the last upload.
int upload_table(q3_session* s)
{
    q3_pool* p = s->pool;
    q3_model* m = p->m;
    const int n = (int)s->blocks.size();
    if (s->uploaded >= n) return Q3_OK;
    int slot;
    int32_t* h = reinterpret_cast<int32_t*>(m->stage_acquire(&slot));
    const int cnt = n - s->uploaded;
    for (int i = 0; i < cnt; ++i) h[i] = s->blocks[s->uploaded + i];
    int rc = m->check(m->stage_copy(slot, p->tables + (size_t)s->slot * p->max_blocks + s->uploaded,
                                    sizeof(int32_t) * cnt), "table upload");
#ifdef Q3_TEST_FAULTS
    // the whole perturbed table of the session; every id stays inside the pool
    if (rc == Q3_OK && p->fault_tables) {
        int fslot;
        int32_t* f = reinterpret_cast<int32_t*>(m->stage_acquire(&fslot));
        for (int i = 0; i < n; ++i) {
            const int b = s->blocks[i];
            f[i] = m->fault == 1 ? i % p->n_blocks                                  // readers ignore the table
                 : m->fault == 3 ? ((b ^ 1) < p->n_blocks ? (b ^ 1) : b)           // readers: a wrong id
                 : (i > 0 ? s->blocks[i - 1] : b);                                 // writers roll back one block
        }
        rc = m->check(m->stage_copy(fslot, p->fault_tables + (size_t)s->slot * p->max_blocks,
                                    sizeof(int32_t) * n), "fault table upload");
    }
#endif
    if (rc == Q3_OK) s->uploaded = n;
    return rc;
}

int eval_round(q3_session* const* S, int ns, const int32_t* tokens, const int* n, float* logits,
               int32_t* argmax, int n_out = 1, const Score* score = nullptr)
{
    q3_pool* pool = S[0]->pool;
    q3_model* m = pool->m;
    if (m->poisoned) return fail(Q3_ERR_POISONED, "model poisoned by an earlier error");
    Round r;
    r.ns = ns;
    r.pool = pool;
    r.tokens = tokens;
    r.logits = logits;
    r.argmax = argmax;
    r.n_out = n_out;
    r.score = score;
    if (n_out < 1 || (ns > 1 && n_out != 1) || (ns == 1 && n_out > n[0]))
        return fail(Q3_ERR_INVALID_ARG, "logit rows %d outside [1, round rows]", n_out);
    for (int i = 0; i < ns; ++i) {
        if (S[i]->pool != pool) return fail(Q3_ERR_INVALID_ARG, "sessions of different pools");
        if (n[i] < 1) return fail(Q3_ERR_INVALID_ARG, "empty round for session %d", i);
        for (int j = 0; j < i; ++j)
            if (S[j] == S[i]) return fail(Q3_ERR_INVALID_ARG, "session listed twice");
        if (S[i]->pos + n[i] > m->c.max_ctx)
            return fail(Q3_ERR_CTX_OVERFLOW, "position %d + %d exceeds max_ctx %d", S[i]->pos, n[i],
                        m->c.max_ctx);
        r.T += n[i];
        r.max_ctx = std::max(r.max_ctx, S[i]->pos + n[i]);
    }
    if (r.T > m->max_rows) return fail(Q3_ERR_INVALID_ARG, "round of %d tokens > max_round_tokens", r.T);
    int rc;
    for (int i = 0; i < ns; ++i) {
        if ((rc = reserve(S[i], S[i]->pos + n[i], nullptr))) return rc;
        if ((rc = upload_table(S[i]))) return rc;
    }
    // row metadata
    int slot;
    int32_t* h = reinterpret_cast<int32_t*>(m->stage_acquire(&slot));
    int t = 0;
    for (int i = 0; i < ns; ++i) {
        for (int j = 0; j < n[i]; ++j, ++t) {
            h[t] = S[i]->pos + j;
            h[m->max_rows + t] = S[i]->slot;
        }
        h[2 * m->max_rows + i] = t - 1;
    }
    // rows by position, latest first: the decode attention launches the rows
    // with the most blocks first, so the longest split CTAs start in the first wave
    {
        int* order = h + 5 * m->max_rows;
        for (int i = 0; i < t; ++i) order[i] = i;
        std::stable_sort(order, order + t, [&](int a, int b) { return h[a] > h[b]; });
    }
    // a one-session round with n_out logit rows: its last n_out rows, in order
    if (ns == 1 && n_out > 1)
        for (int j = 0; j < n_out; ++j) h[2 * m->max_rows + j] = n[0] - n_out + j;
    // Query tiles of the prefill attention, never spanning two sessions,
    // longest context first: 64 rows for the mma.sync kernel, 128 / G for the
    // tcgen05 kernel, which also takes a per-CTA item list built here by
    // longest-processing-time-first assignment (an item is one tile for one
    // KV head; its cost is the number of 128-position K/V tiles it walks).
    size_t meta_ints = 6 * (size_t)m->max_rows;
    if (m->kv4) {
        // the 4-bit cache lists its tiles on the device from the sessions' rows,
        // positions and slots (a round with more rows than sessions has room)
        if (r.T > ns) {
            int row = 0;
            for (int i = 0; i < ns; ++i) {
                h[3 * m->max_rows + i] = row;
                h[4 * m->max_rows + i] = S[i]->pos;
                h[6 * m->max_rows + i] = S[i]->slot;
                row += n[i];
            }
            h[3 * m->max_rows + ns] = row;
            meta_ints += ns;
        }
    }
    r.attn_tc = !m->kv4 && m->prefill_tc && m->prefill_tc_ok;
    if (!m->kv4) {
        const int R = r.attn_tc ? prefill_tc_rows(m->c.n_q_heads, m->c.n_kv_heads) : 64;
        struct Tile { int row0, rows, last_pos; };
        std::vector<Tile> tiles;
        for (int i = 0, row = 0; i < ns; row += n[i], ++i)
            for (int k = 0; k < n[i]; k += R) {
                const int rows = std::min(R, n[i] - k);
                tiles.push_back({row + k, rows, S[i]->pos + k + rows - 1});
            }
        std::stable_sort(tiles.begin(), tiles.end(),
                         [](const Tile& a, const Tile& b) { return a.last_pos > b.last_pos; });
        for (size_t t = 0; t < tiles.size(); ++t) {
            h[3 * m->max_rows + t] = tiles[t].row0;
            h[4 * m->max_rows + t] = tiles[t].rows;
        }
        r.n_tiles = (int)tiles.size();
        if (r.attn_tc) {
            const int n_kv = m->c.n_kv_heads;
            const int n_items = r.n_tiles * n_kv;
            const int grid = std::max(1, std::min({m->n_sm, n_items, SCHED_GRID}));
            // items come longest first (tiles are sorted); each goes to the
            // least-loaded CTA (ties: lowest index)
            std::vector<std::vector<int>> lists(grid);
            std::priority_queue<std::pair<long long, int>, std::vector<std::pair<long long, int>>,
                                std::greater<std::pair<long long, int>>> load;
            for (int c = 0; c < grid; ++c) load.push({0, c});
            for (int t = 0; t < r.n_tiles; ++t) {
                const long long cost = tiles[t].last_pos / 128 + 2;
                for (int kvh = 0; kvh < n_kv; ++kvh) {
                    auto top = load.top();
                    load.pop();
                    lists[top.second].push_back(t * n_kv + kvh);
                    load.push({top.first + cost, top.second});
                }
            }
            int* start = h + 6 * m->max_rows;
            int* items = start + SCHED_GRID + 1;
            int at = 0;
            for (int c = 0; c < grid; ++c) {
                start[c] = at;
                for (int v : lists[c]) items[at++] = v;
            }
            start[grid] = at;
            r.attn_grid = grid;
            meta_ints += SCHED_GRID + 1 + (size_t)at;
        }
    }
    r.last_row = r.T - 1;
    r.decode = (r.T == ns);
    if ((rc = m->check(m->stage_copy(slot, m->meta, sizeof(int32_t) * meta_ints), "meta upload")))
        return rc;
#ifdef Q3_TEST_FAULTS
    if (m->fault_pos) {                  // the writers see every row one position later
        int fslot;
        int32_t* f = reinterpret_cast<int32_t*>(m->stage_acquire(&fslot));
        for (int i = 0; i < t; ++i) f[i] = h[i] + 1;
        if ((rc = m->check(m->stage_copy(fslot, m->fault_pos, sizeof(int32_t) * t), "fault meta upload")))
            return rc;
    }
#endif
    if ((rc = run_round(m, r))) {
        m->poisoned = true;
        return rc;
    }
    for (int i = 0; i < ns; ++i) S[i]->pos += n[i];
    return Q3_OK;
}

void free_model(q3_model* m)
{
    if (!m) return;
    if (m->stream || !m->allocs.empty()) cudaStreamSynchronize(m->stream);
    for (void* p : m->allocs) cudaFree(p);
    for (auto& e : m->stage_ev) cudaEventDestroy(e);
    for (auto& r : m->prof_pending) { cudaEventDestroy(r.a); cudaEventDestroy(r.b); }
    for (auto& e : m->prof_free) cudaEventDestroy(e);
    if (m->stage) cudaFreeHost(m->stage);
    delete m;
}

// Handles are reference counted so that a model, its pools and their
// sessions may be destroyed in any order: memory is freed when the last
// dependent handle goes.
void model_release(q3_model* m)
{
    if (--m->refs == 0) free_model(m);
}

void pool_release(q3_pool* p)
{
    if (--p->refs > 0) return;
    cudaStreamSynchronize(p->m->stream);
    cudaFree(p->kv);
    cudaFree(p->tables);
    cudaFree(p->kv4_ws);
#ifdef Q3_TEST_FAULTS
    cudaFree(p->fault_tables);
#endif
    q3_model* m = p->m;
    delete p;
    model_release(m);
}

}  // namespace

// =====================================================================
// C ABI
// =====================================================================

extern "C" {

const char* q3_last_error(void) { return g_err.c_str(); }

int64_t q3_model_launch_count(const q3_model* m) { return m ? m->launches : 0; }

int q3_model_set_fused_decode(q3_model* m, int on)
{
    if (!m) return fail(Q3_ERR_INVALID_ARG, "model is NULL");
    if (on && !m->step_ok) return fail(Q3_ERR_INVALID_ARG, "fused decode step unsupported for these shapes");
    m->fused_decode = on != 0;
    return Q3_OK;
}

int q3_model_fused_decode(const q3_model* m) { return m && m->step_ok && m->fused_decode ? 1 : 0; }

int q3_model_set_prefill_tc(q3_model* m, int on)
{
    if (!m) return fail(Q3_ERR_INVALID_ARG, "model is NULL");
    if (on && !m->prefill_tc_ok) return fail(Q3_ERR_INVALID_ARG, "tcgen05 prefill attention unsupported here");
    if (!on && m->kv4) return fail(Q3_ERR_INVALID_ARG, "the 4-bit cache has no mma.sync prefill attention");
    m->prefill_tc = on != 0;
    return Q3_OK;
}

int q3_model_prefill_tc(const q3_model* m) { return m && m->prefill_tc_ok && m->prefill_tc ? 1 : 0; }

int q3_model_create(const q3_config* cfg, const q3_weights* w, int max_round_tokens, void* stream,
                    q3_model** out)
{
    if (!out) return fail(Q3_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    int rc = validate_config(cfg);
    if (rc) return rc;
    if (!w || !w->embed || !w->final_norm || !w->layers || (!cfg->tied && !w->lm_head))
        return fail(Q3_ERR_INVALID_ARG, "weights: NULL pointer");
    if (max_round_tokens < 1) return fail(Q3_ERR_INVALID_ARG, "max_round_tokens must be >= 1");
    int dev;
    cudaDeviceProp prop;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaGetDeviceProperties(&prop, dev) != cudaSuccess)
        return fail(Q3_ERR_UNSUPPORTED_DEVICE, "no CUDA device");
    if (prop.major != 10 || prop.minor != 3)
        return fail(Q3_ERR_UNSUPPORTED_DEVICE, "device is sm_%d%d; this library is built for sm_103a",
                    prop.major, prop.minor);
    if (!encode_fn()) return fail(Q3_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");

    q3_model* m = new q3_model();
    m->c = *cfg;
    const q3_config& c = m->c;
    const int H = c.hidden, F = c.ffn;
    m->qw = c.n_q_heads * 128;
    m->kvw = c.n_kv_heads * 128;
    m->qkvw = m->qw + 2 * m->kvw;
    m->max_rows = max_round_tokens;
    m->rows_alloc = (int)round_up(max_round_tokens, 256);
    m->stream = static_cast<cudaStream_t>(stream);
    m->embed = static_cast<const bf16*>(w->embed);
    m->final_norm = static_cast<const bf16*>(w->final_norm);
    m->lm_head = cfg->tied ? m->embed : static_cast<const bf16*>(w->lm_head);
    m->layers.assign(w->layers, w->layers + c.n_layers);
    m->pdl = true;
    m->n_sm = std::min(prop.multiProcessorCount, SCHED_GRID);
    m->kv_q8 = c.kv_scheme == Q3_Q8_0;
    m->kv4 = c.kv_scheme == Q3_AFFINE4;
    // the tcgen05 prefill attention reads the BF16 cache, or the fp16 copy of the
    // 4-bit cache, through a tensor map; the Q8_0 cache takes the mma.sync kernel
    m->prefill_tc_ok = !m->kv_q8 && prefill_tc_rows(c.n_q_heads, c.n_kv_heads) > 0 &&
                       std::max(prefill_tc_smem(), kv4_prefill_smem()) <= (size_t)prop.sharedMemPerBlockOptin;
    if (m->kv4 && !m->prefill_tc_ok) {
        delete m;
        return fail(Q3_ERR_INVALID_ARG, "config: the 4-bit cache needs the tcgen05 prefill attention");
    }

    auto bad = [&](int code, const char* msg) {
        free_model(m);
        return fail(code, "%s", msg);
    };
    if (!aligned16(m->embed) || !aligned16(m->lm_head) || !aligned16(m->final_norm))
        return bad(Q3_ERR_INVALID_ARG, "weights must be 16-byte aligned");
    for (auto& L : m->layers) {
        const void* ps[11] = {L.attn_norm, L.wq, L.wk, L.wv, L.q_norm, L.k_norm, L.wo, L.ffn_norm,
                              L.w_gate, L.w_up, L.w_down};
        for (const void* p : ps)
            if (!p) return bad(Q3_ERR_INVALID_ARG, "weights: NULL layer pointer");
        if (c.scheme == Q3_BF16)
            for (int i : {1, 2, 3, 6, 8, 9, 10})
                if (!aligned16(ps[i])) return bad(Q3_ERR_INVALID_ARG, "weights must be 16-byte aligned");
        if (c.scheme == Q3_AFFINE4)
            for (int i : {1, 2, 3, 6, 8, 9, 10})
                if (reinterpret_cast<uintptr_t>(ps[i]) & 3)
                    return bad(Q3_ERR_INVALID_ARG, "AFFINE4 groups must be 4-byte aligned");
    }

    const size_t R = m->rows_alloc;
    bool ok = true;
    auto A = [&](size_t bytes) {
        void* p = m->dalloc(bytes);
        if (!p) ok = false;
        return p;
    };
    m->status = static_cast<int*>(A(sizeof(int)));
    m->conv_counts = static_cast<unsigned long long*>(A(2 * sizeof(unsigned long long)));
    m->rope = static_cast<float2*>(A(sizeof(float2) * (size_t)c.max_ctx * 64));
    m->x = static_cast<float*>(A(sizeof(float) * R * H));
    m->ha = static_cast<f16*>(A(sizeof(f16) * R * H));
    m->qkv = static_cast<float*>(A(sizeof(float) * R * m->qkvw));
    m->q = static_cast<float*>(A(sizeof(float) * R * m->qw));
    m->att = static_cast<f16*>(A(sizeof(f16) * R * m->qw));
    m->attf = static_cast<float*>(A(sizeof(float) * m->qw));
    m->s = static_cast<f16*>(A(sizeof(f16) * R * F));
    m->sf = static_cast<float*>(A(sizeof(float) * F));
    m->hfin = static_cast<f16*>(A(sizeof(f16) * R * H));
    m->part_rows = ATTN_PART_ROWS;
    m->part_ml = static_cast<float*>(A(sizeof(float) * m->part_rows * c.n_q_heads * 2));
    m->part_o = static_cast<float*>(A(sizeof(float) * m->part_rows * c.n_q_heads * 128));
    m->ws_elems = SPLITK_WS_ELEMS;
    m->ws = static_cast<float*>(A(sizeof(float) * m->ws_elems));
    m->meta = static_cast<int*>(A(sizeof(int) * meta_capacity(m)));
#ifdef Q3_TEST_FAULTS
    // a test build plants one addressing fault in what the host uploads
    // (prefill rounds only: the writer is the q/k-norm/RoPE/append kernel and
    // the reader the prefill attention); one-session decode keeps the fused
    // step off so that no kernel outside those two sees the fault
    if (const char* f = getenv("Q3_FAULT")) m->fault = atoi(f);
    if (m->fault == 2) m->fault_pos = static_cast<int*>(A(sizeof(int) * (size_t)m->max_rows));
#endif
    m->q16 = static_cast<f16*>(A(sizeof(f16) * R * m->qw));
    m->attn_counters = static_cast<int*>(A(sizeof(int) * (size_t)m->max_rows * c.n_kv_heads));
    m->am_val = static_cast<float*>(A(sizeof(float) * gemv_max_grid()));
    m->am_idx = static_cast<int*>(A(sizeof(int) * gemv_max_grid()));
    m->am_counter = static_cast<int*>(A(sizeof(int)));
    m->pre_counter = static_cast<int*>(A(sizeof(int)));
    if (!ok) return bad(Q3_ERR_OOM, "device allocation failed");
    if (cudaMemset(m->status, 0, sizeof(int)) != cudaSuccess ||
        cudaMemset(m->attn_counters, 0, sizeof(int) * (size_t)m->max_rows * c.n_kv_heads) != cudaSuccess ||
        cudaMemset(m->am_counter, 0, sizeof(int)) != cudaSuccess ||
        cudaMemset(m->pre_counter, 0, sizeof(int)) != cudaSuccess ||
        cudaMemset(m->conv_counts, 0, 2 * sizeof(unsigned long long)) != cudaSuccess)
        return bad(Q3_ERR_CUDA, "cudaMemset failed");

    // RoPE table: angle p * theta^(-2i/128) and its cos/sin in double, stored as f32
    {
        std::vector<float2> tab((size_t)c.max_ctx * 64);
        for (int i = 0; i < 64; ++i) {
            const double inv = std::pow((double)c.rope_theta, -(2.0 * i) / 128.0);
            for (int p = 0; p < c.max_ctx; ++p) {
                const double a = (double)p * inv;
                tab[(size_t)p * 64 + i] = make_float2((float)std::cos(a), (float)std::sin(a));
            }
        }
        if (cudaMemcpy(m->rope, tab.data(), sizeof(float2) * tab.size(), cudaMemcpyHostToDevice) !=
            cudaSuccess)
            return bad(Q3_ERR_CUDA, "rope table upload failed");
    }

    // pinned staging ring
    m->stage_slot = round_up(std::max<size_t>(sizeof(int) * meta_capacity(m),
                                              sizeof(int) * ((size_t)c.max_ctx / 32 + 1)), 256);
    m->stage_n = 64;
    if (cudaMallocHost(&m->stage, m->stage_slot * m->stage_n) != cudaSuccess)
        return bad(Q3_ERR_OOM, "pinned staging allocation failed");
    m->stage_ev.resize(m->stage_n);
    m->stage_used.assign(m->stage_n, 0);
    for (auto& e : m->stage_ev)
        if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess)
            return bad(Q3_ERR_CUDA, "event creation failed");

    // Q8_0: derive the int8 / fp16 planes from the canonical blocks, once
    const int proj_rows[N_PROJ] = {m->qw, m->kvw, m->kvw, H, F, F, H};
    const int proj_cols[N_PROJ] = {H, H, H, m->qw, H, H, F};
    if (c.scheme == Q3_Q8_0) {
        m->q8.resize(c.n_layers);
        for (int l = 0; l < c.n_layers && ok; ++l) {
            const q3_layer_weights& L = m->layers[l];
            const void* src[N_PROJ] = {L.wq, L.wk, L.wv, L.wo, L.w_gate, L.w_up, L.w_down};
            m->q8[l].resize(N_PROJ);
            for (int p = 0; p < N_PROJ; ++p) {
                const size_t n = (size_t)proj_rows[p] * proj_cols[p];
                m->q8[l][p].qs = static_cast<int8_t*>(A(n));
                m->q8[l][p].sc = static_cast<__half*>(A(n / 32 * sizeof(__half)));
                if (!ok) break;
                if (launch_q8_split(m->stream, static_cast<const uint8_t*>(src[p]), (int64_t)(n / 32),
                                    m->q8[l][p].qs, m->q8[l][p].sc) != cudaSuccess)
                    return bad(Q3_ERR_CUDA, "Q8_0 plane derivation failed");
            }
        }
        // fp16 copies of the dequantised projections for the tensor-core path
        // (prefill and batched rounds), made once: d * q rounded to fp16
        m->maps.resize(c.n_layers);
        m->w16.resize(c.n_layers);
        const Launch L0{m->stream, false, nullptr};
        for (int l = 0; l < c.n_layers && ok; ++l) {
            m->w16[l].resize(N_PROJ);
            for (int p = 0; p < N_PROJ; ++p) {
                const size_t n = (size_t)proj_rows[p] * proj_cols[p];
                f16* d = static_cast<f16*>(A(n * sizeof(f16)));
                if (!ok) break;
                m->w16[l][p] = d;
                if (launch_q8_to_f16(L0, m->q8[l][p].qs, m->q8[l][p].sc, (int64_t)n, d) != cudaSuccess)
                    return bad(Q3_ERR_CUDA, "Q8_0 dequantisation failed");
                const uint32_t box = (p == P_G || p == P_U) ? 64 : 128;
                if (!tmap_f16(&m->maps[l].m[p], d, proj_rows[p], proj_cols[p], box))
                    return bad(Q3_ERR_CUDA, "tensor map encoding failed");
            }
        }
    } else if (c.scheme == Q3_AFFINE4) {
        // one-token rounds: the format's bytes rearranged lane-major for the
        // 5.0-bit matvec; wider rounds: fp16 copies of the dequantised groups
        // for the tensor-core path, fp16(fma(scale, code, bias))
        m->maps.resize(c.n_layers);
        m->w16.resize(c.n_layers);
        m->a4.resize(c.n_layers);
        for (int l = 0; l < c.n_layers && ok; ++l) {
            const q3_layer_weights& L = m->layers[l];
            const void* src[N_PROJ] = {L.wq, L.wk, L.wv, L.wo, L.w_gate, L.w_up, L.w_down};
            m->w16[l].resize(N_PROJ);
            m->a4[l].resize(N_PROJ);
            for (int p = 0; p < N_PROJ; ++p) {
                const size_t n = (size_t)proj_rows[p] * proj_cols[p];
                m->a4[l][p].codes = A(n / 2);
                m->a4[l][p].sb = A(n / 32 * 4);
                if (!ok) break;
                if (launch_a4_planes(m->stream, static_cast<const uint8_t*>(src[p]), proj_rows[p], proj_cols[p],
                                     m->a4[l][p].codes, m->a4[l][p].sb) != cudaSuccess)
                    return bad(Q3_ERR_CUDA, "AFFINE4 plane derivation failed");
                f16* d = static_cast<f16*>(A(n * sizeof(f16)));
                if (!ok) break;
                m->w16[l][p] = d;
                if (launch_affine4_to_f16(m->stream, static_cast<const uint8_t*>(src[p]), (int64_t)n, d,
                                          m->conv_counts + 1) != cudaSuccess)
                    return bad(Q3_ERR_CUDA, "AFFINE4 dequantisation failed");
                const uint32_t box = (p == P_G || p == P_U) ? 64 : 128;
                if (!tmap_f16(&m->maps[l].m[p], d, proj_rows[p], proj_cols[p], box))
                    return bad(Q3_ERR_CUDA, "tensor map encoding failed");
            }
        }
    } else {
        // fp16 copies of the projections for the tensor-core path
        m->maps.resize(c.n_layers);
        m->w16.resize(c.n_layers);
        for (int l = 0; l < c.n_layers && ok; ++l) {
            const q3_layer_weights& L = m->layers[l];
            const void* src[N_PROJ] = {L.wq, L.wk, L.wv, L.wo, L.w_gate, L.w_up, L.w_down};
            m->w16[l].resize(N_PROJ);
            for (int p = 0; p < N_PROJ; ++p) {
                const size_t n = (size_t)proj_rows[p] * proj_cols[p];
                f16* d = static_cast<f16*>(A(n * sizeof(f16)));
                if (!ok) break;
                m->w16[l][p] = d;
                if (launch_bf16_to_f16(m->stream, static_cast<const bf16*>(src[p]), (int64_t)n, d,
                                       m->conv_counts, m->conv_counts + 1) != cudaSuccess)
                    return bad(Q3_ERR_CUDA, "fp16 weight copy failed");
                const uint32_t box = (p == P_G || p == P_U) ? 64 : 128;
                if (!tmap_f16(&m->maps[l].m[p], d, proj_rows[p], proj_cols[p], box))
                    return bad(Q3_ERR_CUDA, "tensor map encoding failed");
            }
        }
    }
    m->lm16 = static_cast<f16*>(A(sizeof(f16) * (size_t)c.vocab * H));
    if (!ok) return bad(Q3_ERR_OOM, "device allocation failed");
    if (launch_bf16_to_f16(m->stream, m->lm_head, (int64_t)c.vocab * H, m->lm16, m->conv_counts,
                           m->conv_counts + 1) != cudaSuccess)
        return bad(Q3_ERR_CUDA, "fp16 lm_head copy failed");
    if (!tmap_f16(&m->lm_map, m->lm16, c.vocab, H, 128))
        return bad(Q3_ERR_CUDA, "tensor map encoding failed");
    {
        unsigned long long cnt[2] = {0, 0};
        if (cudaMemcpyAsync(cnt, m->conv_counts, sizeof cnt, cudaMemcpyDeviceToHost, m->stream) !=
                cudaSuccess || cudaStreamSynchronize(m->stream) != cudaSuccess)
            return bad(Q3_ERR_CUDA, "fp16 weight copy failed");
        if (cnt[1])
            return bad(Q3_ERR_INVALID_ARG, "weights beyond the fp16 range of the tensor-core path");
        m->inexact_f16 = (int64_t)cnt[0];
    }
    if (!ok) return bad(Q3_ERR_OOM, "device allocation failed");
    if ((rc = setup_decode_step(m, prop.multiProcessorCount))) {
        free_model(m);
        return rc;
    }
    if (cudaStreamSynchronize(m->stream) != cudaSuccess || cudaGetLastError() != cudaSuccess)
        return bad(Q3_ERR_CUDA, "model setup failed");
    *out = m;
    return Q3_OK;
}

void q3_model_destroy(q3_model* m)
{
    if (!m) return;
    model_release(m);
}

int q3_pool_create(q3_model* m, int n_blocks, int max_sessions, q3_pool** out)
{
    if (!m || !out || n_blocks < 1 || max_sessions < 1)
        return fail(Q3_ERR_INVALID_ARG, "pool: bad argument");
    *out = nullptr;
    q3_pool* p = new q3_pool();
    p->m = m;
    p->n_blocks = n_blocks;
    p->max_sessions = max_sessions;
    p->max_blocks = (m->c.max_ctx + 31) / 32;
    p->block_bytes = kv_block_bytes(m);
    const size_t kv_bytes = (size_t)m->c.n_layers * n_blocks * p->block_bytes;
    if (cudaMalloc(&p->kv, kv_bytes) != cudaSuccess) {
        delete p;
        return fail(Q3_ERR_OOM, "pool: cannot allocate %zu bytes of KV", kv_bytes);
    }
    if (!m->kv_q8 && !m->kv4 && !tmap_kv(&p->kv_map, p->kv, kv_bytes / 256)) {
        cudaFree(p->kv);
        delete p;
        return fail(Q3_ERR_CUDA, "pool: tensor map encoding failed");
    }
    // zeroed once so positions a block has not been written hold finite values
    // (zero codes and zero scales for the Q8_0 cache)
    if (cudaMemsetAsync(p->kv, 0, kv_bytes, m->stream) != cudaSuccess) {
        cudaFree(p->kv);
        delete p;
        return fail(Q3_ERR_CUDA, "pool: memset failed");
    }
    if (cudaMalloc(&p->tables, sizeof(int) * (size_t)max_sessions * p->max_blocks) != cudaSuccess) {
        cudaFree(p->kv);
        delete p;
        return fail(Q3_ERR_OOM, "pool: cannot allocate block tables");
    }
    if (cudaMemsetAsync(p->tables, 0xff, sizeof(int) * (size_t)max_sessions * p->max_blocks,
                        m->stream) != cudaSuccess) {
        cudaFree(p->kv);
        cudaFree(p->tables);
        delete p;
        return fail(Q3_ERR_CUDA, "pool: memset failed");
    }
    if (m->kv4) {
        const size_t wb = kv4_workspace(std::min(max_sessions, m->max_rows), m->max_rows, m->c.n_q_heads, m->c.n_kv_heads,
                                        p->max_blocks, n_blocks).bytes;
        if (cudaMalloc(&p->kv4_ws, wb) != cudaSuccess) {
            cudaFree(p->kv);
            cudaFree(p->tables);
            delete p;
            return fail(Q3_ERR_OOM, "pool: cannot allocate %zu bytes of prefill workspace", wb);
        }
    }
#ifdef Q3_TEST_FAULTS
    if (m->fault == 1 || m->fault == 3 || m->fault == 4) {
        const size_t tb = sizeof(int) * (size_t)max_sessions * p->max_blocks;
        if (cudaMalloc(&p->fault_tables, tb) != cudaSuccess ||
            cudaMemsetAsync(p->fault_tables, 0xff, tb, m->stream) != cudaSuccess) {
            cudaFree(p->fault_tables);
            cudaFree(p->kv);
            cudaFree(p->tables);
            cudaFree(p->kv4_ws);
            delete p;
            return fail(Q3_ERR_OOM, "pool: fault tables");
        }
    }
#endif
    for (int b = 0; b < n_blocks; ++b) p->free_blocks.insert(p->free_blocks.end(), b);
    p->holders.assign(n_blocks, 0);
    p->slot_used.assign(max_sessions, 0);
    ++m->refs;
    *out = p;
    return Q3_OK;
}

void q3_pool_destroy(q3_pool* p)
{
    if (!p) return;
    pool_release(p);
}

int q3_session_create(q3_pool* p, q3_session** out)
{
    if (!p || !out) return fail(Q3_ERR_INVALID_ARG, "session: bad argument");
    *out = nullptr;
    int slot = -1;
    for (int i = 0; i < p->max_sessions; ++i)
        if (!p->slot_used[i]) { slot = i; break; }
    if (slot < 0) return fail(Q3_ERR_INVALID_ARG, "pool has no free session slot");
    q3_session* s = new q3_session();
    s->pool = p;
    s->slot = slot;
    p->slot_used[slot] = 1;
    ++p->refs;
    *out = s;
    return Q3_OK;
}

void q3_session_destroy(q3_session* s)
{
    if (!s) return;
    q3_pool* p = s->pool;
    for (int b : s->blocks) drop_block(p, b);
    p->slot_used[s->slot] = 0;
    delete s;
    pool_release(p);
}

int q3_session_set_block_table(q3_session* s, const int32_t* ids, int n)
{
    if (!s || (n > 0 && !ids) || n < 0) return fail(Q3_ERR_INVALID_ARG, "set_block_table: bad argument");
    if (s->pos != 0) return fail(Q3_ERR_INVALID_ARG, "set_block_table: session is not empty");
    q3_pool* p = s->pool;
    if (n > p->max_blocks) return fail(Q3_ERR_INVALID_ARG, "set_block_table: more blocks than max_ctx");
    for (int b : s->blocks) drop_block(p, b);
    s->blocks.clear();
    std::set<int> seen;
    for (int i = 0; i < n; ++i) {
        if (ids[i] < 0 || ids[i] >= p->n_blocks || !p->free_blocks.count(ids[i]) || seen.count(ids[i])) {
            s->n_fixed = 0;
            s->uploaded = 0;
            return fail(Q3_ERR_INVALID_ARG, "set_block_table: block %d not free or out of range", ids[i]);
        }
        seen.insert(ids[i]);
    }
    for (int i = 0; i < n; ++i) {
        p->free_blocks.erase(ids[i]);
        p->holders[ids[i]] = 1;
        s->blocks.push_back(ids[i]);
    }
    s->n_fixed = n;
    s->uploaded = 0;
    return Q3_OK;
}

int q3_session_eval(q3_session* s, const int32_t* tokens_dev, int n, float* logits_dev,
                    int32_t* argmax_dev)
{
    if (!s || !tokens_dev || !logits_dev || n < 1) return fail(Q3_ERR_INVALID_ARG, "eval: bad argument");
    q3_model* m = s->pool->m;
    if (s->pos + n > m->c.max_ctx)
        return fail(Q3_ERR_CTX_OVERFLOW, "position %d + %d exceeds max_ctx %d", s->pos, n, m->c.max_ctx);
    for (int off = 0; off < n; off += m->max_rows) {
        const int k = std::min(m->max_rows, n - off);
        int rc = eval_round(&s, 1, tokens_dev + off, &k, logits_dev, argmax_dev);
        if (rc) return rc;
    }
    return Q3_OK;
}

int q3_session_eval_n(q3_session* s, const int32_t* tokens_dev, int n, int n_logits, float* logits_dev,
                      int32_t* argmax_dev)
{
    if (!s || !tokens_dev || !logits_dev || n < 1 || n_logits < 1 || n_logits > n)
        return fail(Q3_ERR_INVALID_ARG, "eval_n: bad argument");
    q3_model* m = s->pool->m;
    if (s->pos + n > m->c.max_ctx)
        return fail(Q3_ERR_CTX_OVERFLOW, "position %d + %d exceeds max_ctx %d", s->pos, n, m->c.max_ctx);
    // rounds of at most max_round_tokens rows; the last n_logits rows of the
    // call are a suffix of its last rounds
    const int first = n - n_logits;
    for (int off = 0; off < n; off += m->max_rows) {
        const int k = std::min(m->max_rows, n - off);
        const int lo = std::max(off, first);
        const int rows = off + k - lo;                          // this round's logit rows (a suffix)
        int rc;
        if (rows >= 1)
            rc = eval_round(&s, 1, tokens_dev + off, &k, logits_dev + (size_t)(lo - first) * m->c.vocab,
                            argmax_dev ? argmax_dev + (lo - first) : nullptr, rows);
        else
            rc = eval_round(&s, 1, tokens_dev + off, &k, logits_dev, nullptr, 1);   // overwritten later
        if (rc) return rc;
    }
    return Q3_OK;
}

int q3_session_score(q3_session* s, const int32_t* tokens_dev, int n, int n_score, const int32_t* targets_dev, int top_k,
                     float* logprob_dev, float* entropy_dev, int32_t* top_ids_dev, float* top_logprob_dev)
{
    if (!s || !tokens_dev || n < 1 || n_score < 1 || n_score > n || (logprob_dev && !targets_dev))
        return fail(Q3_ERR_INVALID_ARG, "score: bad argument");
    q3_model* m = s->pool->m;
    if (top_k < 0 || top_k > m->c.vocab || top_k > Q3_LOGPROB_MAX_TOP)
        return fail(Q3_ERR_INVALID_ARG, "score: top_k outside [0, %d]", Q3_LOGPROB_MAX_TOP);
    if (n > m->c.max_ctx - s->pos)
        return fail(Q3_ERR_CTX_OVERFLOW, "position %d + %d exceeds max_ctx %d", s->pos, n, m->c.max_ctx);
    if (m->poisoned) return fail(Q3_ERR_POISONED, "model poisoned by an earlier error");
    if (!m->score_logits) {
        const size_t rows = std::min(SCORE_ROWS, m->max_rows);
        m->score_logits = static_cast<float*>(m->dalloc(sizeof(float) * rows * m->c.vocab));
        if (!m->score_logits) {
            cudaGetLastError();
            return fail(Q3_ERR_OOM, "score: cannot allocate the logits of %zu rows", rows);
        }
    }
    const int first = n - n_score;
    for (int off = 0; off < n; off += m->max_rows) {
        const int k = std::min(m->max_rows, n - off);
        const int lo = std::max(off, first);
        const int rows = off + k - lo;                          // this round's scored rows (a suffix)
        int rc;
        if (rows >= 1) {
            const size_t at = lo - first;
            const Score sc{targets_dev ? targets_dev + at : nullptr, top_ids_dev || top_logprob_dev ? top_k : 0,
                           logprob_dev ? logprob_dev + at : nullptr, entropy_dev ? entropy_dev + at : nullptr,
                           top_ids_dev ? top_ids_dev + at * top_k : nullptr,
                           top_logprob_dev ? top_logprob_dev + at * top_k : nullptr};
            rc = eval_round(&s, 1, tokens_dev + off, &k, m->score_logits, nullptr, rows, &sc);
        } else {
            rc = eval_round(&s, 1, tokens_dev + off, &k, m->score_logits, nullptr, 1);   // overwritten later
        }
        if (rc) return rc;
    }
    return Q3_OK;
}

int q3_eval_batch(q3_session* const* sessions, int ns, const int32_t* tokens_dev, const int* n,
                  float* logits_dev, int32_t* argmax_dev)
{
    if (!sessions || ns < 1 || !tokens_dev || !n || !logits_dev)
        return fail(Q3_ERR_INVALID_ARG, "eval_batch: bad argument");
    for (int i = 0; i < ns; ++i)
        if (!sessions[i]) return fail(Q3_ERR_INVALID_ARG, "eval_batch: NULL session");
    return eval_round(sessions, ns, tokens_dev, n, logits_dev, argmax_dev);
}

int q3_session_truncate(q3_session* s, int n_pos)
{
    if (!s || n_pos < 0 || n_pos > s->pos) return fail(Q3_ERR_INVALID_ARG, "truncate: bad position");
    q3_pool* p = s->pool;
    const int keep = std::max((n_pos + 31) / 32, s->n_fixed);
    while ((int)s->blocks.size() > keep) {
        drop_block(p, s->blocks.back());
        s->blocks.pop_back();
    }
    // the block position n_pos falls in is written next: a shared one is
    // copied to a block of the session's own first (all layers, K and V)
    const int last = n_pos / 32;
    if (n_pos % 32 && last < (int)s->blocks.size() && shared_block(p, s->blocks[last])) {
        q3_model* m = p->m;
        const int b = s->blocks[last], nb = take_block(p);
        if (nb < 0) return fail(Q3_ERR_POOL_EXHAUSTED, "truncate: no block for the copy of a shared block");
        const size_t blk = p->block_bytes;
        uint8_t* base = reinterpret_cast<uint8_t*>(p->kv);
        for (int l = 0; l < m->c.n_layers; ++l) {
            const int rc = m->check(cudaMemcpyAsync(base + ((size_t)l * p->n_blocks + nb) * blk,
                                                    base + ((size_t)l * p->n_blocks + b) * blk,
                                                    blk, cudaMemcpyDeviceToDevice, m->stream),
                                    "shared block copy");
            if (rc) return rc;
        }
        drop_block(p, b);
        s->blocks[last] = nb;
        s->uploaded = std::min(s->uploaded, last);
    }
    s->pos = n_pos;
    s->uploaded = std::min(s->uploaded, (int)s->blocks.size());
    return Q3_OK;
}

int q3_session_reset(q3_session* s) { return q3_session_truncate(s, 0); }

int q3_pool_enable_prefix(q3_pool* p, int hash_bits)
{
    if (!p || hash_bits < 0 || hash_bits > 24) return fail(Q3_ERR_INVALID_ARG, "enable_prefix: bad argument");
    if (p->prefix_on) return fail(Q3_ERR_INVALID_ARG, "enable_prefix: already enabled");
    const size_t n = (size_t)p->n_blocks;
    p->bucket_mask = ((uint64_t)1 << hash_bits) - 1;
    p->parent_of.assign(n, -1);
    p->successors.assign(n, 0);
    p->last_use.assign(n, 0);
    p->block_tokens.assign(n * 32, 0);
    p->published.assign(n, 0);
    p->prefix_on = true;
    return Q3_OK;
}

int q3_session_publish(q3_session* s, const int32_t* tokens, int n, int* n_published)
{
    if (!s || (n > 0 && !tokens) || n != (s ? s->pos : 0))
        return fail(Q3_ERR_INVALID_ARG, "publish: tokens must cover the session's positions");
    q3_pool* p = s->pool;
    if (!p->prefix_on || s->n_fixed) return fail(Q3_ERR_INVALID_ARG, "publish: no prefix index, or a fixed table");
    int parent = -1, count = 0;
    for (int i = 0; i < s->pos / 32; ++i) {
        int b = s->blocks[i];
        const int32_t* t = tokens + (size_t)i * 32;
        if (!p->published[b]) {
            const int e = find_published(p, parent, t);
            if (e >= 0) {                      // an equal block: share it, free ours
                ++p->holders[e];
                drop_block(p, b);
                s->blocks[i] = e;
                s->uploaded = std::min(s->uploaded, i);
                b = e;
            } else {
                std::memcpy(&p->block_tokens[(size_t)b * 32], t, 32 * sizeof(int32_t));
                p->parent_of[b] = parent;
                p->buckets[prefix_key(parent, t) & p->bucket_mask].push_back(b);
                p->published[b] = 1;
                p->last_use[b] = ++p->use_clock;
                ++p->holders[b];
                if (parent >= 0) ++p->successors[parent];
                ++count;
            }
        }
        parent = b;
    }
    if (n_published) *n_published = count;
    return Q3_OK;
}

int q3_session_attach_prefix(q3_session* s, const int32_t* tokens, int n, int* n_attached)
{
    if (!s || !tokens || n < 1) return fail(Q3_ERR_INVALID_ARG, "attach_prefix: bad argument");
    q3_pool* p = s->pool;
    if (!p->prefix_on || s->pos != 0 || s->n_fixed)
        return fail(Q3_ERR_INVALID_ARG, "attach_prefix: no prefix index, a non-empty session or a fixed table");
    if (n > p->m->c.max_ctx) return fail(Q3_ERR_CTX_OVERFLOW, "attach_prefix: prompt exceeds max_ctx");
    for (int b : s->blocks) drop_block(p, b);
    s->blocks.clear();
    int parent = -1;
    for (int i = 0; i < (n - 1) / 32; ++i) {          // at least one token stays to evaluate
        const int e = find_published(p, parent, tokens + (size_t)i * 32);
        if (e < 0) break;
        ++p->holders[e];
        p->last_use[e] = ++p->use_clock;
        s->blocks.push_back(e);
        parent = e;
    }
    s->pos = 32 * (int)s->blocks.size();
    s->uploaded = 0;
    if (n_attached) *n_attached = s->pos;
    return Q3_OK;
}

int q3_session_pos(const q3_session* s) { return s ? s->pos : -1; }

int q3_sync(q3_model* m)
{
    if (!m) return fail(Q3_ERR_INVALID_ARG, "sync: NULL model");
    if (m->poisoned) return fail(Q3_ERR_POISONED, "model poisoned by an earlier error");
    int rc = m->check(cudaStreamSynchronize(m->stream), "stream");
    if (rc) return rc;
    int st = 0;
    if ((rc = m->check(cudaMemcpy(&st, m->status, sizeof(int), cudaMemcpyDeviceToHost), "status read")))
        return rc;
    if (st) {
        cudaMemset(m->status, 0, sizeof(int));
        m->poisoned = true;
        return fail(Q3_ERR_DEVICE_CHECK, "device check failed (status 0x%x)", st);
    }
    return Q3_OK;
}

int q3_quantize_q8_0(const void* w_dev, int64_t n, void* blocks_dev, void* stream)
{
    if (!w_dev || !blocks_dev || n < 0 || n % 32) return fail(Q3_ERR_INVALID_ARG, "quantize: bad argument");
    if (n == 0) return Q3_OK;
    cudaError_t e = launch_quantize_q8_0(static_cast<cudaStream_t>(stream), static_cast<const bf16*>(w_dev),
                                         n, static_cast<uint8_t*>(blocks_dev));
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "quantize: %s", cudaGetErrorString(e));
    return Q3_OK;
}

int q3_quantize_affine4(const void* w_dev, int64_t n, void* groups_dev, void* stream)
{
    if (!w_dev || !groups_dev || n < 0 || n % 32 || !aligned16(w_dev) ||
        (reinterpret_cast<uintptr_t>(groups_dev) & 3))
        return fail(Q3_ERR_INVALID_ARG, "quantize: bad argument");
    if (n == 0) return Q3_OK;
    cudaError_t e = launch_quantize_affine4(static_cast<cudaStream_t>(stream), static_cast<const bf16*>(w_dev),
                                            n, static_cast<uint8_t*>(groups_dev));
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "quantize: %s", cudaGetErrorString(e));
    return Q3_OK;
}

int q3_affine4_to_f16(const void* groups_dev, int64_t n, void* out_dev, void* stream)
{
    if (!groups_dev || !out_dev || n < 0 || n % 32 || !aligned16(out_dev) ||
        (reinterpret_cast<uintptr_t>(groups_dev) & 3))
        return fail(Q3_ERR_INVALID_ARG, "dequantize: bad argument");
    if (n == 0) return Q3_OK;
    cudaError_t e = launch_affine4_to_f16(static_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(groups_dev),
                                          n, static_cast<f16*>(out_dev), nullptr);
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "dequantize: %s", cudaGetErrorString(e));
    return Q3_OK;
}

int q3_model_profile(q3_model* m, int on)
{
    if (!m) return fail(Q3_ERR_INVALID_ARG, "profile: NULL model");
    if (m->prof_on && !on && m->prof_collect() != Q3_OK) return fail(Q3_ERR_CUDA, "profile: sync failed");
    m->prof_on = on != 0;
    return Q3_OK;
}

int q3_model_profile_reset(q3_model* m)
{
    if (!m) return fail(Q3_ERR_INVALID_ARG, "profile: NULL model");
    if (m->prof_collect() != Q3_OK) return fail(Q3_ERR_CUDA, "profile: sync failed");
    for (int i = 0; i < Q3_K_CLASSES; ++i) { m->prof_ms[i] = 0; m->prof_n[i] = 0; }
    return Q3_OK;
}

int q3_model_profile_read(q3_model* m, int cls, double* total_ms, int64_t* launches)
{
    if (!m || cls < 0 || cls >= Q3_K_CLASSES || !total_ms || !launches)
        return fail(Q3_ERR_INVALID_ARG, "profile_read: bad argument");
    if (m->prof_collect() != Q3_OK) return fail(Q3_ERR_CUDA, "profile: sync failed");
    *total_ms = m->prof_ms[cls];
    *launches = m->prof_n[cls];
    return Q3_OK;
}

int q3_model_kv_bytes_per_position(const q3_model* m)
{
    return m ? (int)(kv_block_bytes(m) / 32) : -1;
}

int q3_op_kv_pack_q8_0(const float* rows_dev, int n_rows, void* out_dev, void* stream)
{
    if (!rows_dev || !out_dev || n_rows < 1 || !aligned16(rows_dev))
        return fail(Q3_ERR_INVALID_ARG, "op_kv_pack_q8_0: bad argument");
    const cudaError_t e = launch_kv_pack_q8(static_cast<cudaStream_t>(stream), rows_dev, n_rows,
                                            static_cast<uint8_t*>(out_dev));
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "op_kv_pack_q8_0: %s", cudaGetErrorString(e));
    return Q3_OK;
}

// One GEMM of the operator gates on caller buffers: planned (block_n 0) or
// forced tile width and split-K, with the prefill path's epilogues.  Owns a
// status word and, for split-K, a partial-sum workspace for the call, and
// returns once the kernels have finished: a bounded device wait that ran out
// (or an fp16 output beyond range) is reported, never hidden.
int op_gemm_sync(const char* name, const void* w_dev, const void* w2_dev, const void* x_dev, int M, int N,
                 int K, int epi, void* out_dev, int block_n, int k_splits, void* stream)
{
    const bool pair = epi == EPI_SWIGLU_F16;
    const int MA = pair ? 2 * M : M;          // GEMM rows: gate and up rows interleaved by 64-row tiles
    int bn = block_n, splits = k_splits;
    if (bn == 0 || splits == 0) {
        int pbn, ps;
        plan_gemm_impl(MA, N, K, k_splits == 0 ? (size_t)8 * N * MA : 0, &pbn, &ps);
        if (bn == 0) bn = pbn;
        if (splits == 0) splits = ps;
    }
    if (!gemm_block_n_supported(bn)) return fail(Q3_ERR_INVALID_ARG, "%s: unsupported block_n", name);
    if (splits < 1 || splits > 8 || K / 64 < splits)
        return fail(Q3_ERR_INVALID_ARG, "%s: k_splits must be in [1, 8] and at most K/64", name);
    CUtensorMap a0, a1, b;
    if (!tmap_f16(&a0, w_dev, M, K, pair ? 64 : 128) || (pair && !tmap_f16(&a1, w2_dev, M, K, 64)) ||
        !tmap_f16(&b, x_dev, round_up(N, 256), K, bn))
        return fail(Q3_ERR_CUDA, "%s: tensor map encoding failed", name);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int* status = nullptr;
    float* ws = nullptr;
    auto release = [&]() {
        if (status) cudaFree(status);
        if (ws) cudaFree(ws);
    };
    if (cudaMalloc(&status, sizeof(int)) != cudaSuccess ||
        (splits > 1 && cudaMalloc(&ws, sizeof(float) * (size_t)splits * N * MA) != cudaSuccess)) {
        release();
        return fail(Q3_ERR_OOM, "%s: workspace allocation failed", name);
    }
    GemmArgs g{};
    g.M = MA; g.N = N; g.K = K;
    g.a_tiles0 = g.a_tiles1 = MA / 128;
    g.pair = pair ? 1 : 0;
    g.k_splits = splits;
    g.epi = epi;
    g.out = out_dev; g.ldo = M;
    g.ws = ws;
    g.status = status;
    Launch L{st, false, nullptr};
    cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int), st);
    if (e == cudaSuccess) e = launch_gemm(L, a0, pair ? a1 : a0, a0, b, bn, g);
    if (e == cudaSuccess && splits > 1) e = launch_gemm_splitk_reduce(L, g);
    int word = 0;
    if (e == cudaSuccess) e = cudaMemcpyAsync(&word, status, sizeof(int), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    release();
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
    if (word) return fail(Q3_ERR_DEVICE_CHECK, "%s: device status 0x%x", name, word);
    return Q3_OK;
}

int q3_op_matmul(const void* w_dev, const void* x_dev, int M, int N, int K, float* y_dev, int block_n,
                 void* stream)
{
    if (!w_dev || !x_dev || !y_dev || M < 128 || M % 128 || K < 64 || K % 64 || N < 1 ||
        !aligned16(w_dev) || !aligned16(x_dev))
        return fail(Q3_ERR_INVALID_ARG, "op_matmul: bad argument");
    return op_gemm_sync("op_matmul", w_dev, nullptr, x_dev, M, N, K, EPI_STORE_F32, y_dev, block_n, 1, stream);
}

int q3_attention_plan(int n_kv_heads, int T, int max_ctx, int* n_splits)
{
    if (!n_splits || n_kv_heads < 1 || n_kv_heads > 64 || T < 1 || T > (1 << 16) || max_ctx < 1 ||
        max_ctx > (1 << 24))
        return fail(Q3_ERR_INVALID_ARG, "attention_plan: bad argument");
    *n_splits = attention_splits_impl(n_kv_heads, T, max_ctx, ATTN_PART_ROWS);
    return Q3_OK;
}

int q3_gemm_plan(int M, int N, int K, int* block_n, int* k_splits)
{
    // sizes up to 2^18 keep the planner's tile and round counts inside int
    constexpr int LIMIT = 1 << 18;
    if (!block_n || !k_splits || M < 128 || M % 128 || K < 64 || K % 64 || N < 1 || M > LIMIT || N > LIMIT ||
        K > LIMIT)
        return fail(Q3_ERR_INVALID_ARG, "gemm_plan: bad argument");
    plan_gemm_impl(M, N, K, SPLITK_WS_ELEMS, block_n, k_splits);
    return Q3_OK;
}

int q3_op_gemm(const void* w_dev, const void* w2_dev, const void* x_dev, int M, int N, int K, int epi,
               void* out_dev, int block_n, int k_splits, void* stream)
{
    const bool pair = epi == Q3_OP_SWIGLU;
    if (!w_dev || !x_dev || !out_dev || (pair && !w2_dev) || N < 1 || K < 64 || K % 64 ||
        M < (pair ? 64 : 128) || M % (pair ? 64 : 128) || !aligned16(w_dev) || !aligned16(x_dev) ||
        (pair && !aligned16(w2_dev)) || k_splits < 0 || block_n < 0)
        return fail(Q3_ERR_INVALID_ARG, "op_gemm: bad argument");
    int kepi;
    switch (epi) {
    case Q3_OP_STORE: kepi = EPI_STORE_F32; break;
    case Q3_OP_ADD: kepi = EPI_ADD_F32; break;
    case Q3_OP_SWIGLU: kepi = EPI_SWIGLU_F16; break;
    default: return fail(Q3_ERR_INVALID_ARG, "op_gemm: unknown epilogue %d", epi);
    }
    return op_gemm_sync("op_gemm", w_dev, w2_dev, x_dev, M, N, K, kepi, out_dev, block_n, k_splits, stream);
}

int q3_op_matvec(const void* w_dev, const void* scales_dev, const float* x_dev, int M, int K,
                 float* y_dev, void* stream)
{
    if (!w_dev || !x_dev || !y_dev || M < 8 || M % 8 || K < 256 || K % 256 || !aligned16(w_dev) ||
        !aligned16(x_dev) || (scales_dev && !aligned16(scales_dev)))
        return fail(Q3_ERR_INVALID_ARG, "op_matvec: bad argument");
    GemvArgs a{};
    a.w[0] = w_dev;
    a.scales[0] = static_cast<const __half*>(scales_dev);
    a.rows[0] = M;
    a.n_tensors = 1;
    a.K = K;
    a.warps_per_row = gemv_warps_per_row(M, K, scales_dev ? Q3_Q8_0 : Q3_BF16, 0);
    a.x = x_dev;
    a.epi = EPI_STORE_F32;
    a.out = y_dev;
    Launch L{static_cast<cudaStream_t>(stream), false, nullptr};
    cudaError_t e = launch_gemv(L, scales_dev ? Q3_Q8_0 : Q3_BF16, a);
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "op_matvec: %s", cudaGetErrorString(e));
    return Q3_OK;
}

int q3_op_matvec_affine4(const void* groups_dev, const float* x_dev, int M, int K, float* y_dev, void* stream)
{
    if (!groups_dev || !x_dev || !y_dev || M < 8 || M % 8 || K < 128 || K % 128 || K > 32768 ||
        (reinterpret_cast<uintptr_t>(groups_dev) & 3) || !aligned16(x_dev))
        return fail(Q3_ERR_INVALID_ARG, "op_matvec_affine4: bad argument");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* codes = nullptr;
    void* sb = nullptr;
    int* status = nullptr;
    auto release = [&]() { cudaFree(codes); cudaFree(sb); cudaFree(status); };
    const size_t n = (size_t)M * K;
    if (cudaMalloc(&codes, n / 2) != cudaSuccess || cudaMalloc(&sb, n / 32 * 4) != cudaSuccess ||
        cudaMalloc(&status, sizeof(int)) != cudaSuccess) {
        release();
        return fail(Q3_ERR_OOM, "op_matvec_affine4: allocation failed");
    }
    GemvArgs a{};
    a.w[0] = codes;
    a.scales[0] = static_cast<const __half*>(sb);
    a.rows[0] = M;
    a.n_tensors = 1;
    a.K = K;
    a.warps_per_row = gemv_a4_warps_per_tile(M, K, 0);
    a.x = x_dev;
    a.epi = EPI_STORE_F32;
    a.out = y_dev;
    a.status = status;
    Launch L{st, false, nullptr};
    cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int), st);
    if (e == cudaSuccess) e = launch_a4_planes(st, static_cast<const uint8_t*>(groups_dev), M, K, codes, sb);
    if (e == cudaSuccess) e = launch_gemv_a4(L, a);
    int word = 0;
    if (e == cudaSuccess) e = cudaMemcpyAsync(&word, status, sizeof(int), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    release();
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "op_matvec_affine4: %s", cudaGetErrorString(e));
    if (word) return fail(Q3_ERR_DEVICE_CHECK, "op_matvec_affine4: device status 0x%x", word);
    return Q3_OK;
}

int q3_op_prefill_attention(const void* q_dev, const void* kv_dev, const int32_t* table_dev, int n_table,
                            int n_blocks, int pos0, int T, int n_q, int n_kv, void* out_dev, int use_tc,
                            void* stream)
{
    if (!q_dev || !kv_dev || !table_dev || !out_dev || T < 1 || pos0 < 0 || n_kv < 1 || n_q < 1 ||
        n_q % n_kv || n_blocks < 1 || n_table < (pos0 + T + 31) / 32 || !aligned16(q_dev) ||
        !aligned16(kv_dev) || !aligned16(out_dev))
        return fail(Q3_ERR_INVALID_ARG, "op_prefill_attention: bad argument");
    if (use_tc && prefill_tc_rows(n_q, n_kv) < 1)
        return fail(Q3_ERR_INVALID_ARG, "op_prefill_attention: tcgen05 kernel unsupported for these heads");
    int dev = 0, n_sm = 0, optin = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
        return fail(Q3_ERR_CUDA, "op_prefill_attention: no CUDA device");
    if (use_tc && prefill_tc_smem() > (size_t)optin)
        return fail(Q3_ERR_INVALID_ARG, "op_prefill_attention: not enough shared memory");
    // host-built metadata, as a round builds it: rows, tiles (longest
    // context first), schedule, then the work counter and the status word
    const int R = use_tc ? prefill_tc_rows(n_q, n_kv) : 64;
    std::vector<int> row_pos(T), row_slot(T, 0), t_row0, t_rows;
    for (int t = 0; t < T; ++t) row_pos[t] = pos0 + t;
    for (int k = ((T - 1) / R) * R; k >= 0; k -= R) {
        t_row0.push_back(k);
        t_rows.push_back(std::min(R, T - k));
    }
    const int n_tiles = (int)t_row0.size();
    std::vector<int> start, items;
    int grid = 0;
    if (use_tc) {
        const int n_items = n_tiles * n_kv;
        grid = std::max(1, std::min({n_sm, n_items, SCHED_GRID}));
        std::vector<std::vector<int>> lists(grid);
        std::vector<long long> load(grid, 0);
        for (int t = 0; t < n_tiles; ++t) {
            const long long cost = (pos0 + t_row0[t] + t_rows[t] - 1) / 128 + 2;
            for (int h = 0; h < n_kv; ++h) {
                const int c = (int)(std::min_element(load.begin(), load.end()) - load.begin());
                lists[c].push_back(t * n_kv + h);
                load[c] += cost;
            }
        }
        for (int c = 0; c < grid; ++c) {
            start.push_back((int)items.size());
            items.insert(items.end(), lists[c].begin(), lists[c].end());
        }
        start.push_back((int)items.size());
    }
    std::vector<int> meta;
    auto put = [&](const std::vector<int>& v) { size_t at = meta.size(); meta.insert(meta.end(), v.begin(), v.end()); return at; };
    const size_t o_pos = put(row_pos), o_slot = put(row_slot), o_r0 = put(t_row0), o_rows = put(t_rows);
    const size_t o_start = put(start), o_items = put(items), o_ctr = put({0, 0});
    int* dmeta = nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMalloc(&dmeta, sizeof(int) * meta.size()) != cudaSuccess)
        return fail(Q3_ERR_OOM, "op_prefill_attention: metadata allocation failed");
    PrefillAttnArgs pa{};
    pa.q = static_cast<const __half*>(q_dev);
    pa.T = T; pa.n_q = n_q; pa.n_kv = n_kv;
    pa.row_pos = dmeta + o_pos; pa.row_slot = dmeta + o_slot;
    pa.tile_row0 = dmeta + o_r0; pa.tile_rows = dmeta + o_rows; pa.n_tiles = n_tiles;
    pa.work_counter = dmeta + o_ctr;
    pa.sched_start = dmeta + o_start; pa.sched_items = dmeta + o_items;
    pa.tables = table_dev; pa.max_blocks = n_table;
    pa.kv_layer = static_cast<const bf16*>(kv_dev); pa.n_blocks = n_blocks;
    pa.out = static_cast<__half*>(out_dev);
    pa.status = dmeta + o_ctr + 1;
    pa.kv_row0 = 0;
    CUtensorMap tkv;
    if (use_tc && !tmap_kv(&tkv, kv_dev, (uint64_t)n_blocks * 2 * n_kv * 32)) {
        cudaFree(dmeta);
        return fail(Q3_ERR_CUDA, "op_prefill_attention: tensor map encoding failed");
    }
    Launch L{st, false, nullptr};
    cudaError_t e = cudaMemcpyAsync(dmeta, meta.data(), sizeof(int) * meta.size(), cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = use_tc ? launch_prefill_attention_tc(L, tkv, pa, grid) : launch_prefill_attention(L, pa);
    int status = 0;
    if (e == cudaSuccess) e = cudaMemcpyAsync(&status, pa.status, sizeof(int), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    cudaFree(dmeta);
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "op_prefill_attention: %s", cudaGetErrorString(e));
    if (status) return fail(Q3_ERR_DEVICE_CHECK, "op_prefill_attention: device status 0x%x", status);
    return Q3_OK;
}

// ---------------------------------------------------------------- 4-bit cache and scoring operators

namespace {

// what the three cache operators share: heads, tables, pool
bool kv4_counts_ok(int T, int n_q, int n_kv, int max_blocks, int n_blocks)
{
    return T >= 0 && n_kv >= 1 && n_kv <= 4096 && (int64_t)T * n_kv <= 0x7fffffff && n_q >= 1 && n_q <= 8 * n_kv &&
           n_q % n_kv == 0 && max_blocks >= 1 && max_blocks <= (1 << 20) && n_blocks >= 1;
}
bool kv4_sizes_ok(int T, int n_q, int n_kv, const void* tables, int n_slots, int max_blocks, const void* kv, int n_blocks)
{
    return kv4_counts_ok(T, n_q, n_kv, max_blocks, n_blocks) && tables && n_slots >= 1 && kv && aligned16(kv);
}

// rows of 128 in the prefill attention's copy: 32-bit coordinates of its tensor map
bool kv4_copy_ok(const Kv4Workspace& w, int n_kv) { return w.blocks * 2 * n_kv * 32 <= 0x7fffffffll; }

// A programmatic launch: a call's set-up overlaps the end of the kernel before it on
// the stream, whichever that is, and the call's kernels wait for that one before they
// read or write (calls in a row: one decode row 8.3 -> 6.4 us, a 701-row ragged prefill
// 20.6 -> 18.0).
Launch op_launch(void* stream) { return Launch{static_cast<cudaStream_t>(stream), true, nullptr}; }

bool row_stride_ok(int64_t stride, int type, int64_t width)
{
    return stride >= width && stride % (type == Q3_TYPE_F32 ? 4 : 8) == 0;
}

}  // namespace

int q3_op_kv4_append(const void* qkv_dev, int qkv_type, int64_t qkv_stride, const void* q_gain_dev,
                     const void* k_gain_dev, float eps, const float* rope_dev, int rope_len,
                     const int32_t* row_pos_dev, const int32_t* row_slot_dev, int T, int n_q, int n_kv,
                     const int32_t* tables_dev, int n_slots, int max_blocks, void* kv_dev, int n_blocks,
                     void* q_out_dev, void* kv_out_dev, int32_t* status_dev, void* stream)
{
    if (!qkv_dev || !q_gain_dev || !k_gain_dev || !rope_dev || !row_pos_dev || !row_slot_dev || rope_len < 1 ||
        !(eps >= 0.f) || !kv4_sizes_ok(T, n_q, n_kv, tables_dev, n_slots, max_blocks, kv_dev, n_blocks))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_append: bad argument");
    if (qkv_type < Q3_TYPE_F32 || qkv_type > Q3_TYPE_BF16)
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_append: unknown type %d", qkv_type);
    if (!row_stride_ok(qkv_stride, qkv_type, (int64_t)(n_q + 2 * n_kv) * 128))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_append: row stride too small or not a multiple of 16 bytes");
    if (!aligned16(qkv_dev) || !aligned16(rope_dev) || !aligned16(q_gain_dev) || !aligned16(k_gain_dev) ||
        !aligned16(q_out_dev) || !aligned16(kv_out_dev))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_append: pointers must be 16-byte aligned");
    if (T == 0) return Q3_OK;
    Kv4AppendArgs a{};
    a.qkv = qkv_dev; a.qkv_stride = qkv_stride;
    a.q_gain = static_cast<const bf16*>(q_gain_dev); a.k_gain = static_cast<const bf16*>(k_gain_dev);
    a.eps = eps;
    a.rope = reinterpret_cast<const float2*>(rope_dev); a.rope_len = rope_len;
    a.row_pos = row_pos_dev; a.row_slot = row_slot_dev;
    a.T = T; a.n_q = n_q; a.n_kv = n_kv;
    a.tables = tables_dev; a.n_slots = n_slots; a.max_blocks = max_blocks;
    a.kv = static_cast<uint8_t*>(kv_dev); a.n_blocks = n_blocks;
    a.q_out = static_cast<f16*>(q_out_dev); a.kv_out = static_cast<f16*>(kv_out_dev);
    a.status = status_dev;
    const Launch L = op_launch(stream);
    const cudaError_t e = launch_kv4_append(L, a, qkv_type);
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "op_kv4_append: %s", cudaGetErrorString(e));
    return Q3_OK;
}

int q3_op_kv4_decode_attention(const void* q_dev, int q_type, int64_t q_stride, const int32_t* row_pos_dev,
                               const int32_t* row_slot_dev, int T, int n_q, int n_kv, const int32_t* tables_dev,
                               int n_slots, int max_blocks, int max_ctx, const void* kv_dev, int n_blocks,
                               void* out_dev, int out_type, int32_t* status_dev, void* stream)
{
    if (!q_dev || !row_pos_dev || !row_slot_dev || !out_dev || max_ctx < 0 ||
        !kv4_sizes_ok(T, n_q, n_kv, tables_dev, n_slots, max_blocks, kv_dev, n_blocks) || max_ctx > 32 * max_blocks)
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_decode_attention: bad argument");
    if ((q_type != Q3_TYPE_F32 && q_type != Q3_TYPE_F16) || (out_type != Q3_TYPE_F32 && out_type != Q3_TYPE_F16))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_decode_attention: q and out are f32 or fp16");
    if (!row_stride_ok(q_stride, q_type, (int64_t)n_q * 128))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_decode_attention: row stride too small or not a multiple of 16 bytes");
    if (!aligned16(q_dev) || !aligned16(out_dev))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_decode_attention: pointers must be 16-byte aligned");
    if (T == 0) return Q3_OK;
    Kv4DecodeArgs a{};
    a.q = q_dev; a.q_stride = q_stride;
    a.row_pos = row_pos_dev; a.row_slot = row_slot_dev;
    a.T = T; a.n_q = n_q; a.n_kv = n_kv;
    a.tables = tables_dev; a.n_slots = n_slots; a.max_blocks = max_blocks;
    a.max_ctx = max_ctx ? max_ctx : 32 * max_blocks;
    a.kv = static_cast<const uint8_t*>(kv_dev); a.n_blocks = n_blocks;
    a.out = out_dev; a.status = status_dev;
    const Launch L = op_launch(stream);
    const cudaError_t e = launch_kv4_decode(L, a, q_type, out_type);
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "op_kv4_decode_attention: %s", cudaGetErrorString(e));
    return Q3_OK;
}

int q3_kv4_prefill_workspace(int ns, int T, int n_q, int n_kv, int max_blocks, int n_blocks, int64_t* bytes)
{
    if (!bytes || ns < 0 || !kv4_counts_ok(T, n_q, n_kv, max_blocks, n_blocks))
        return fail(Q3_ERR_INVALID_ARG, "kv4_prefill_workspace: bad argument");
    const Kv4Workspace w = kv4_workspace(ns, T, n_q, n_kv, max_blocks, n_blocks);
    if (!kv4_copy_ok(w, n_kv)) return fail(Q3_ERR_INVALID_ARG, "kv4_prefill_workspace: more than 2^31 cache rows in one call");
    *bytes = (int64_t)w.bytes;
    return Q3_OK;
}

int q3_op_kv4_prefill_attention(const void* q_dev, int64_t q_stride, const int32_t* seq_rows_dev,
                                const int32_t* seq_pos_dev, const int32_t* seq_slot_dev, int ns, int T, int n_q,
                                int n_kv, const int32_t* tables_dev, int n_slots, int max_blocks, const void* kv_dev,
                                int n_blocks, void* out_dev, void* workspace_dev, int64_t workspace_bytes,
                                int32_t* status_dev, void* stream)
{
    if (!q_dev || !seq_rows_dev || !seq_pos_dev || !out_dev || ns < 0 ||
        !kv4_sizes_ok(T, n_q, n_kv, tables_dev, n_slots, max_blocks, kv_dev, n_blocks) || (!seq_slot_dev && ns > n_slots))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_prefill_attention: bad argument");
    if (!row_stride_ok(q_stride, Q3_TYPE_F16, (int64_t)n_q * 128))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_prefill_attention: row stride too small or not a multiple of 16 bytes");
    const Kv4Workspace w = kv4_workspace(ns, T, n_q, n_kv, max_blocks, n_blocks);
    if (!kv4_copy_ok(w, n_kv))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_prefill_attention: more than 2^31 cache rows in one call");
    if (T > 0 && ns > 0 && (!workspace_dev || workspace_bytes < (int64_t)w.bytes || (reinterpret_cast<uintptr_t>(workspace_dev) & 255)))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_prefill_attention: workspace of %lld bytes, 256-byte aligned", (long long)w.bytes);
    if (!aligned16(q_dev) || !aligned16(out_dev))
        return fail(Q3_ERR_INVALID_ARG, "op_kv4_prefill_attention: pointers must be 16-byte aligned");
    if (T == 0 || ns == 0) return Q3_OK;
    Kv4PrefillArgs a{};
    a.q = static_cast<const f16*>(q_dev); a.q_stride = q_stride;
    a.seq_rows = seq_rows_dev; a.seq_pos = seq_pos_dev; a.seq_slot = seq_slot_dev;
    a.ns = ns; a.T = T; a.n_q = n_q; a.n_kv = n_kv;
    a.tables = tables_dev; a.n_slots = n_slots; a.max_blocks = max_blocks;
    a.kv = static_cast<const uint8_t*>(kv_dev); a.n_blocks = n_blocks;
    a.out = static_cast<f16*>(out_dev); a.status = status_dev;
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return fail(Q3_ERR_CUDA, "op_kv4_prefill_attention: no CUDA device");
    const Launch L = op_launch(stream);
    const cudaError_t e = run_kv4_prefill(L, a, static_cast<uint8_t*>(workspace_dev), n_sm);
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "op_kv4_prefill_attention: %s", cudaGetErrorString(e));
    return Q3_OK;
}

int q3_op_token_logprobs(const void* logits_dev, int type, int64_t stride, int N, int V, const int32_t* targets_dev,
                         int top_k, float* logprob_dev, float* entropy_dev, int32_t* top_ids_dev,
                         float* top_logprob_dev, int32_t* status_dev, void* stream)
{
    if (!logits_dev || N < 0 || V < 1 || stride < V || (logprob_dev && !targets_dev))
        return fail(Q3_ERR_INVALID_ARG, "op_token_logprobs: bad argument");
    if (type < Q3_TYPE_F32 || type > Q3_TYPE_BF16)
        return fail(Q3_ERR_INVALID_ARG, "op_token_logprobs: unknown type %d", type);
    if (reinterpret_cast<uintptr_t>(logits_dev) & (type == Q3_TYPE_F32 ? 3 : 1))
        return fail(Q3_ERR_INVALID_ARG, "op_token_logprobs: logits not aligned to their type");
    if (top_k < 0 || top_k > V || top_k > Q3_LOGPROB_MAX_TOP)
        return fail(Q3_ERR_INVALID_ARG, "op_token_logprobs: top_k outside [0, min(V, %d)]", Q3_LOGPROB_MAX_TOP);
    if (N == 0) return Q3_OK;
    LogprobArgs a{};
    a.logits = logits_dev; a.stride = stride; a.N = N; a.V = V;
    a.top = top_ids_dev || top_logprob_dev ? top_k : 0;
    a.targets = targets_dev; a.logprob = logprob_dev; a.entropy = entropy_dev;
    a.top_ids = top_ids_dev; a.top_logprob = top_logprob_dev;
    a.status = status_dev;
    const Launch L = op_launch(stream);
    const cudaError_t e = launch_logprobs(L, a, type);
    if (e != cudaSuccess) return fail(Q3_ERR_CUDA, "op_token_logprobs: %s", cudaGetErrorString(e));
    return Q3_OK;
}

}  // extern "C"
