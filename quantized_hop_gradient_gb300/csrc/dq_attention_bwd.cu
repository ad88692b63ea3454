// dq_attention_bwd.cu -- the attention backward kernels.
//
// Two kernels, so that every sum has one owner and no result depends on the
// order of blocks: one owns a tile of queries and sums dq over the keys, one
// owns a tile of keys and sums dk and dv over the queries and over the heads
// of its group.  Both compute the scores and dP again: seven products where a
// single kernel that adds dq up in turns, key tile by key tile, would need five
// and as many fp32 additions to memory as there are key tiles.
//
//   P = exp(scale q k^T - lse);  dP = dout v^T;  dS = P (dP - delta) scale
//   delta = sum_j P dP = dout . out;  dq = dS k;  dk = dS^T q;  dv = P^T dout
//
// P and dS are rounded to 16 bits because the tensor core multiplies them with
// 16-bit operands; delta of rows with more than one key tile comes from out as
// it is stored, in 16 bits, since a sum of P dP would need another pass over
// the keys.  These roundings are what the gradients' error over the plain
// 32-bit form's comes from (0.0024 against 0.0017 of their norm in bf16).
//
// What bounds them (bf16, causal): 12,291 tokens of 32 heads of 128 over 8: dq
// 581 us, dk and dv 783 us, 1.76 PFLOP/s over the seven products, 0.93 of the
// library's plain product; tensor pipe 78% and 76% active, issue slots 40% and
// 33%; in a long loop the card is at its power limit.  5,096 tokens of 32 heads of
// 64 over 8: 71 and 71 us, tensor pipe 32% and 41%, issue slots 42% and 50%,
// exp's unit 23% and 23%: the arithmetic between the products, which are half as
// long there, one tile's at a time.  fp16, with its factors (below): 28 us of
// norms, 612 and 814 us; 10, 73 and 75 us.
#include <float.h>

#include <algorithm>

#include "dq_attention.cuh"

namespace dq {
namespace {

using namespace tc;

constexpr float kLog2e = 1.44269504088896340736f;

// P is held times a power of two until the last step.  bf16, 2^16: so that
// exp2, which gives 0 below 2^-126, loses nothing that bf16 can hold (down to
// 2^-133).  fp16, 2^12: its steps are 2^-24 below 2^-14, which is the average
// weight of 16,384 keys, and P is at most 1 but for the rounding of scores and
// lse, to which a factor of 15 is left (scores beyond 10^7).
template <typename T> __host__ __device__ constexpr float p_shift() { return __is_same(T, __nv_bfloat16) ? 16.0f : 12.0f; }
template <typename T> __host__ __device__ constexpr float p_unshift() { return __is_same(T, __nv_bfloat16) ? 1.0f / 65536.0f : 1.0f / 4096.0f; }

// ------------------------------------------------------------------ fp16's range
// dP - delta can pass 65,504 where the gradients do not (12,000 x 128 elements),
// and dS of small gradients lies below 2^-24 where they do not.  So fp16 holds
// dS times a power of two F with |dP - delta| F <= 1, times P's 2^12:
// |dP_ij| <= |dout_i| |v_j|, and delta, a mean of dP, is below the largest, so
// |dP - delta| <= B = 2 |dout_i| max |v_j|.  dq is summed over keys and takes an
// F for each row, from the keys that its tile reads; dk is summed over rows and
// takes one for a tile of keys, from the rows that it reads (a row whose dout is
// 2^-20 of the largest one's then loses bits of its share).  Both depend on
// their own sequence only.  Norms that are not finite are left out: every
// gradient that their row or key enters is not finite either.
__device__ __forceinline__ float range_factor(float bound)   // F in (1 / (2 B), 1 / B]
{
    return bound > 0.0f ? __uint_as_float((253u - (__float_as_uint(bound) >> 23)) << 23) : 1.0f;
}
__device__ __forceinline__ float range_inverse(float factor) { return __uint_as_float((254u << 23) - __float_as_uint(factor)); }

// The largest of the norms of `n` tiles of each of `heads` heads that lie n_tokens apart, `first` being the first one's
// first row; called by whole warps.
__device__ __forceinline__ float largest_norm(const float *norms, int64_t first, int n, int heads, int64_t n_tokens)
{
    float m = 0.0f;
    for (int i = threadIdx.x & 31; i < n * heads; i += 32) m = fmaxf(m, norms[first + i / n * n_tokens + i % n * kTile]);
    return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(m)));   // not negative: ordered as their bits are
}

// Norms of dout's rows and the largest of each tile of dout and v.  Bound by
// memory, as dout and v are read once more: 12,291 tokens of 32 heads of 128 over
// 8, 126 MB, 28 us, 4.5 TB/s; by the search and the loads behind it when there
// are few: 300 tokens of 4 heads 7 us.  A warp takes 32 rows of a tile, a row on
// 8 or 16 lanes.
template <typename T, int BOXES> __global__ void __launch_bounds__(128) attention_norms_kernel(const __grid_constant__ AttentionParams P)
{
    constexpr int kLanes = 8 * BOXES, kAtOnce = 32 / kLanes, kLoads = 8;
    __shared__ float part[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / kLanes, piece = lane % kLanes * 8;
    Slot S;
    if (!find_slot(P.cu, P.n_seqs, P.n_tokens, blockIdx.x, kTile, S) || S.padding) return;
    const int first = S.row + 32 * warp, live = S.len - first;   // rows of this warp that exist
    for (int y = blockIdx.y; y < P.n_heads + P.n_kv; y += gridDim.y) {
        const bool is_v = y >= P.n_heads;
        const Heads<T> x = heads<T>(is_v ? P.v : P.dout);
        const int h = is_v ? y - P.n_heads : y;
        float top = 0.0f;
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += kLoads * kAtOnce) {
            Raw8<T> g[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int r = r0 + k * kAtOnce + sub;
                g[k] = Raw8<T>{};
                if (r < live && piece < P.dim) g[k] = load8(x.at(S.lo + first + r, h) + piece);
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int r = r0 + k * kAtOnce + sub;
                const F8 a = widen<T>(g[k]);
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(a.v[e], a.v[e], sum);
#pragma unroll
                for (int m = kLanes / 2; m; m >>= 1) sum += __shfl_xor_sync(kFull, sum, m);
                const float norm = sum <= FLT_MAX ? sqrtf(sum) : 0.0f;
                top = fmaxf(top, norm);
                if (!is_v && piece == 0 && r < live) P.row_norms[(int64_t)h * P.n_tokens + S.lo + first + r] = norm;
            }
        }
        top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
        __syncthreads();   // the last head's are read
        if (lane == 0) part[warp] = top;
        __syncthreads();
        if (threadIdx.x == 0)
            P.tile_norms[(int64_t)y * P.n_tokens + S.lo + S.row] = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    }
}

// lse log2(e), less the shift: exp2(S scale log2(e) - this) is P, shifted.  A row
// without any weight (lse = -inf) has P = 0, as if its lse were infinite.
template <typename T> __device__ __forceinline__ float scaled_lse(float lse)
{
    return lse == -INFINITY ? INFINITY : lse * kLog2e - p_shift<T>();
}

// N columns of a thread's own row from tensor memory, and N values packed to
// 16 bits and stored over the first half of N columns.
template <int N> __device__ __forceinline__ void load_part(uint32_t t, uint32_t *s)
{
#pragma unroll
    for (int i = 0; i < N; i += 32) tmem_load32(t + i, s + i);
    wait_ld();
}
template <typename T, int N> __device__ __forceinline__ void store_part(uint32_t t, const float2 *v)
{
#pragma unroll
    for (int h = 0; h < N / 32; ++h) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack2(v[16 * h + i].x, v[16 * h + i].y, T());
        tmem_store16(t + 16 * h, w);
    }
}

// For a block that gives up, by its product warp after the block's last barrier.
__device__ __forceinline__ void drain_products(uint32_t bar)
{
    if (elect_one()) commit(bar);
    __syncwarp();
    mbar_land(bar, 0);
}

// ------------------------------------------------------------------ dq
// Warp 0: products, by one thread; 1: the tiles and copies; 2: clearing; 4-7:
// the rows' lse and delta; 8-15 (columns 0-63 and 64-127 of a tile): P and dS,
// a thread half a row.  (Four warpgroups with a quarter each: 644 against 626
// us for 12,291 tokens of 32 heads, and no registers left to load ahead.)
// Registers: 4 warpgroups of 128 at launch = 2 x 168 + 2 x 88.
constexpr int kThreadsQ = 512, kLaunchRegsQ = 128, kComputeRegs = 168, kOtherRegs = 88, kPartsQ = 2;
static_assert(2 * kComputeRegs + 2 * kOtherRegs == 4 * kLaunchRegsQ, "register shares");
constexpr int kProductWarp = 0, kCopyWarp = 1, kClearWarpQ = 2, kRowWarpsQ = 4, kComputeWarpQ = 8;
template <int BOXES> __host__ __device__ constexpr int stages_k() { return BOXES == 1 ? 5 : 3; }
template <int BOXES> __host__ __device__ constexpr int stages_v() { return BOXES == 1 ? 4 : 2; }

template <int BOXES> struct BarsQ {
    ItemQueue queue;
    unsigned long long q_full, q_empty, k_full[stages_k<BOXES>()], k_clear[stages_k<BOXES>()], k_empty[stages_k<BOXES>()];
    unsigned long long v_full[stages_v<BOXES>()], v_empty[stages_v<BOXES>()], rows_full, rows_empty;
    unsigned long long s_full[2], dp_full, ds_ready, delta_ready, done, dq_free, drained;
    uint32_t tmem;
    int abort;
    float rows[3][kTile];         // lse log2(e) (shifted), delta and (fp16) F of the item's queries
    float delta[kPartsQ][kTile];   // the parts' shares of a delta that comes from P dP
};

template <int BOXES> constexpr int smem_bytes_q()
{
    return (2 + stages_k<BOXES>() + stages_v<BOXES>()) * BOXES * kBoxBytes + (int)sizeof(BarsQ<BOXES>);
}
static_assert(smem_bytes_q<2>() <= 227 * 1024, "shared memory");

template <typename T, int STEPS, bool SPLIT> __global__ void __launch_bounds__(kThreadsQ, 1)
    attention_dq_kernel(const __grid_constant__ AttentionParams P)
{
    constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
    constexpr int BOXES = boxes(STEPS);
    constexpr int kDim = 64 * BOXES, kK = stages_k<BOXES>(), kV = stages_v<BOXES>();
    constexpr uint32_t kTileBytes = BOXES * kBoxBytes;
    // Wide heads take the next item with four copies of this one to come: its rows' delta takes 8,600 cycles to load and
    // add up, longer than the copies run ahead (12,291 tokens of 32 heads in two sequences: 583 us, 600 without; 8,192 in
    // four: 160, 170; narrow heads, whose copies run further ahead: nothing gained).
    constexpr int kAhead = BOXES == 1 ? 0 : 4;
    extern __shared__ __align__(1024) uint8_t smem[];
    auto *bars = reinterpret_cast<BarsQ<BOXES> *>(smem + (2 + kK + kV) * kTileBytes);
    const uint32_t s_q = smem_addr(smem), s_do = s_q + kTileBytes, s_k = s_do + kTileBytes, s_v = s_k + kK * kTileBytes;
    const uint32_t q_full = smem_addr(&bars->q_full), q_empty = smem_addr(&bars->q_empty);
    const uint32_t k_full = smem_addr(bars->k_full), k_clear = smem_addr(bars->k_clear), k_empty = smem_addr(bars->k_empty);
    const uint32_t v_full = smem_addr(bars->v_full), v_empty = smem_addr(bars->v_empty), s_full = smem_addr(bars->s_full);
    const uint32_t dp_full = smem_addr(&bars->dp_full), ds_ready = smem_addr(&bars->ds_ready);
    const uint32_t rows_full = smem_addr(&bars->rows_full), rows_empty = smem_addr(&bars->rows_empty);
    const uint32_t delta_ready = smem_addr(&bars->delta_ready), done = smem_addr(&bars->done);
    const uint32_t dq_free = smem_addr(&bars->dq_free);
    volatile int *abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == kCopyWarp) {
        if (lane == 0) {
            prefetch_map(&P.map_q);
            prefetch_map(&P.map_dout);
            prefetch_map(&P.map_k);
            prefetch_map(&P.map_v);
            init_queue(&bars->queue, 14);   // products, clearing, 4 of rows, 8 of P and dS
            mbar_init(q_full, 1);
            mbar_init(q_empty, 1);
            for (int i = 0; i < kK; ++i) {
                mbar_init(k_full + 8 * i, 1);
                mbar_init(k_clear + 8 * i, 1);
                mbar_init(k_empty + 8 * i, 1);
            }
            for (int i = 0; i < kV; ++i) {
                mbar_init(v_full + 8 * i, 1);
                mbar_init(v_empty + 8 * i, 1);
            }
            mbar_init(rows_full, 4);
            mbar_init(rows_empty, 4 * kPartsQ);
            mbar_init(s_full, 1);
            mbar_init(s_full + 8, 1);
            mbar_init(dp_full, 1);
            mbar_init(ds_ready, 4 * kPartsQ);
            mbar_init(delta_ready, 4 * kPartsQ);
            mbar_init(done, 1);
            mbar_init(dq_free, 4 * kPartsQ);
            mbar_init(smem_addr(&bars->drained), 1);
            bars->abort = P.give_up;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == kProductWarp) {
        tmem_alloc<512>(smem_addr(&bars->tmem));
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars->tmem, t_dp = tmem + 2 * kTile, t_dq = tmem + 3 * kTile;   // S: two buffers from 0
    const int group = P.n_heads / P.n_kv;
    Tiles tiles{&bars->queue, abort};
    Item it;
    const int split = SPLIT ? P.split : 1, rank = SPLIT ? cluster_rank() : 0;
    auto key_tiles = [&](const Item &x) { return ((P.causal ? min(x.row + kTile, x.len) : x.len) + kTile - 1) / kTile; };
    // the block's key tiles [first, first + n); with a cluster a block may have none
    auto part_of = [&](const Item &x) { return Part(key_tiles(x), rank, split); };
    Ring<kK> rk;        // key tiles copied, cleared or scored
    Ring<kV> rv;
    int copied_q = 0;   // query tiles copied (copy warp)

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------ tiles and copies
        give_registers<kOtherRegs>();
        const int slots = gridDim.x / (P.y * split);
        auto padding = [&](const Slot &S, int y) {
            if (rank == 0) zero_heads<T>(P.dqv, S.lo + S.row, min(kTile, S.len - S.row), y, P.dim);
        };
        Taker taker{&bars->queue, abort, blockIdx.x / split};
        taker.claims = !SPLIT;   // a cluster does its one tile
        bool ok = true;
        int n = 0, hk = 0, j0 = 0;
        auto begin = [&]() {
            const Part part = part_of(it);
            n = part.n, j0 = SPLIT ? part.first : 0, hk = it.y / group;
            if (SPLIT && !n) return true;
            if (copied_q && !mbar_wait(q_empty, (copied_q - 1) & 1, abort)) return false;
            if (lane == 0) {
                mbar_expect(q_full, 2 * kTileBytes);
                for (int b = 0; b < BOXES; ++b) {
                    load_box(s_q + b * kBoxBytes, &P.map_q, 64 * b, it.y, it.lo + it.row, q_full);
                    load_box(s_do + b * kBoxBytes, &P.map_dout, 64 * b, it.y, it.lo + it.row, q_full);
                }
            }
            ++copied_q;
            return true;
        };
        auto copy = [&](int j) {
            if (rk.laps && !mbar_wait(k_empty + 8 * rk.stage, rk.phase ^ 1, abort)) return false;
            if (lane == 0) {
                mbar_expect(k_full + 8 * rk.stage, kTileBytes);
                for (int b = 0; b < BOXES; ++b)
                    load_box(s_k + rk.stage * kTileBytes + b * kBoxBytes, &P.map_k, 64 * b, hk, it.lo + (j0 + j) * kTile,
                             k_full + 8 * rk.stage);
            }
            __syncwarp();
            rk.step();
            if (rv.laps && !mbar_wait(v_empty + 8 * rv.stage, rv.phase ^ 1, abort)) return false;
            if (lane == 0) {
                mbar_expect(v_full + 8 * rv.stage, kTileBytes);
                for (int b = 0; b < BOXES; ++b)
                    load_box(s_v + rv.stage * kTileBytes + b * kBoxBytes, &P.map_v, 64 * b, hk, it.lo + (j0 + j) * kTile,
                             v_full + 8 * rv.stage);
            }
            __syncwarp();
            rv.step();
            return true;
        };
        if constexpr (kAhead == 0) {
            while (ok && taker.next<false, true>(P, slots, kTile, it, padding) == Taker::kTaken) {
                ok = begin();
                for (int j = 0; ok && j < n; ++j) ok = copy(j);
            }
        } else {
            // One place that looks for the next item, from step `ask` of the one before on (code that a block runs once or
            // twice is read from memory; narrow heads in this form: 8 sequences of 1,024 86.7 us, 84 in the plain one).  One
            // block's slot for each copy: slots without a tile may be many, and the copies are waited for.
            Item next;
            Taker::Found found = Taker::kNothing;
            for (int j = 0, ask = 0; ok; ++j) {
                if (j >= ask && found == Taker::kNothing) {
                    do found = taker.next<false, true, true>(P, slots, kTile, next, padding);
                    while (found == Taker::kNothing && j == n);
                    if (!(ok = found != Taker::kOutOfTime)) break;
                }
                if (j == n) {
                    if (found == Taker::kEnd) break;
                    it = next;
                    found = Taker::kNothing;
                    if (!(ok = begin())) break;
                    j = 0, ask = n > kAhead ? n - kAhead : n;
                    if (SPLIT && !n) {   // the part of a cluster that has no keys
                        --j;
                        continue;
                    }
                }
                ok = copy(j);
            }
        }
    } else if (warp == kProductWarp) {
        // ------------------------------------------------------------ products: one thread
        give_registers<kOtherRegs>();
        constexpr uint32_t kInstrS = instr(kBf16, kTile, false), kInstrD = instr(kBf16, 16 * STEPS, true);
        if (elect_one()) {   // (alone: with a second condition the compiler no longer sees one thread, 843 us for 798)
            const uint32_t o_q = operand<SPLIT>(s_q), o_do = operand<SPLIT>(s_do), o_k = operand<SPLIT>(s_k), o_v = operand<SPLIT>(s_v);
            Ring<kK> rd;                   // the key tile of the next dq product
            uint32_t scored = 0, begun = 0, used = 0, items = 0;   // S, dP and dq products issued, items begun
            bool ok = true;
            while (ok && tiles.next<true>(it)) {
                const int n = part_of(it).n;
                if (SPLIT && !n) continue;
                auto scores = [&]() {      // S of the next tile, into the buffers in turn
                    if (!mbar_wait_one(k_clear + 8 * rk.stage, rk.phase, abort)) return false;
                    product_abt<STEPS>(tmem + (scored & 1) * kTile, o_q, o_k + rk.stage * kTileBytes, kInstrS);
                    commit(s_full + 8 * (scored & 1));
                    ++scored;
                    rk.step();
                    return true;
                };
                auto grads = [&](int j) {  // dP of tile j
                    product_abt<STEPS>(t_dp, o_do, o_v + rv.stage * kTileBytes, kInstrS);
                    commit(dp_full);
                    commit(v_empty + 8 * rv.stage);
                    if (j + 1 == n) commit(q_empty);   // the last product that reads q or dout
                    ++begun;
                    rv.step();
                };
                if (!(ok = mbar_wait_one(q_full, items & 1, abort) && scores() && mbar_wait_one(v_full + 8 * rv.stage, rv.phase, abort)))
                    break;
                if (n > 1) {
                    grads(0);
                    if (!(ok = scores())) break;
                } else {
                    grads(0);
                }
                for (int j = 0; j < n; ++j) {
                    if (j + 1 < n && !(ok = mbar_wait_one(v_full + 8 * rv.stage, rv.phase, abort))) break;
                    if (!(ok = mbar_wait_one(ds_ready, used & 1, abort))) break;
                    fence_after();
                    // dP of the next tile first: the threads need it next, and they are done with this one's
                    if (j + 1 < n) grads(j + 1);
                    if (j == 0 && items && !(ok = mbar_wait_one(dq_free, (items - 1) & 1, abort))) break;   // read
                    if (j == 0) fence_after();
                    product_ab<kPartsQ>(t_dq, tmem + (used & 1) * kTile, o_k + rd.stage * kTileBytes, kInstrD, j > 0);
                    commit(k_empty + 8 * rd.stage);
                    if (j + 1 == n) commit(done);
                    ++used;
                    rd.step();
                    if (j + 2 < n && !(ok = scores())) break;   // over this tile's dS: products run in order
                }
                ++items;
            }
        }
        __syncwarp();
    } else if (warp == kClearWarpQ) {
        // ------------------------------------------------------------ key rows behind the sequence's end
        // have dS = 0, which a NaN or an infinity would survive; every tile passes here, so that no barrier can run a
        // phase ahead of its waiters
        give_registers<kOtherRegs>();
        bool ok = true;
        while (ok && tiles.next(it)) {
            const Part part = part_of(it);
            for (int j = part.first; j < part.first + part.n; ++j) {
                if (!(ok = mbar_wait(k_full + 8 * rk.stage, rk.phase, abort))) break;
                if ((j + 1) * kTile > it.len) zero_rows<BOXES>(s_k + rk.stage * kTileBytes, it.len - j * kTile, lane);
                if (lane == 0) mbar_arrive(k_clear + 8 * rk.stage);
                __syncwarp();
                rk.step();
            }
        }
    } else if (warp < kRowWarpsQ) {
        give_registers<kOtherRegs>();
    } else if (warp < kComputeWarpQ) {
        // ------------------------------------------------------------ the queries' lse and delta
        give_registers<kOtherRegs>();
        constexpr int kLanes = kDim / 8, kAtOnce = 32 / kLanes, kLoads = 32 / kAtOnce < 8 ? 32 / kAtOnce : 8;
        const int first = 32 * (warp - kRowWarpsQ), sub = lane / kLanes, piece = lane % kLanes * 8;   // kLanes lanes a row
        bool ok = true;
        for (int items = 0; ok && tiles.next(it); ++items) {
            const Heads<T> out = heads<T>(P.out), dout = heads<T>(P.dout);
            const int64_t at = (int64_t)it.y * P.n_tokens + it.lo + it.row;
            const int live = it.len - it.row - first;   // rows of this warp that exist
            float l = 0.0f, d = 0.0f, f = 1.0f;
            if constexpr (!kBf16) {
                const float v_max = largest_norm(P.tile_norms, (int64_t)(P.n_heads + it.y / group) * P.n_tokens + it.lo, key_tiles(it), 1, 0);
                if (lane < live) f = range_factor(2.0f * P.row_norms[at + first + lane] * v_max);
            }
            if (lane < live) l = scaled_lse<T>(P.lse[at + first + lane]);
            // Where all of a row's keys lie in one tile delta is the sum of P dP instead of dout out, which it equals:
            // the rows with few keys, whose gradients are the largest, are then free of out's rounding to 16 bits
            // (without, dq is off by 1.57 times the rounding of its own storage).
            if (key_tiles(it) > 1) {
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += kLoads * kAtOnce) {
                    Raw8<T> o[kLoads], g[kLoads];   // all on their way at once: the next tile's start waits for this
#pragma unroll
                    for (int k = 0; k < kLoads; ++k) {
                        const int r = r0 + k * kAtOnce + sub;
                        o[k] = Raw8<T>{};
                        g[k] = Raw8<T>{};
                        if (r < live && piece < P.dim) {
                            o[k] = load8(out.at(it.lo + it.row + first + r, it.y) + piece);
                            g[k] = load8(dout.at(it.lo + it.row + first + r, it.y) + piece);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kLoads; ++k) {
                        const F8 a = widen<T>(o[k]), b = widen<T>(g[k]);
                        float part = 0.0f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) part = fmaf(a.v[e], b.v[e], part);
#pragma unroll
                        for (int m = kLanes / 2; m; m >>= 1) part += __shfl_xor_sync(kFull, part, m);
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {   // row r0 + k kAtOnce + i from the i-th group of lanes
                            const float v = __shfl_sync(kFull, part, i * kLanes);
                            if (lane == r0 + k * kAtOnce + i) d = v;
                        }
                    }
                }
                if (lane < live && rank == 0) P.delta[at + first + lane] = d;
            }
            if (items && !(ok = mbar_wait(rows_empty, (items - 1) & 1, abort))) break;
            bars->rows[0][first + lane] = l;
            bars->rows[1][first + lane] = d;
            if constexpr (!kBf16) bars->rows[2][first + lane] = f;
            __syncwarp();
            if (lane == 0) mbar_arrive(rows_full);
        }
    } else {
        // ------------------------------------------------------------ P and dS
        take_registers<kComputeRegs>();
        constexpr int kCols = kTile / kPartsQ;
        const int part = (warp - kComputeWarpQ) >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const float2 c2 = make_float2(P.scale_log2, P.scale_log2);
        int g = 0, items = 0, shared = 0;   // tiles, items, and items whose delta came from their one tile
        bool ok = true;
        for (; ok && tiles.next(it); ++items) {
            const Part part_j = part_of(it);
            const int n = part_j.n, j0 = SPLIT ? part_j.first : 0, row = it.row + r;
            const bool lone = key_tiles(it) == 1;   // delta from the one tile
            if (!(ok = mbar_wait(rows_full, items & 1, abort))) break;
            const float lse2 = bars->rows[0][r];
            float delta = bars->rows[1][r];
            const float range = kBf16 ? 1.0f : bars->rows[2][r];
            __syncwarp();
            if (lane == 0) mbar_arrive(rows_empty);
            for (int j = 0; j < n; ++j, ++g) {
                if (!(ok = mbar_wait(s_full + 8 * (g & 1), (g >> 1) & 1, abort))) break;
                fence_after();
                const uint32_t t_s = tmem + (g & 1) * kTile + kCols * part + lanes;
                uint32_t s[kCols];
                float2 p[kCols / 2];
                load_part<kCols>(t_s, s);
                const float2 b2 = make_float2(-lse2, -lse2);
#pragma unroll
                for (int i = 0; i < kCols / 2; ++i) {
                    p[i] = f2_fma(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, b2);
                    p[i].x = exp2_fast(p[i].x);
                    p[i].y = exp2_fast(p[i].y);
                }
                if (!(ok = mbar_wait(dp_full, g & 1, abort))) break;
                fence_after();
                load_part<kCols>(t_dp + kCols * part + lanes, s);
                const int first = (j0 + j) * kTile + kCols * part;   // keys that the row does not see
                if (first + kCols > it.len || (P.causal && first + kCols > it.row)) {
                    const int seen = (P.causal ? min(row + 1, it.len) : it.len) - first;
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        if (i >= seen) {
                            (i & 1 ? p[i / 2].y : p[i / 2].x) = 0.0f;
                            s[i] = 0u;
                        }
                }
                if (lone) {
                    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i)
                        sum = f2_fma(p[i], make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sum);
                    // (one key: its weight is 1, not exp of a difference of rounded numbers, and dS is 0)
                    const bool sole = part == 0 && (P.causal ? min(row + 1, it.len) : it.len) == 1;
                    bars->delta[part][r] = sole ? __uint_as_float(s[0]) : (sum.x + sum.y) * p_unshift<T>();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(delta_ready);
                    if (!(ok = mbar_wait(delta_ready, shared++ & 1, abort))) break;
                    delta = bars->delta[0][r] + bars->delta[1][r];
                    if (part == 0 && row < it.len) P.delta[(int64_t)it.y * P.n_tokens + it.lo + row] = delta;
                }
                if constexpr (kBf16) {
                    const float2 d2 = make_float2(-delta, -delta);
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i)
                        p[i] = f2_mul(p[i], add2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), d2));
                } else {
                    const float2 f2 = make_float2(range, range), d2 = make_float2(-delta * range, -delta * range);
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i)
                        p[i] = f2_mul(p[i], f2_fma(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), f2, d2));
                }
                store_part<T, kCols>(t_s, p);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_ready);
            }
            if (!ok || !(ok = (SPLIT && !n) || mbar_wait(done, items & 1, abort))) break;
            fence_after();
            // each part stores its share of the columns
            constexpr int kShare = kDim / kPartsQ;
            const Heads<T> out = heads<T>(P.dqv);
            const float unrange = kBf16 ? 1.0f : range_inverse(range);
#pragma unroll
            for (int i = 0; i < kShare; i += 32) {
                uint32_t o[32];
                tmem_load32(t_dq + kShare * part + lanes + i, o);
                wait_ld();
                if (i + 32 == kShare) {   // dq may be written again
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(dq_free);
                }
                if (SPLIT) {   // in the tiles' place: this block's only item is done
                    if constexpr (!kBf16)
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * unrange);
                    leave_columns(reinterpret_cast<float *>(smem) + r * pitch<kDim>() + kShare * part + i, o, n == 0);
                } else
                    store_columns(o, P.scale * p_unshift<T>() * unrange, out.at(it.lo, it.y), out.ts, it.row + 32 * (warp & 3), it.len,
                                  kShare * part + i, P.dim);
            }
        }
    }

    fence_before();
    __syncthreads();
    if (*abort) {   // let this block's own copies and products land before its memory goes
        if (warp == kCopyWarp) {
            mbar_land(q_full, (copied_q - 1) & 1);
            for (int i = 0; i < kK; ++i, rk.step()) mbar_land(k_full + 8 * rk.stage, rk.phase ^ 1);
            for (int i = 0; i < kV; ++i, rv.step()) mbar_land(v_full + 8 * rv.stage, rv.phase ^ 1);
            if (lane == 0) *P.status = DQ_DEVICE_WAIT_TIMEOUT;
        } else if (warp == kProductWarp) {
            drain_products(smem_addr(&bars->drained));
        }
        __syncthreads();
    }
    if (warp == kProductWarp) {
        fence_after();
        tmem_free<512>(tmem);
    }
    if (SPLIT) {
        // what follows is built for the registers of the launch, and all warps run it
        __syncthreads();
        if (warp < kComputeWarpQ)
            take_registers<kLaunchRegsQ>();
        else
            give_registers<kLaunchRegsQ>();
        cluster_sync();
        it = bars->queue.item[0];   // the one item, if the cluster had any
        if (it.len >= 0 && !*abort) {
            const Heads<T> out = heads<T>(P.dqv);
            add_up_rows<T, kDim>(smem_addr(smem), rank, split, P.scale * p_unshift<T>(), out.at(it.lo, it.y), out.ts, it.row, it.len,
                                 P.dim);
        }
        cluster_sync();
    }
}

// ------------------------------------------------------------------ dk, dv
// Warp 0: products, by one thread; 1: the tiles and copies; 2: the rows' lse and delta; 3:
// clearing; from 4 on: P^T and dS^T, a thread a part of a key's row: quarters
// for narrow heads, whose products are short and leave the arithmetic to be
// hidden (80 against 88 us for 5,096 tokens of 32 heads), halves for wide ones
// (799 against 839 us for 12,291 tokens of 32 heads).  A block goes on from
// tile to tile, so that one's sums are stored beside the next one's first
// products (20 sequences of 300 tokens, 8 heads of 64: 20.3 us, 25.2 with a
// block a tile; 12,291 tokens: the same).
constexpr int kRowWarp = 2, kComputeWarp = 4;
template <int BOXES> __host__ __device__ constexpr int parts_kv() { return BOXES == 1 ? 4 : 2; }
template <int BOXES> __host__ __device__ constexpr int threads_kv() { return 128 * (1 + parts_kv<BOXES>()); }
// Registers with quarters: 5 warpgroups of 96 at launch = 4 x 104 + 64; with
// halves 3 of 168, kept.
constexpr int kLaunchRegsKV = 96, kComputeRegsKV = 104, kOtherRegsKV = 64;
static_assert(4 * kComputeRegsKV + kOtherRegsKV == 5 * kLaunchRegsKV, "register shares");
// q and dout tiles in turn: tile 2i is q of step i, 2i + 1 its dout
template <int BOXES> __host__ __device__ constexpr int ring() { return BOXES == 1 ? 9 : 5; }

// What an item reads: its steps [first, first + n) are tiles of queries, head by head.
struct Queries {
    int tile0, per_head, first, n, tiles;   // tiles: of the sequence; tile0: the first one that sees the keys
    bool ragged;                            // each head's last tile is
    __device__ __forceinline__ Queries(const AttentionParams &P, const Item &it, int rank, int split)
        : tile0(P.causal ? it.row / kTile : 0), tiles((it.len + kTile - 1) / kTile)
    {
        per_head = tiles - tile0;
        const Part part(P.n_heads / P.n_kv * per_head, rank, split);
        first = split > 1 ? part.first : 0;
        n = part.n;
        ragged = tiles * kTile > it.len;
    }
};

template <int kRing> struct BarsKV {
    ItemQueue queue;
    unsigned long long kv_full, kv_empty, sums_free, full[kRing], clear[kRing], empty[kRing], rows_full[2];
    unsigned long long s_full[2], p_ready[2], dp_full, ds_ready, done, drained;
    uint32_t tmem;
    int abort;
    float4 rows[2][2][kTile / 4];   // -lse log2(e) (shifted) and -delta (fp16: times F) of the tile's queries
    float range[4];                 // fp16: F of item i at i mod 4
};

template <int BOXES> constexpr int smem_bytes_kv()
{
    return (2 + ring<BOXES>()) * BOXES * kBoxBytes + (int)sizeof(BarsKV<ring<BOXES>()>);
}
static_assert(smem_bytes_kv<2>() <= 227 * 1024, "shared memory");

template <typename T, int STEPS, bool SPLIT> __global__ void __launch_bounds__(threads_kv<boxes(STEPS)>(), 1)
    attention_dkv_kernel(const __grid_constant__ AttentionParams P)
{
    constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
    constexpr int BOXES = boxes(STEPS);
    constexpr int kDim = 64 * BOXES;
    constexpr int kRing = ring<BOXES>(), kParts = parts_kv<BOXES>(), kCols = kTile / kParts;
    // Heads of up to 64 elements leave tensor memory for two S: the scores then run two steps ahead, and a warp may be done
    // with P of a step before another one is with P of the step before.  So the steps take turns at two p_ready barriers (dP
    // of a step follows dS of the one before, by all warps: one ds_ready).
    constexpr int kLead = BOXES == 1 ? 2 : 1;
    constexpr uint32_t kTileBytes = BOXES * kBoxBytes;
    extern __shared__ __align__(1024) uint8_t smem[];
    auto *bars = reinterpret_cast<BarsKV<kRing> *>(smem + (2 + kRing) * kTileBytes);
    const uint32_t s_k = smem_addr(smem), s_v = s_k + kTileBytes, s_ring = s_v + kTileBytes;
    const uint32_t kv_full = smem_addr(&bars->kv_full), full = smem_addr(bars->full), clear = smem_addr(bars->clear);
    const uint32_t empty = smem_addr(bars->empty);
    const uint32_t rows_full = smem_addr(bars->rows_full), s_full = smem_addr(bars->s_full);
    const uint32_t p_ready = smem_addr(bars->p_ready), dp_full = smem_addr(&bars->dp_full);
    const uint32_t ds_ready = smem_addr(&bars->ds_ready), done = smem_addr(&bars->done);
    volatile int *abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t kv_empty = smem_addr(&bars->kv_empty), sums_free = smem_addr(&bars->sums_free);
    const int split = SPLIT ? P.split : 1, rank = SPLIT ? cluster_rank() : 0, group = P.n_heads / P.n_kv;

    if (warp == kCopyWarp) {
        if (lane == 0) {
            prefetch_map(&P.map_q);
            prefetch_map(&P.map_dout);
            prefetch_map(&P.map_k);
            prefetch_map(&P.map_v);
            init_queue(&bars->queue, 3 + 4 * kParts);   // products, rows, clearing, those of P and dS
            mbar_init(kv_full, 1);
            mbar_init(kv_empty, 1);
            mbar_init(sums_free, 4 * kParts);
            for (int i = 0; i < kRing; ++i) {
                mbar_init(full + 8 * i, 1);
                mbar_init(clear + 8 * i, 1);
                mbar_init(empty + 8 * i, 1);
            }
            mbar_init(rows_full, 1);
            mbar_init(rows_full + 8, 1);
            mbar_init(s_full, 1);
            mbar_init(s_full + 8, 1);
            mbar_init(p_ready, 4 * kParts);
            mbar_init(p_ready + 8, 4 * kParts);
            mbar_init(dp_full, 1);
            mbar_init(ds_ready, 4 * kParts);
            mbar_init(done, 1);
            mbar_init(smem_addr(&bars->drained), 1);
            bars->abort = P.give_up;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == kProductWarp) {
        tmem_alloc<512>(smem_addr(&bars->tmem));
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars->tmem, t_dp = tmem + kLead * kTile, t_dv = t_dp + kTile, t_dk = t_dv + kDim;
    auto t_s = [&](int i) { return tmem + i % kLead * kTile; };
    Tiles tiles{&bars->queue, abort};
    Item it;
    int loaded = 0, items = 0;   // copies issued into the ring, items begun (copy warp)
    // steps are counted over all items: step s is in buffers s % kLead and s & 1, and its tiles are the ring's 2 s and 2 s + 1

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------ tiles and copies
        if constexpr (BOXES == 1) give_registers<kOtherRegsKV>();
        const int slots = gridDim.x / (P.y * split);
        auto padding = [&](const Slot &S, int y) {
            if (rank) return;
            zero_heads<T>(P.dk, S.lo + S.row, min(kTile, S.len - S.row), y, P.dim);
            zero_heads<T>(P.dv, S.lo + S.row, min(kTile, S.len - S.row), y, P.dim);
        };
        Taker taker{&bars->queue, abort, blockIdx.x / split};
        taker.claims = !SPLIT;   // a cluster does its one tile
        bool ok = true;
        while (ok && taker.next<true, false>(P, slots, kTile, it, padding) == Taker::kTaken) {
            const Queries Q(P, it, rank, split);
            if (SPLIT && !Q.n) continue;
            if (items && !(ok = mbar_wait(kv_empty, (items - 1) & 1, abort))) break;
            if (lane == 0) {
                mbar_expect(kv_full, 2 * kTileBytes);
                for (int b = 0; b < BOXES; ++b) {
                    load_box(s_k + b * kBoxBytes, &P.map_k, 64 * b, it.y, it.lo + it.row, kv_full);
                    load_box(s_v + b * kBoxBytes, &P.map_v, 64 * b, it.y, it.lo + it.row, kv_full);
                }
            }
            ++items;
            int head = it.y * group + Q.first / Q.per_head, at = Q.first % Q.per_head;   // of the step
            for (int e = 0; e < 2 * Q.n; ++e, ++loaded) {
                const int st = loaded % kRing;
                if (loaded >= kRing && !(ok = mbar_wait(empty + 8 * st, (loaded / kRing - 1) & 1, abort))) break;
                if (lane == 0) {
                    mbar_expect(full + 8 * st, kTileBytes);
                    for (int b = 0; b < BOXES; ++b)
                        load_box(s_ring + st * kTileBytes + b * kBoxBytes, e & 1 ? &P.map_dout : &P.map_q, 64 * b,
                                 head, it.lo + (Q.tile0 + at) * kTile, full + 8 * st);
                }
                __syncwarp();
                if (e & 1 && ++at == Q.per_head) at = 0, ++head;
            }
        }
    } else if (warp == kProductWarp) {
        // ------------------------------------------------------------ products: one thread
        if constexpr (BOXES == 1) give_registers<kOtherRegsKV>();
        constexpr uint32_t kInstrS = instr(kBf16, kTile, false), kInstrD = instr(kBf16, 16 * STEPS, true);
        if (elect_one()) {   // (alone: with a second condition the compiler no longer sees one thread, 843 us for 798)
            const uint32_t o_k = operand<SPLIT>(s_k), o_v = operand<SPLIT>(s_v), o_ring = operand<SPLIT>(s_ring);
            auto landed = [&](int e) {
                return mbar_wait_one(clear + 8 * (e % kRing), (e / kRing) & 1, abort);
            };
            auto tile = [&](int e) { return o_ring + e % kRing * kTileBytes; };
            auto scores = [&](int i) {   // S^T = k q^T
                if (!landed(2 * i)) return false;
                product_abt<STEPS>(t_s(i), o_k, tile(2 * i), kInstrS);
                commit(s_full + 8 * (i % kLead));
                return true;
            };
            auto grads = [&](int i) {    // dP^T = v dout^T
                if (!landed(2 * i + 1)) return false;
                product_abt<STEPS>(t_dp, o_v, tile(2 * i + 1), kInstrS);
                commit(dp_full);
                return true;
            };
            bool ok = true;
            for (int items = 0, s0 = 0; ok && tiles.next<true>(it);) {
                const int n = Queries(P, it, rank, split).n;
                if (SPLIT && !n) continue;
                // (S and dP of the first step go over the last item's P and dS: products run in the order of their issue)
                ok = mbar_wait_one(kv_full, items & 1, abort) && scores(s0) && grads(s0) && (kLead == 1 || n < 2 || scores(s0 + 1));
                if (ok && n == 1) commit(kv_empty);
                for (int i = s0; i < s0 + n && ok; ++i) {
                    if (!(ok = mbar_wait_one(p_ready + 8 * (i & 1), (i >> 1) & 1, abort))) break;
                    if (i == s0 && items && !(ok = mbar_wait_one(sums_free, (items - 1) & 1, abort))) break;   // read
                    fence_after();
                    product_ab<kParts>(t_dv, t_s(i), tile(2 * i + 1), kInstrD, i > s0);
                    commit(empty + 8 * ((2 * i + 1) % kRing));
                    if (i + kLead < s0 + n && !(ok = scores(i + kLead))) break;   // over P
                    if (!(ok = mbar_wait_one(ds_ready, i & 1, abort))) break;
                    fence_after();
                    product_ab<kParts>(t_dk, t_dp, tile(2 * i), kInstrD, i > s0);
                    commit(empty + 8 * (2 * i % kRing));
                    if (i + 1 < s0 + n) {
                        ok = grads(i + 1);
                        if (ok && i + 2 == s0 + n) commit(kv_empty);   // the last product that reads k or v
                    }
                }
                if (ok) commit(done);
                ++items;
                s0 += n;
            }
        }
        __syncwarp();
    } else if (warp == kRowWarp) {
        // ------------------------------------------------------------ the queries' lse and delta
        if constexpr (BOXES == 1) give_registers<kOtherRegsKV>();
        bool ok = true;
        for (int step = 0, items = 0; ok && tiles.next(it); ++items) {
            const Queries Q(P, it, rank, split);
            float range = 1.0f;
            if constexpr (!kBf16) {
                // (four places: this warp is at most two steps ahead of the factor's readers)
                const float v_max = largest_norm(P.tile_norms, (int64_t)(P.n_heads + it.y) * P.n_tokens + it.lo, Q.tiles, 1, 0);
                range = range_factor(2.0f * v_max *
                                     largest_norm(P.tile_norms, (int64_t)it.y * group * P.n_tokens + it.lo + Q.tile0 * kTile,
                                                  Q.per_head, group, P.n_tokens));
                if (lane == 0) bars->range[items & 3] = range;
            }
            int head = it.y * group + Q.first / Q.per_head, tile = Q.first % Q.per_head;
            for (int i = 0; i < Q.n; ++i, ++step) {
                const int first = (Q.tile0 + tile) * kTile;
                const int64_t at = (int64_t)head * P.n_tokens + it.lo + first;
                if (++tile == Q.per_head) tile = 0, ++head;
                float l[kTile / 32], d[kTile / 32];
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k) {
                    const int r = lane + 32 * k;
                    const bool in = first + r < it.len;   // no weight behind the end
                    l[k] = in ? -scaled_lse<T>(P.lse[at + r]) : -INFINITY;
                    d[k] = in ? -P.delta[at + r] * range : 0.0f;
                }
                // the buffer's last readers were done before dk of step - 2, which freed that step's q
                const int e = 2 * step - 4;
                if (step >= 2 && !(ok = mbar_wait(empty + 8 * (e % kRing), (e / kRing) & 1, abort))) break;
                float *rows = reinterpret_cast<float *>(bars->rows[step & 1]);
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k) {
                    rows[lane + 32 * k] = l[k];
                    rows[kTile + lane + 32 * k] = d[k];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(rows_full + 8 * (step & 1));
            }
        }
    } else if (warp < kComputeWarp) {
        // ------------------------------------------------------------ rows of ragged tiles behind the end
        if constexpr (BOXES == 1) give_registers<kOtherRegsKV>();
        // cleared, so that P = 0 and dS = 0 meet finite values there; every tile passes here, so that no barrier can
        // run a phase ahead of its waiters
        bool ok = true;
        for (int cleared = 0; ok && tiles.next(it);) {
            const Queries Q(P, it, rank, split);
            for (int e = 0; e < 2 * Q.n; ++e, ++cleared) {
                const int st = cleared % kRing;
                if (!(ok = mbar_wait(full + 8 * st, (cleared / kRing) & 1, abort))) break;
                if (Q.ragged && (Q.first + (e >> 1)) % Q.per_head == Q.per_head - 1)
                    zero_rows<BOXES>(s_ring + st * kTileBytes, it.len - (Q.tiles - 1) * kTile, lane);
                if (lane == 0) mbar_arrive(clear + 8 * st);
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------------------ P^T and dS^T
        if constexpr (BOXES == 1) take_registers<kComputeRegsKV>();
        const int part = (warp - kComputeWarp) >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21, t_g = t_dp + kCols * part + lanes;
        const float2 c2 = make_float2(P.scale_log2, P.scale_log2);
        bool ok = true;
        for (int items = 0, i = 0; ok && tiles.next(it); ++items) {
            const Queries Q(P, it, rank, split);
            const int row = it.row + r, n = Q.n;
            int at = Q.first % Q.per_head;
            for (int j = Q.first; j < Q.first + n; ++j, ++i) {
                if (!(ok = mbar_wait(rows_full + 8 * (i & 1), (i >> 1) & 1, abort) &&
                          mbar_wait(s_full + 8 * (i % kLead), (i / kLead) & 1, abort)))
                    break;
                fence_after();
                const float4 *lse = bars->rows[i & 1][0] + kCols / 4 * part, *delta = bars->rows[i & 1][1] + kCols / 4 * part;
                const uint32_t t_p = t_s(i) + kCols * part + lanes;
                uint32_t s[kCols];
                float2 p[kCols / 2];
                load_part<kCols>(t_p, s);
#pragma unroll
                for (int k = 0; k < kCols / 2; k += 2) {
                    const float4 l = lse[k / 2];
                    p[k] = f2_fma(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), c2, make_float2(l.x, l.y));
                    p[k + 1] = f2_fma(make_float2(__uint_as_float(s[2 * k + 2]), __uint_as_float(s[2 * k + 3])), c2,
                                      make_float2(l.z, l.w));
                    p[k].x = exp2_fast(p[k].x);
                    p[k].y = exp2_fast(p[k].y);
                    p[k + 1].x = exp2_fast(p[k + 1].x);
                    p[k + 1].y = exp2_fast(p[k + 1].y);
                }
                const int first = (Q.tile0 + at) * kTile + kCols * part;
                if (++at == Q.per_head) at = 0;
                if (P.causal && first < it.row + kTile) {   // queries before the key
                    const int hidden = row - first;
#pragma unroll
                    for (int k = 0; k < kCols; ++k)
                        if (k < hidden) (k & 1 ? p[k / 2].y : p[k / 2].x) = 0.0f;
                }
                store_part<T, kCols>(t_p, p);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + 8 * (i & 1));
                if (!(ok = mbar_wait(dp_full, i & 1, abort))) break;
                fence_after();
                load_part<kCols>(t_g, s);
                const float range = kBf16 ? 1.0f : bars->range[items & 3];
                auto minus_delta = [&](int k, float a, float b) {   // (dP - delta) F
                    const float2 x = make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
                    return kBf16 ? add2(x, make_float2(a, b)) : f2_fma(x, make_float2(range, range), make_float2(a, b));
                };
#pragma unroll
                for (int k = 0; k < kCols / 2; k += 2) {
                    const float4 d = delta[k / 2];
                    p[k] = f2_mul(p[k], minus_delta(k, d.x, d.y));
                    p[k + 1] = f2_mul(p[k + 1], minus_delta(k + 1, d.z, d.w));
                }
                store_part<T, kCols>(t_g, p);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_ready);
            }
            if (!ok || !(ok = (SPLIT && !n) || mbar_wait(done, items & 1, abort))) break;
            fence_after();
            // half the parts store dv, half dk, each its share of the columns
            constexpr int kShare = 2 * kDim / kParts;
            const bool is_k = part >= kParts / 2;
            const Heads<T> out = heads<T>(is_k ? P.dk : P.dv);
            T *dst = out.at(it.lo, it.y);
            const float unrange = kBf16 || SPLIT ? 1.0f : range_inverse(bars->range[items & 3]);   // (a cluster: at the end)
            const float f = is_k ? P.scale * p_unshift<T>() * unrange : p_unshift<T>();
            const int k0 = part % (kParts / 2) * kShare;
            float *sums = reinterpret_cast<float *>(smem);   // the tiles' place: all products are done
#pragma unroll 1
            for (int k = k0; k < k0 + kShare; k += 32) {
                uint32_t o[32];
                tmem_load32((is_k ? t_dk : t_dv) + lanes + k, o);
                wait_ld();
                if (k + 32 == k0 + kShare) {   // the sums may be written again
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sums_free);
                }
                if (SPLIT)
                    leave_columns(sums + (is_k * kTile + (int)(threadIdx.x & 127)) * pitch<kDim>() + k, o, n == 0);
                else
                    store_columns(o, f, dst, out.ts, it.row + 32 * (warp & 3), it.len, k, P.dim);
            }
        }
    }

    fence_before();
    __syncthreads();
    if (*abort) {
        if (warp == kCopyWarp) {
            mbar_land(kv_full, (items - 1) & 1);
            for (int e = max(0, loaded - kRing); e < loaded; ++e) mbar_land(full + 8 * (e % kRing), (e / kRing) & 1);
            if (lane == 0) *P.status = DQ_DEVICE_WAIT_TIMEOUT;
        } else if (warp == kProductWarp) {
            drain_products(smem_addr(&bars->drained));
        }
        __syncthreads();
    }
    if (warp == kProductWarp) {
        fence_after();
        tmem_free<512>(tmem);
    }
    if (SPLIT) {
        if constexpr (BOXES == 1) {   // what follows is built for the registers of the launch, and all warps run it
            __syncthreads();
            if (warp < kComputeWarp)
                take_registers<kLaunchRegsKV>();
            else
                give_registers<kLaunchRegsKV>();
        }
        cluster_sync();
        it = bars->queue.item[0];   // the one item, if the cluster had any
        const Heads<T> dv = heads<T>(P.dv), dk = heads<T>(P.dk);
        constexpr uint32_t kSum = kTile * pitch<kDim>() * 4;
        static_assert(2 * kSum <= (2 + kRing) * kTileBytes, "accumulators fit the tiles' place");
        if (it.len >= 0 && !*abort) {
            add_up_rows<T, kDim>(smem_addr(smem), rank, split, p_unshift<T>(), dv.at(it.lo, it.y), dv.ts, it.row, it.len, P.dim);
            const float unrange = kBf16 ? 1.0f : range_inverse(bars->range[0]);   // the same in every block
            add_up_rows<T, kDim>(smem_addr(smem) + kSum, rank, split, P.scale * p_unshift<T>() * unrange, dk.at(it.lo, it.y), dk.ts, it.row,
                                 it.len, P.dim);
        }
        cluster_sync();
    }
}

template <typename T, int STEPS, bool SPLIT> cudaError_t launch_dq(const AttentionParams &P, int64_t blocks, cudaStream_t st)
{
    static std::atomic<uint64_t> set[2];
    constexpr int kSmem = smem_bytes_q<boxes(STEPS)>();
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(attention_dq_kernel<T, STEPS, SPLIT>), kSmem, set);
    return e == cudaSuccess ? launch_split(attention_dq_kernel<T, STEPS, SPLIT>, P, blocks, kThreadsQ, kSmem, st) : e;
}

template <typename T, int STEPS, bool SPLIT> cudaError_t launch_dkv(const AttentionParams &P, int64_t blocks, cudaStream_t st)
{
    static std::atomic<uint64_t> set[2];
    constexpr int kSmem = smem_bytes_kv<boxes(STEPS)>();
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(attention_dkv_kernel<T, STEPS, SPLIT>), kSmem, set);
    return e == cudaSuccess ? launch_split(attention_dkv_kernel<T, STEPS, SPLIT>, P, blocks, threads_kv<boxes(STEPS)>(), kSmem, st) : e;
}

template <typename T, int STEPS> cudaError_t launch(const AttentionParams &P, int64_t slots, cudaStream_t st)
{
    if constexpr (__is_same(T, __half)) {
        attention_norms_kernel<T, boxes(STEPS)>
            <<<dim3((unsigned)slots, (unsigned)std::min(P.n_heads + P.n_kv, 65535)), 128, 0, st>>>(P);
        note_launches(1);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const int sms = sm_count();
    const Choice q = choose_dq(P.n_tokens, P.n_seqs, P.n_heads, sms), kv = choose_dkv(P.n_tokens, P.n_seqs, P.n_heads, P.n_kv, sms);
    const cudaError_t e = q.split > 1 ? launch_dq<T, STEPS, true>(chosen(P, q), q.blocks, st)
                                      : launch_dq<T, STEPS, false>(chosen(P, q), q.blocks, st);
    if (e != cudaSuccess) return e;
    return kv.split > 1 ? launch_dkv<T, STEPS, true>(chosen(P, kv), kv.blocks, st)
                        : launch_dkv<T, STEPS, false>(chosen(P, kv), kv.blocks, st);
}

}  // namespace

cudaError_t launch_attention_backward(const AttentionParams &P, bool bf16, cudaStream_t st)
{
    const int64_t slots = slot_count(P.n_tokens, P.n_seqs, kTile);
    if (bf16)
        return P.dim <= 64   ? launch<__nv_bfloat16, 4>(P, slots, st)
               : P.dim <= 96 ? launch<__nv_bfloat16, 6>(P, slots, st)
                             : launch<__nv_bfloat16, 8>(P, slots, st);
    return P.dim <= 64   ? launch<__half, 4>(P, slots, st)
           : P.dim <= 96 ? launch<__half, 6>(P, slots, st)
                         : launch<__half, 8>(P, slots, st);
}

}  // namespace dq
