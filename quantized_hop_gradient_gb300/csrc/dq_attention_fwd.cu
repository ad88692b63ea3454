// dq_attention_fwd.cu -- the attention forward kernel.
//
// A block takes two row tiles of 128 queries that read the same keys: two
// heads of a group, or two tiles of one head.  Per key tile and row tile:
// S = q k^T into tensor memory, softmax warps turn S into P (16 bits, over
// S's own columns), O += P v with P read from tensor memory.  While the
// softmax of one row tile runs, the products of the other do.
// (Heads of up to 64 elements: P beside S, see kApart.)
// With few tiles the blocks of a cluster share a tile's keys, and join their
// O, references and sums through shared memory at the end.
//
// What bounds it (bf16, causal): heads of 128, 15,193 tokens of 32 heads over
// 8: 600 us in a loop, 1.59 PFLOP/s, 0.83 of the library's plain product and
// 0.92 of what that sustains, the card being at its power limit; 541 us alone;
// tensor pipe 78% active, issue slots 43%, DRAM 280 MB.  Heads of 64, 5,096
// tokens of 32 over 8: 46 us, tensor pipe 31% active, issue slots 49%, exp's
// unit 35%: no unit is full, the chain S, maximum, exp, P, O of each row tile
// is, of which two run at a time (tensor memory would hold a third's
// accumulators, but the registers no third set of threads with 128 scores each:
// with two, and P waiting in registers, 28 bytes a thread are spilled, heads of
// more than 64 none; 72 where a cluster shares a tile, 24 with wide heads).
//
// Softmax with one pass over the keys (Milakov and Gimelshein, 2018, arXiv
// 1805.02867), two row tiles in turns (Shah et al., 2024, arXiv 2407.08608):
// p = exp2(c s - c m) with a reference m that only moves when the row's maximum
// has grown by more than 2^8 = 256 times; then O and the sum are rescaled.  Any
// m gives the same quotient, so this costs no accuracy: p stays below 2^8, its
// sum in fp32.  p is rounded to 16 bits because the tensor core multiplies it
// with 16-bit v: bf16 with the same relative rounding at every magnitude; fp16
// (up to 256 of 65,504) with steps of 2^-24 below 2^-14, by which n small
// weights lose at most n 2^-25 of a sum of at least 1, half of fp16's own
// rounding for 8,192 keys.  That rounding is what the output's error over the
// plain 32-bit form's comes from (0.0020 against 0.0016 of its norm in bf16).
#include "dq_attention.cuh"

namespace dq {
namespace {

using namespace tc;

// Three warpgroups of 168 registers a thread at launch: 2 x 208 for the
// softmax, which holds a row of 128 scores, 88 for the rest (504 = 3 x 168).
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs == 3 * kLaunchRegs, "register shares");
// Warps 0 and 1: products of row tile 0 and 1, each by one thread, so that the
// waits of one pass behind the other's products; 2: copies, 3: clearing; 4-7
// and 8-11: softmax of row tile 0 and 1, a thread a row.  The product threads
// must not wait for issue slots: the older warps go first.
constexpr int kProductWarps = 2, kCopyWarp = 2, kClearWarp = 3, kSoftmaxWarp = 4;
// Key and value tiles in flight: what shared memory holds beside two query tiles.
template <int BOXES> __host__ __device__ constexpr int stages_k() { return BOXES == 1 ? 4 : 3; }
template <int BOXES> __host__ __device__ constexpr int stages_v() { return BOXES == 1 ? 4 : 2; }
constexpr float kGrowth = 8.0f;   // log2 of the growth of a row's maximum that moves its reference

template <int BOXES> struct Bars {
    ItemQueue queue;
    unsigned long long q_full[2], q_empty[2], k_full[stages_k<BOXES>()], k_empty[stages_k<BOXES>()];
    unsigned long long v_full[stages_v<BOXES>()], v_clear[stages_v<BOXES>()], v_empty[stages_v<BOXES>()];
    unsigned long long s_full[2], s_free[2], p_ready[2], o_done[2], o_free[2], all_done;
    unsigned long long drained[2];   // a block that gives up: the products of row tile 0 and 1
    uint32_t tmem;
    int abort;
    int lead;   // items of which row tile 0 has its first weights
};

template <int BOXES> constexpr int smem_bytes()
{
    return (2 + stages_k<BOXES>() + stages_v<BOXES>()) * BOXES * kBoxBytes + (int)sizeof(Bars<BOXES>);
}
static_assert(smem_bytes<2>() <= 227 * 1024, "shared memory");

// The maximum of a row's 128 scores, in eight chains.
__device__ __forceinline__ float max128(const uint32_t *s)
{
    float a[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = __uint_as_float(s[k]);
#pragma unroll
    for (int i = 8; i < 120; i += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = max3(a[k], __uint_as_float(s[i + k]), __uint_as_float(s[i + 8 + k]));
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = fmaxf(a[k], __uint_as_float(s[120 + k]));
    return max3(max3(a[0], a[1], a[2]), max3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
}

// A row whose every score is -inf has no weights and an output of 0, with an
// lse of -inf.
__device__ __forceinline__ float inverse_sum(float total) { return total == 0.0f ? 0.0f : 1.0f / total; }

// The two row tiles of an item; with a cluster, the block's part of their keys.
struct Rows {
    int head[2], row[2], n[2], hk, first, n_max;   // n: key tiles, from `first` on
    __device__ __forceinline__ Rows(const AttentionParams &P, const Item &it, int rank, int split)
    {
        head[0] = P.pair_heads ? 2 * it.y : it.y;
        head[1] = P.pair_heads ? head[0] + 1 : head[0];
        row[0] = it.row;
        row[1] = P.pair_heads ? it.row : it.row + kTile;
        hk = head[0] / (P.n_heads / P.n_kv);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int end = P.causal ? min(row[u] + kTile, it.len) : it.len;
            n[u] = row[u] < it.len ? (end + kTile - 1) / kTile : 0;
        }
        const Part part(max(n[0], n[1]), rank, split);
        first = split > 1 ? part.first : 0;
        n_max = part.n;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (split > 1) n[u] = min(max(n[u] - first, 0), n_max);
    }
};

template <typename T, int STEPS, bool SPLIT> __global__ void __launch_bounds__(kThreads, 1)
    attention_forward_kernel(const __grid_constant__ AttentionParams P)
{
    constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
    constexpr int BOXES = boxes(STEPS);
    constexpr int kDim = 64 * BOXES;
    // Heads of up to 64 elements leave tensor memory for P beside S: then the scores of the next key tile are computed
    // as soon as the softmax holds this tile's in registers, not behind O += P v.
    constexpr bool kApart = BOXES == 1;
    constexpr uint32_t kTileBytes = BOXES * kBoxBytes;
    constexpr int kK = stages_k<BOXES>(), kV = stages_v<BOXES>();
    // a cluster's block leaves O of both row tiles, then the rows' references and sums, in the tiles' place
    constexpr uint32_t kMaxima = 2 * kTile * pitch<kDim>() * 4;
    static_assert(kMaxima + 4 * kTile * 4 <= (2 + kK + kV) * kTileBytes, "they fit");
    extern __shared__ __align__(1024) uint8_t smem[];
    auto *bars = reinterpret_cast<Bars<BOXES> *>(smem + (2 + kK + kV) * kTileBytes);
    const uint32_t s_q = smem_addr(smem), s_k = s_q + 2 * kTileBytes, s_v = s_k + kK * kTileBytes;
    const uint32_t q_full = smem_addr(bars->q_full), q_empty = smem_addr(bars->q_empty);
    const uint32_t k_full = smem_addr(bars->k_full), k_empty = smem_addr(bars->k_empty);
    const uint32_t v_full = smem_addr(bars->v_full), v_clear = smem_addr(bars->v_clear), v_empty = smem_addr(bars->v_empty);
    const uint32_t s_full = smem_addr(bars->s_full);
    const uint32_t s_free = smem_addr(bars->s_free), p_ready = smem_addr(bars->p_ready);
    const uint32_t o_done = smem_addr(bars->o_done), o_free = smem_addr(bars->o_free);
    const uint32_t all_done = smem_addr(&bars->all_done);   // a cluster's block: the products of both row tiles
    volatile int *abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == kCopyWarp) {
        if (lane == 0) {
            prefetch_map(&P.map_q);
            prefetch_map(&P.map_k);
            prefetch_map(&P.map_v);
            init_queue(&bars->queue, 11);   // 2 of products, clearing, 8 of the softmax
            for (int u = 0; u < 2; ++u) {
                mbar_init(q_full + 8 * u, 1);
                mbar_init(q_empty + 8 * u, 1);
                mbar_init(s_full + 8 * u, 1);
                mbar_init(s_free + 8 * u, 4);
                mbar_init(p_ready + 8 * u, 4);
                mbar_init(o_done + 8 * u, 1);
                mbar_init(o_free + 8 * u, 4);
            }
            for (int i = 0; i < kK; ++i) {
                mbar_init(k_full + 8 * i, 1);
                mbar_init(k_empty + 8 * i, 2);
            }
            for (int i = 0; i < kV; ++i) {
                mbar_init(v_full + 8 * i, 1);
                mbar_init(v_clear + 8 * i, 1);
                mbar_init(v_empty + 8 * i, 2);
            }
            mbar_init(all_done, kProductWarps);
            for (int u = 0; u < kProductWarps; ++u) mbar_init(smem_addr(&bars->drained[u]), 1);
            bars->abort = P.give_up;
            bars->lead = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == 0) {
        tmem_alloc<512>(smem_addr(&bars->tmem));
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars->tmem;
    Tiles tiles{&bars->queue, abort};
    Item it;
    const int split = SPLIT ? P.split : 1, rank = SPLIT ? cluster_rank() : 0;
    Ring<kK> rk;          // key tiles: copied (copy warp) or consumed (product warps)
    Ring<kV> rv;
    int loaded_q[2] = {0, 0};   // query tiles copied (copy warp)

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------ tiles, and copies: q, then k0, v0, k1, v1, ...
        give_registers<kOtherRegs>();
        const int rows = P.pair_heads ? kTile : 2 * kTile, slots = gridDim.x / (P.y * split);
        auto padding = [&](const Slot &S, int y) {
            if (SPLIT && rank) return;
            const Rows R(P, Item{S.lo, S.len, S.row, y}, 0, 1);
            for (int u = 0; u < 2; ++u) {
                const int n = min(kTile, S.len - R.row[u]);
                zero_heads<T>(P.out, S.lo + R.row[u], n, R.head[u], P.dim);
                for (int i = lane; i < n; i += 32)
                    P.lse[(int64_t)R.head[u] * P.n_tokens + S.lo + R.row[u] + i] = -INFINITY;
            }
        };
        Taker taker{&bars->queue, abort, blockIdx.x / split};
        taker.claims = !SPLIT;   // a cluster does its one tile
        bool ok = true;
        while (ok && taker.next<true, true>(P, slots, rows, it, padding) == Taker::kTaken) {
            const Rows R(P, it, rank, split);
            for (int u = 0; u < 2; ++u) {
                if (!R.n[u]) continue;
                if (loaded_q[u] && !(ok = mbar_wait(q_empty + 8 * u, (loaded_q[u] - 1) & 1, abort))) break;
                if (lane == 0) {
                    mbar_expect(q_full + 8 * u, kTileBytes);
                    for (int b = 0; b < BOXES; ++b)
                        load_box(s_q + u * kTileBytes + b * kBoxBytes, &P.map_q, 64 * b, R.head[u], it.lo + R.row[u],
                                 q_full + 8 * u);
                }
                ++loaded_q[u];
            }
            for (int j = 0; ok && j < R.n_max; ++j) {
                if (rk.laps && !(ok = mbar_wait(k_empty + 8 * rk.stage, rk.phase ^ 1, abort))) break;
                if (lane == 0) {
                    mbar_expect(k_full + 8 * rk.stage, kTileBytes);
                    for (int b = 0; b < BOXES; ++b)
                        load_box(s_k + rk.stage * kTileBytes + b * kBoxBytes, &P.map_k, 64 * b, R.hk, it.lo + (R.first + j) * kTile,
                                 k_full + 8 * rk.stage);
                }
                __syncwarp();
                rk.step();
                if (rv.laps && !(ok = mbar_wait(v_empty + 8 * rv.stage, rv.phase ^ 1, abort))) break;
                if (lane == 0) {
                    mbar_expect(v_full + 8 * rv.stage, kTileBytes);
                    for (int b = 0; b < BOXES; ++b)
                        load_box(s_v + rv.stage * kTileBytes + b * kBoxBytes, &P.map_v, 64 * b, R.hk, it.lo + (R.first + j) * kTile,
                                 v_full + 8 * rv.stage);
                }
                __syncwarp();
                rv.step();
            }
        }
    } else if (warp < kProductWarps) {
        // ------------------------------------------------------------ products of row tile u: one thread
        give_registers<kOtherRegs>();
        constexpr uint32_t kInstrS = instr(kBf16, kTile, false), kInstrO = instr(kBf16, 16 * STEPS, true);
        if (elect_one()) {
            const int u = warp;
            const uint32_t t_s = tmem + u * kTile, t_o = tmem + 2 * kTile + u * kDim;
            const uint32_t t_p = kApart ? tmem + 2 * kTile + 2 * kDim + u * 64 : t_s, tile_q = operand<SPLIT>(s_q) + u * kTileBytes;
            const uint32_t o_k = operand<SPLIT>(s_k), o_v = operand<SPLIT>(s_v);
            uint32_t items = 0, scored = 0, summed = 0;   // items begun; tiles whose S, whose O += P v was issued
            bool ok = true;
            while (ok && tiles.next<true>(it)) {
                const Rows R(P, it, rank, split);
                const int n = u ? R.n[1] : R.n[0], n_max = R.n_max;
                // S of key tile j, which is then given back
                auto scores = [&](int j) {
                    if (!mbar_wait_one(k_full + 8 * rk.stage, rk.phase, abort)) return false;
                    if (j < n) {
                        if (kApart && scored && !mbar_wait_one(s_free + 8 * u, (scored - 1) & 1, abort)) return false;
                        fence_after();
                        product_abt<STEPS>(t_s, tile_q, o_k + rk.stage * kTileBytes, kInstrS);
                        commit(s_full + 8 * u);
                        commit(k_empty + 8 * rk.stage);
                        if (j + 1 == n) commit(q_empty + 8 * u);
                        ++scored;
                    } else {
                        mbar_arrive(k_empty + 8 * rk.stage);
                    }
                    rk.step();
                    return true;
                };
                if (SPLIT && !n_max) {
                    commit(all_done);
                    continue;
                }
                if (kApart && !SPLIT && u) {
                    // Row tile 1 stays half a step behind, so that one's exp meets the other's maxima and waits, not its
                    // exp (46 us against 48 for 5,096 tokens of 32 heads of 64; two boxes: 114 against 107 us for 8,192,
                    // whose products fill the step).  Nothing depends on it: the wait is bounded and goes on.
                    const long long start = clock64();
                    while (*(volatile int *)&bars->lead <= (int)items && clock64() - start < 4096) {
                    }
                }
                if (n && !(ok = mbar_wait_one(q_full + 8 * u, items & 1, abort))) break;
                if (!(ok = scores(0))) break;
                for (int j = 0; j < n_max; ++j) {
                    if (kApart && j + 1 < n_max && !(ok = scores(j + 1))) break;
                    if (!(ok = mbar_wait_one(v_clear + 8 * rv.stage, rv.phase, abort))) break;
                    if (j < n) {
                        // the last item's O has been read
                        if (j == 0 && items && !(ok = mbar_wait_one(o_free + 8 * u, (items - 1) & 1, abort))) break;
                        if (!(ok = mbar_wait_one(p_ready + 8 * u, summed & 1, abort))) break;
                        fence_after();
                        product_ab<1>(t_o, t_p, o_v + rv.stage * kTileBytes, kInstrO, j > 0);
                        commit(v_empty + 8 * rv.stage);
                        ++summed;
                        if (kApart || j + 1 == n) commit(o_done + 8 * u);   // apart: after each tile
                    } else {
                        mbar_arrive(v_empty + 8 * rv.stage);
                    }
                    rv.step();
                    // S of the next tile goes over this P: products run in the order of their issue
                    if (!kApart && j + 1 < n_max && !(ok = scores(j + 1))) break;
                }
                if (n) ++items;
                if (SPLIT && ok) commit(all_done);
            }
        }
        __syncwarp();
    } else if (warp == kClearWarp) {
        // ------------------------------------------------------------ v rows behind the sequence's end
        give_registers<kOtherRegs>();
        // their p is 0, which a NaN or an infinity would survive; every tile passes here, so that no barrier can run a
        // phase ahead of its waiters
        bool ok = true;
        while (ok && tiles.next(it)) {
            const Rows R(P, it, rank, split);
            for (int j = 0; j < R.n_max; ++j) {
                const int behind = it.len - (R.first + j) * kTile;
                if (!(ok = mbar_wait(v_full + 8 * rv.stage, rv.phase, abort))) break;
                if (behind < kTile) zero_rows<BOXES>(s_v + rv.stage * kTileBytes, behind, lane);
                if (lane == 0) mbar_arrive(v_clear + 8 * rv.stage);
                __syncwarp();
                rv.step();
            }
        }
    } else {
        // ------------------------------------------------------------ softmax: a thread a row
        take_registers<kSoftmaxRegs>();
        const int u = (warp - kSoftmaxWarp) >> 2;
        const uint32_t t_s = tmem + u * kTile + ((uint32_t)(warp & 3) << 21);   // lane 32 (warp mod 4), bits 16 up
        const uint32_t t_o = t_s - u * kTile + 2 * kTile + u * kDim;
        const uint32_t t_p = kApart ? t_s - u * kTile + 2 * kTile + 2 * kDim + u * 64 : t_s;
        const float c = P.scale_log2;
        int done = 0, items = 0;   // tiles and items of this row tile
        bool ok = true;
        while (ok && tiles.next(it)) {
            const bool second = u == 1;
            const int row0 = second && !P.pair_heads ? it.row + kTile : it.row, row = row0 + (int)(threadIdx.x & 127);
            const int head = P.pair_heads ? 2 * it.y + u : it.y;
            int n, j0 = 0;
            if (SPLIT) {
                const Rows R(P, it, rank, split);
                n = u ? R.n[1] : R.n[0];
                j0 = R.first;
            } else {
                const int end = P.causal ? min(row0 + kTile, it.len) : it.len;
                n = row0 < it.len ? (end + kTile - 1) / kTile : 0;
                if (!n) continue;
            }
            float m = -INFINITY;
            float2 sum = make_float2(0.0f, 0.0f);
            for (int j = 0; j < n; ++j, ++done) {
                if (!(ok = mbar_wait(s_full + 8 * u, done & 1, abort))) break;
                fence_after();
                uint32_t s[128];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_load32(t_s + 32 * i, s + 32 * i);
                wait_ld();
                if (kApart) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_free + 8 * u);
                }
                // keys that the row does not see: behind its own place, or behind the sequence's end
                const int first = (j0 + j) * kTile;
                if (first + kTile > it.len || (P.causal && first + kTile > row0)) {
                    const int seen = (P.causal ? min(row + 1, it.len) : it.len) - first;
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i >= seen) s[i] = __float_as_uint(-INFINITY);
                }
                const float top = fmaxf(m, max128(s));
                if (j == 0) m = top;
                const bool grown = (top - m) * c > kGrowth;
                if (__any_sync(kFull, grown)) {
                    // O must be at rest; where P lies over S, this tile's S was issued behind the last O += P v
                    if (kApart && !(ok = mbar_wait(o_done + 8 * u, (done - 1) & 1, abort))) break;
                    fence_after();
                    const float f = grown ? exp2_fast((m - top) * c) : 1.0f;
                    if (grown) m = top;
                    sum.x *= f;
                    sum.y *= f;
#pragma unroll 1
                    for (int i = 0; i < kDim; i += 16) {
                        uint32_t o[16];
                        tmem_load16(t_o + i, o);
                        wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_store16(t_o + i, o);
                    }
                }
                // (a row whose scores so far are all -inf has weights of 0, not of -inf + inf)
                const float at = m == -INFINITY ? 0.0f : -m * c;
                const float2 c2 = make_float2(c, c), b2 = make_float2(at, at);
                uint32_t p[64];
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    float2 x = f2_fma(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, b2);
                    x.x = exp2_fast(x.x);
                    x.y = exp2_fast(x.y);
                    sum = add2(sum, x);
                    p[i] = pack2(x.x, x.y, T());
                    if (!kApart && i % 16 == 15) tmem_store16(t_p + i - 15, p + i - 15);
                }
                if (kApart) {   // P waits in registers for the last O += P v to be done with its place
                    if (j > 0 && !(ok = mbar_wait(o_done + 8 * u, (done - 1) & 1, abort))) break;
                    fence_after();
                    tmem_store32(t_p, p);
                    tmem_store32(t_p + 32, p + 32);
                }
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + 8 * u);
                if (kApart && !SPLIT && j == 0 && warp == kSoftmaxWarp) *(volatile int *)&bars->lead = items + 1;
            }
            if (!ok) break;
            if (SPLIT) {
                // O as it is, with the row's reference and sum, in the tiles' place once all products are done
                if (!(ok = mbar_wait(all_done, 0, abort))) break;
                fence_after();
                float *sums = reinterpret_cast<float *>(smem) + (u * kTile + (int)(threadIdx.x & 127)) * pitch<kDim>();
#pragma unroll 1
                for (int i = 0; i < kDim; i += 32) {
                    uint32_t o[32];
                    tmem_load32(t_o + i, o);
                    wait_ld();
                    leave_columns(sums + i, o, n == 0);
                }
                float *ml = reinterpret_cast<float *>(smem + kMaxima) + u * kTile + (threadIdx.x & 127);
                ml[0] = m;
                ml[2 * kTile] = sum.x + sum.y;
                continue;
            }
            if (!(ok = mbar_wait(o_done + 8 * u, (kApart ? done - 1 : items) & 1, abort))) break;
            ++items;
            fence_after();
            const float total = sum.x + sum.y, inv = inverse_sum(total);
            const Heads<T> out = heads<T>(P.out);
            T *dst = out.at(it.lo, head);
            const int warp_row = row0 + 32 * (warp & 3);
#pragma unroll 1
            for (int i = 0; i < kDim; i += 32) {
                uint32_t o[32];
                tmem_load32(t_o + i, o);
                wait_ld();
                if (i + 32 == kDim) {   // O may be written again
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_free + 8 * u);
                }
                store_columns(o, inv, dst, out.ts, warp_row, it.len, i, P.dim);
            }
            if (row < it.len) P.lse[(int64_t)head * P.n_tokens + it.lo + row] = fmaf(m, P.scale, logf(total));
        }
        if (!ok) wait_st();   // given up between a store to tensor memory and its wait
    }

    fence_before();
    __syncthreads();
    if (*abort) {
        // a wait ran out: let this block's own copies and products land before its memory goes
        if (warp == kCopyWarp) {
            for (int u = 0; u < 2; ++u) mbar_land(q_full + 8 * u, (loaded_q[u] - 1) & 1);
            for (int i = 0; i < kK; ++i, rk.step()) mbar_land(k_full + 8 * rk.stage, rk.phase ^ 1);
            for (int i = 0; i < kV; ++i, rv.step()) mbar_land(v_full + 8 * rv.stage, rv.phase ^ 1);
            if (lane == 0) *P.status = DQ_DEVICE_WAIT_TIMEOUT;
        } else if (warp < kProductWarps) {
            const uint32_t bar = smem_addr(&bars->drained[warp]);
            if (elect_one()) commit(bar);
            __syncwarp();
            mbar_land(bar, 0);
        }
        __syncthreads();
    }
    if (warp == 0) {
        fence_after();
        tmem_free<512>(tmem);
    }
    if (SPLIT) {
        // what follows is built for the registers of the launch, and all warps run it
        __syncthreads();
        if (warp < kSoftmaxWarp)
            take_registers<kLaunchRegs>();
        else
            give_registers<kLaunchRegs>();
        cluster_sync();
        it = bars->queue.item[0];   // the one item, if the cluster had any
        if (it.len >= 0 && !*abort) {
            const Rows R(P, it, 0, 1);
            const Heads<T> out = heads<T>(P.out);
            const int share = kTile / split, pieces = kDim / 8;
            for (int i = threadIdx.x; i < 2 * share * pieces; i += kThreads) {
                const int u = i / (share * pieces), r = rank * share + i / pieces % share, c = i % pieces * 8;
                const int row = (u ? R.row[1] : R.row[0]) + r, head = u ? R.head[1] : R.head[0];
                if (row >= it.len || c >= P.dim) continue;
                // parts joined at the largest reference, in the order of the ranks
                const uint32_t ml = smem_addr(smem) + kMaxima + (u * kTile + r) * 4;
                float m = -INFINITY;
                for (int s = 0; s < split; ++s) m = fmaxf(m, load_peer1(ml, s));
                float total = 0.0f;
                F8 o{};
                for (int s = 0; s < split; ++s) {
                    const float part = load_peer1(ml + 2 * kTile * 4, s);
                    if (part == 0.0f) continue;   // no keys of this row
                    const float f = exp2_fast((load_peer1(ml, s) - m) * P.scale_log2);
                    const uint32_t at = smem_addr(smem) + ((u * kTile + r) * pitch<kDim>() + c) * 4;
                    const float4 a = load_peer(at, s), b = load_peer(at + 16, s);
                    total = fmaf(f, part, total);
                    o.v[0] = fmaf(f, a.x, o.v[0]); o.v[1] = fmaf(f, a.y, o.v[1]);
                    o.v[2] = fmaf(f, a.z, o.v[2]); o.v[3] = fmaf(f, a.w, o.v[3]);
                    o.v[4] = fmaf(f, b.x, o.v[4]); o.v[5] = fmaf(f, b.y, o.v[5]);
                    o.v[6] = fmaf(f, b.z, o.v[6]); o.v[7] = fmaf(f, b.w, o.v[7]);
                }
                const float inv = inverse_sum(total);
#pragma unroll
                for (int e = 0; e < 8; ++e) o.v[e] *= inv;
                store8<T>(out.at(it.lo + row, head) + c, o);
                if (c == 0) P.lse[(int64_t)head * P.n_tokens + it.lo + row] = fmaf(m, P.scale, logf(total));
            }
        }
        cluster_sync();
    }
}

template <typename T, int STEPS, bool SPLIT> cudaError_t launch(const AttentionParams &P, int64_t blocks, cudaStream_t st)
{
    static std::atomic<uint64_t> set[2];
    constexpr int kSmem = smem_bytes<boxes(STEPS)>();
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(attention_forward_kernel<T, STEPS, SPLIT>), kSmem, set);
    return e == cudaSuccess ? launch_split(attention_forward_kernel<T, STEPS, SPLIT>, P, blocks, kThreads, kSmem, st) : e;
}

template <typename T> cudaError_t launch_type(const AttentionParams &P, int64_t blocks, cudaStream_t st)
{
    if (P.dim <= 64) return P.split > 1 ? launch<T, 4, true>(P, blocks, st) : launch<T, 4, false>(P, blocks, st);
    if (P.dim <= 96) return P.split > 1 ? launch<T, 6, true>(P, blocks, st) : launch<T, 6, false>(P, blocks, st);
    return P.split > 1 ? launch<T, 8, true>(P, blocks, st) : launch<T, 8, false>(P, blocks, st);
}

}  // namespace

cudaError_t launch_attention_forward(const AttentionParams &P0, bool bf16, cudaStream_t st)
{
    const Choice c = choose_forward(P0.n_tokens, P0.n_seqs, P0.n_heads, P0.n_kv, sm_count());
    AttentionParams P = chosen(P0, c);
    P.pair_heads = pairs_heads(P.n_heads, P.n_kv);
    return bf16 ? launch_type<__nv_bfloat16>(P, c.blocks, st) : launch_type<__half>(P, c.blocks, st);
}

}  // namespace dq
