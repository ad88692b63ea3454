// dq_attention.cuh -- what the forward and backward attention kernels share:
// parameters, and where a block's rows lie in the pack.
#pragma once

#include <cuda.h>

#include "dq_act.cuh"
#include "dq_common.cuh"
#include "dq_internal.h"
#include "dq_tc.cuh"

namespace dq {

struct AttentionParams {
    CUtensorMap map_q, map_k, map_v, map_dout;
    dq_heads q, k, v, out, dout, dqv, dk, dv;
    float *lse, *delta;
    float *row_norms;          // fp16, backward: |dout| of each row, n_heads x n_tokens
    float *tile_norms;         // and the largest of each tile, at its first row: of dout, then of v, (n_heads + n_kv) x n_tokens
    int32_t *status;
    const int32_t *cu;
    int32_t n_tokens, n_seqs, n_heads, n_kv, dim, causal;
    float scale, scale_log2;   // of the scores; times log2(e), for exp2
    int32_t y;                 // blocks of the grid that share a slot
    int32_t pair_heads;        // a block's two row tiles: two heads, or two tiles of a head
    int32_t ordered;           // tiles are taken in the order of their work over all sequences
    int32_t split;             // blocks (a cluster) that share a tile's loop: 1, 2, 4 or 8
    int32_t give_up;           // 1: waits have run out from the start (a test)
};

// The kernels are built for heads of up to 64, 96 and 128 elements: products
// over 4, 6 and 8 steps of 16, tiles of one or two boxes of 64.
__host__ __device__ constexpr int boxes(int steps) { return (steps + 3) / 4; }

// Row tiles are numbered without knowing the lengths on the host: sequence s
// owns the slots from floor(cu[s] / rows) + s on.  Those starts ascend
// strictly and leave room for ceil(length / rows) tiles each, since
// ceil(n / r) <= floor((c + n) / r) - floor(c / r) + 1, so a slot's sequence
// is found by a search of cu alone; a slot without a tile is empty.  The
// tokens behind the last sequence are numbered as one more.
struct Slot {
    int lo, len;    // the sequence: its first token, its length
    int row;        // first row of the tile within the sequence
    bool padding;   // tokens of no sequence
};

inline int64_t slot_count(int64_t n_tokens, int64_t n_seqs, int rows) { return n_tokens / rows + n_seqs + 1; }

// Whether the slot has a tile; called by whole warps (32-way search).
__device__ __forceinline__ bool find_slot(const int32_t *cu, int n_seqs, int n_tokens, int slot, int rows, Slot &r)
{
    const int lane = threadIdx.x & 31;
    int a = 0, b = n_seqs + 1;   // the largest s in [a, b) whose first slot is <= slot
    while (b - a > 1) {
        const int step = (b - a + 31) / 32, s = a + step * lane;
        const bool below = s < b && min(max(cu[min(s, n_seqs)], 0), n_tokens) / rows + s <= slot;
        const int n = __popc(__ballot_sync(kFull, below));
        a += step * (n ? n - 1 : 0);
        b = min(b, a + step);
    }
    const int lo = min(max(cu[a], 0), n_tokens);
    const int hi = a < n_seqs ? min(max(cu[a + 1], 0), n_tokens) : n_tokens;
    r.lo = lo;
    r.len = hi - lo;
    r.padding = a == n_seqs;
    r.row = (slot - (lo / rows + a)) * rows;
    return r.row >= 0 && r.row < r.len;
}

// Up to 31 sequences, a lane each: the tile that is number `rank` in the order
// of work, the most first, so that no block is left with a long tile at the
// end.  Under the causal mask a tile's work is its place in the sequence from
// the start (up) or from the end, else the sequence's number of tiles.  It is
// found by the largest T with more than `rank` tiles of work >= T; the tokens
// behind the last sequence come last.
__device__ __forceinline__ bool find_largest(const AttentionParams &P, int rank, int rows, bool up, Slot &r)
{
    const int lane = threadIdx.x & 31;
    const int lo = min(max(P.cu[min(lane, P.n_seqs)], 0), P.n_tokens);
    const int next = lane < P.n_seqs ? min(max(P.cu[lane + 1], 0), P.n_tokens) : P.n_tokens;
    const int len = lane <= P.n_seqs ? max(next - lo, 0) : 0, tiles = lane < P.n_seqs ? (len + rows - 1) / rows : 0;
    auto count = [&](int t) {
        return __reduce_add_sync(kFull, P.causal ? max(tiles - t + 1, 0) : (tiles >= t ? tiles : 0));
    };
    const int all = count(1);
    int s = P.n_seqs;
    r.padding = rank >= all;
    if (r.padding) {
        r.row = (rank - all) * rows;
    } else {
        int t = 1, above = __reduce_max_sync(kFull, tiles) + 1;
        while (above - t > 1) {
            const int m = (t + above) / 2;
            if (count(m) > rank)
                t = m;
            else
                above = m;
        }
        const int k = rank - count(t + 1), i = P.causal ? k : k / t;   // the i-th of the sequences that have such tiles
        const unsigned have = __ballot_sync(kFull, P.causal ? tiles >= t : tiles == t);
        s = __ffs(__ballot_sync(kFull, (have >> lane & 1) && __popc(have & ((1u << lane) - 1)) == i)) - 1;
        const int of = __shfl_sync(kFull, tiles, s);
        r.row = (P.causal ? (up ? t - 1 : of - t) : k % t) * rows;
    }
    r.lo = __shfl_sync(kFull, lo, s);
    r.len = __shfl_sync(kFull, len, s);
    return r.row < r.len;
}

// The tile of block number `index` of `slots`: in the order of work, or in that
// of the slots, from the last (up) or the first on, which under the causal
// mask is the order of work within a sequence.
template <bool BY_WORK = true>
__device__ __forceinline__ bool find_tile(const AttentionParams &P, int index, int slots, int rows, bool up, Slot &r)
{
    if (BY_WORK && P.ordered) return find_largest(P, index, rows, up, r);
    return find_slot(P.cu, P.n_seqs, P.n_tokens, up ? slots - 1 - index : index, rows, r);
}

// A block works through tiles until the grid has none left: its own index
// first, then those of blocks that have not started, which it takes over.  So
// tensor memory and barriers are set up once, and the next tile's first copies
// and products run behind this one's last.  The copy warp takes and decodes a
// tile when it has sent off the last copy for the one before, or a few copies
// earlier: a tile taken ahead is one that an idle block cannot have (two whole
// tiles ahead cost 10%).
struct Item {
    int lo, len;   // the sequence; len < 0: no more work
    int row, y;    // the tile's first row; which of the blocks that share a slot
};

struct ItemQueue {
    unsigned long long full[2], empty[2], claim;
    alignas(16) unsigned long long answer[2];
    alignas(16) Item item[2];
};

// One thread, before the block's first barrier; readers: warps that call next().
__device__ __forceinline__ void init_queue(ItemQueue *q, int readers)
{
    for (int i = 0; i < 2; ++i) {
        tc::mbar_init(smem_addr(&q->full[i]), 1);
        tc::mbar_init(smem_addr(&q->empty[i]), readers);
    }
    tc::mbar_init(smem_addr(&q->claim), 1);
}

// The copy warp's side.  padding(S, y) writes the results of tokens of no
// sequence.
struct Taker {
    ItemQueue *q;
    volatile int *abort;
    unsigned block;
    int published = 0, asked = 0;
    bool own = true;    // the block's own index is still to be done
    bool claims = true; // it may take over others

    enum Found { kTaken, kEnd, kOutOfTime, kNothing };

    // The next tile, published to the readers too, or the end of work, or a wait ran out.  With ONE it looks at one block
    // only, and publishes nothing if that has no tile.  UP: a tile's work grows with its row under the causal mask.
    template <bool BY_WORK, bool UP, bool ONE = false, typename Padding>
    __device__ __forceinline__ Found next(const AttentionParams &P, int slots, int rows, Item &it, Padding padding)
    {
        const int lane = threadIdx.x & 31;
        const uint32_t claim = smem_addr(&q->claim), answer = smem_addr(q->answer);
        bool more = true;
        for (bool found = false; !found;) {
            if (!own && !claims) {
                more = false;
            } else if (!own) {
                if (lane == 0) tc::claim_block(answer, claim);
                if (!tc::mbar_wait(claim, asked & 1, abort)) {
                    tc::mbar_land(claim, asked & 1);   // the answer, before this block's memory goes
                    return kOutOfTime;
                }
                ++asked;
                more = tc::claimed_block(answer, block);
                tc::fence_smem_to_async();   // read before the next answer is written
                __syncwarp();
            }
            own = false;
            if (!more) break;
            const int y = block % P.y;
            Slot S;
            found = find_tile<BY_WORK>(P, block / P.y, slots, rows, UP, S);
            if (found && S.padding) {
                padding(S, y);
                found = false;
            }
            if (ONE && !found) return kNothing;
            it = Item{S.lo, S.len, S.row, y};
        }
        if (!more) it = Item{0, -1, 0, 0};
        const int s = published & 1;
        if (published >= 2 && !tc::mbar_wait(smem_addr(&q->empty[s]), (published / 2 - 1) & 1, abort)) return kOutOfTime;
        if (lane == 0) {
            q->item[s] = it;
            tc::mbar_arrive(smem_addr(&q->full[s]));
        }
        __syncwarp();
        ++published;
        return more ? kTaken : kEnd;
    }
};

// The other warps' (or threads') view of the queue.
struct Tiles {
    ItemQueue *q;
    volatile int *abort;
    int read = 0;
    // false when there is no more work or a wait ran out
    template <bool ONE = false> __device__ __forceinline__ bool next(Item &it)
    {
        const int s = read & 1;
        const uint32_t full = smem_addr(&q->full[s]), parity = (read >> 1) & 1;
        if (!(ONE ? tc::mbar_wait_one(full, parity, abort, tc::kQueueCycles) : tc::mbar_wait(full, parity, abort, tc::kQueueCycles)))
            return false;
        it = q->item[s];
        if (!ONE) __syncwarp();
        if (ONE || (threadIdx.x & 31) == 0) tc::mbar_arrive(smem_addr(&q->empty[s]));
        ++read;
        return it.len >= 0;
    }
};

// A warp writes zeros to n tokens of a head.
template <typename T> __device__ __forceinline__ void zero_heads(const dq_heads &view, int64_t t0, int n, int h, int dim)
{
    const Heads<T> x = heads<T>(view);
    const F8 zero{};
    const int chunks = dim / 8;
    for (int i = threadIdx.x & 31; i < n * chunks; i += 32) store8<T>(x.at(t0 + i / chunks, h) + i % chunks * 8, zero);
}

// A position in a ring of N stages.
template <int N> struct Ring {
    int stage = 0;
    uint32_t phase = 0, laps = 0;   // phase: of the stage's current use; laps: 0 on the first
    __device__ __forceinline__ void step()
    {
        if (++stage == N) {
            stage = 0;
            phase ^= 1;
            laps = 1;
        }
    }
};

// 32 columns of an accumulator, scaled by f (the row's own factor), rounded
// and written to `dst` + row * stride.  A thread holds a row, but a warp that
// wrote 16 bytes of each of its 32 rows would take 32 cycles of the memory
// pipe for each store (5,500 cycles for a 128 x 128 tile); so four lanes
// exchange their pieces first, and write 64 bytes of one row together.
// `row` is the warp's first row; rows from `rows` on are not written.
template <typename T>
__device__ __forceinline__ void store_columns(const uint32_t *acc, float f, T *dst, int64_t stride, int row, int rows, int col,
                                              int dim)
{
    const int lane = threadIdx.x & 31;
    uint32_t w[4][4];   // four pieces of eight elements
#pragma unroll
    for (int i = 0; i < 16; ++i)
        w[i / 4][i % 4] = pack2(__uint_as_float(acc[2 * i]) * f, __uint_as_float(acc[2 * i + 1]) * f, T());
#pragma unroll
    for (int m = 1; m < 4; m *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(i & m)) {
                const bool low = !(lane & m);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t got = __shfl_xor_sync(kFull, low ? w[i | m][k] : w[i][k], m);
                    if (low)
                        w[i | m][k] = got;
                    else
                        w[i][k] = got;
                }
            }
    const int at = col + (lane & 3) * 8;
    if (at < dim) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row + (lane & ~3) + i;
            if (r < rows) *reinterpret_cast<uint4 *>(dst + r * stride + at) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        }
    }
}

// ---- few tiles: the blocks of a cluster share one tile's loop
// Each sums its part of the loop and leaves its fp32 accumulators in its
// shared memory; then each adds up a share of the rows, reading the others'
// shared memory in the order of their ranks, so the result does not depend on
// which block is first.
__device__ __forceinline__ int cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ void cluster_sync()
{
    __syncthreads();   // the cluster's barrier takes converged warps
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 load_peer(uint32_t addr, int rank)
{
    float4 v;
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float load_peer1(uint32_t addr, int rank)
{
    float v;
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// The part of a loop of n steps that a block of the cluster takes.
struct Part {
    int first, n;
    __device__ __forceinline__ Part(int all, int rank, int split) : first(all * rank / split), n(all * (rank + 1) / split - first) {}
};

// Rows of accumulators in shared memory lie four floats further apart than they
// are long, so that the lanes of a warp write them without conflicts.
template <int DIM> __host__ __device__ constexpr int pitch() { return DIM + 4; }

// 32 columns of a thread's own row, or zeros.
__device__ __forceinline__ void leave_columns(float *row, const uint32_t *acc, bool zero)
{
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float4 v = make_float4(__uint_as_float(acc[i]), __uint_as_float(acc[i + 1]), __uint_as_float(acc[i + 2]),
                                     __uint_as_float(acc[i + 3]));
        *reinterpret_cast<float4 *>(row + i) = zero ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : v;
    }
}

// The block's share of the rows of a [128][DIM] sum over the cluster, times f,
// to dst + row * stride; `row` is the tile's first row, rows from `rows` on
// are not written.  All threads of the block, between two cluster_sync.
template <typename T, int DIM>
__device__ __forceinline__ void add_up_rows(uint32_t acc, int rank, int split, float f, T *dst, int64_t stride, int row, int rows,
                                            int dim)
{
    const int share = tc::kTile / split;
    for (int i = threadIdx.x; i < share * (DIM / 8); i += blockDim.x) {
        const int r = rank * share + i / (DIM / 8), c = i % (DIM / 8) * 8;
        if (row + r >= rows || c >= dim) continue;
        const uint32_t at = acc + (uint32_t)(r * pitch<DIM>() + c) * 4;
        F8 sum{};
        for (int s = 0; s < split; ++s) {
            const float4 a = load_peer(at, s), b = load_peer(at + 16, s);
            sum.v[0] += a.x; sum.v[1] += a.y; sum.v[2] += a.z; sum.v[3] += a.w;
            sum.v[4] += b.x; sum.v[5] += b.y; sum.v[6] += b.z; sum.v[7] += b.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] *= f;
        store8<T>(dst + (int64_t)(row + r) * stride + c, sum);
    }
}

// The order of work pays where an SM has a few tiles: dk, dv of 5,096 tokens in
// four sequences, 8 heads of 64, 360 blocks: 74 us against 82; forward of 4,427
// tokens in 12, both ways, 480 blocks: 20.6 us against 22.7.  With more tiles it
// is better to go sequence by sequence, whose keys and rows then stay in L2: dq
// of 12,291 tokens in two, 32 heads of 128, 3,168 blocks: 619 us against 597;
// with one tile or none an SM the order does not matter.
inline int32_t by_work(int64_t blocks, int64_t n_seqs, int sms) { return n_seqs <= 31 && blocks > sms && blocks <= 4 * sms; }

// How many blocks share a tile: as many as (nearly) all run at once, some slots
// being empty, up to 8, while each keeps four steps of the loop that a tile of
// the pack's mean length has (the lengths themselves are not known here):
// shorter parts cost more than they give, 22 against 12 us for the dk, dv of 38
// sequences of 54 tokens.
inline int split_for(int64_t blocks, int64_t steps, int sms)
{
    int split = 1;
    while (split < 8 && blocks * split * 2 <= sms * 3 / 2 && split * 8 <= steps) split *= 2;
    return split;
}

// How a kernel is launched: `blocks` tiles' slots, or as many clusters.
struct Choice {
    int64_t blocks;
    int32_t y, ordered, split;
};

inline int64_t mean_tiles(int64_t n_tokens, int64_t n_seqs) { return n_seqs ? (n_tokens / n_seqs + tc::kTile - 1) / tc::kTile : 1; }

// The forward kernel takes two heads of a group, or two tiles of one head.
inline bool pairs_heads(int32_t n_heads, int32_t n_kv) { return n_heads / n_kv % 2 == 0; }

inline Choice choose_forward(int64_t n_tokens, int64_t n_seqs, int32_t n_heads, int32_t n_kv, int sms)
{
    const bool pair = pairs_heads(n_heads, n_kv);
    Choice c{};
    c.y = pair ? n_heads / 2 : n_heads;
    c.blocks = slot_count(n_tokens, n_seqs, pair ? tc::kTile : 2 * tc::kTile) * c.y;
    // Few tiles: the blocks of a cluster share the keys.  bf16, causal, us without and with: one sequence of 2,048, 4/2
    // heads of 128: 32.5, 23.3; 4,096, 2/1 heads of 64: 40.7, 21.6; 8,192, one head of 128: 95.1, 42.0.  Below 12 key
    // tiles the cluster's barriers and the joining cost what they give: 1,381, 4/2 heads of 96: 22.0, 22.7.
    const int64_t steps = mean_tiles(n_tokens, n_seqs);
    c.ordered = by_work(c.blocks, n_seqs, sms);
    c.split = steps < 12 ? 1 : split_for(c.blocks, steps, sms);
    return c;
}

inline Choice choose_dq(int64_t n_tokens, int64_t n_seqs, int32_t n_heads, int sms)
{
    Choice c{};
    c.y = n_heads;
    c.blocks = slot_count(n_tokens, n_seqs, tc::kTile) * n_heads;
    // (by work: many tiles, or few short ones, and nothing gained: 20 sequences of 300, 8 heads: 20.4 us, by work 21.4)
    c.split = split_for(c.blocks, mean_tiles(n_tokens, n_seqs), sms);
    return c;
}

inline Choice choose_dkv(int64_t n_tokens, int64_t n_seqs, int32_t n_heads, int32_t n_kv, int sms)
{
    Choice c{};
    c.y = n_kv;
    c.blocks = slot_count(n_tokens, n_seqs, tc::kTile) * n_kv;
    const int64_t steps = mean_tiles(n_tokens, n_seqs);
    // (the first tile waits for the search: not for short sequences, 43.5 against 41 us for the backward pass of 20 of 300
    // tokens, 8 heads of 64)
    c.ordered = steps >= 4 && by_work(c.blocks, n_seqs, sms);
    c.split = split_for(c.blocks, steps * (n_heads / n_kv), sms);
    return c;
}

// The parameters with a choice, and its launch.
inline AttentionParams chosen(const AttentionParams &P, const Choice &c)
{
    AttentionParams Q = P;
    Q.y = c.y;
    Q.ordered = c.ordered;
    Q.split = c.split;
    return Q;
}
inline cudaError_t launch_split(void (*kernel)(AttentionParams), const AttentionParams &P, int64_t blocks, int threads, int smem,
                                cudaStream_t st)
{
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(blocks * P.split));
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = P.split;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    c.attrs = &a;
    c.numAttrs = P.split > 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, P);
    note_launches(1);
    return e;
}

cudaError_t launch_attention_forward(const AttentionParams &P, bool bf16, cudaStream_t st);
cudaError_t launch_attention_backward(const AttentionParams &P, bool bf16, cudaStream_t st);

}  // namespace dq
