// dq_attention.cu -- attention over packed sequences, forward and backward
// (dq_attention_forward, dq_attention_backward).
//
//   S = scale q k^T under the mask, lse = log sum exp S, out = exp(S - lse) v
//   P = exp(S - lse), dP = dout v^T, delta = rowsum(dout out)
//   dv = P^T dout, dS = scale P (dP - delta), dq = dS k, dk = dS^T q
//
// Argument checks and tensor maps; the kernels are in dq_attention_fwd.cu and
// dq_attention_bwd.cu.
#include <cudaTypedefs.h>
#include <math.h>

#include "dq_attention.cuh"

namespace dq {
namespace {

dq_status check(const dq_attention *a)
{
    if (!a || (a->dtype != DQ_BF16 && a->dtype != DQ_FP16)) return DQ_ERR_INVALID_ARG;
    if (a->n_heads < 1 || a->n_heads > 65535 || a->n_kv_heads < 1 || a->n_heads % a->n_kv_heads || a->head_dim < 8 ||
        a->head_dim > 128 || a->head_dim % 8 || (a->causal != 0 && a->causal != 1) ||
        !(a->scale > 0.0f && a->scale <= 3.4e38f) || a->n_tokens < 0 || a->n_tokens > INT32_MAX - 128 || a->n_seqs < 0 ||
        a->n_seqs > (1 << 24) || !a->cu_seqlens)
        return DQ_ERR_INVALID_ARG;
    // the largest grid: a block for each slot of 128 rows and head
    if (slot_count(a->n_tokens, a->n_seqs, tc::kTile) * a->n_heads > INT32_MAX) return DQ_ERR_INVALID_ARG;
    return (uintptr_t)a->cu_seqlens & 3u ? DQ_ERR_ALIGNMENT : DQ_OK;
}

std::atomic<int32_t> g_give_up{0};   // dq_attention_give_up_selftest

void fill(AttentionParams &P, const dq_attention *a)
{
    P.cu = a->cu_seqlens;
    P.n_tokens = (int32_t)a->n_tokens;
    P.n_seqs = a->n_seqs;
    P.n_heads = a->n_heads;
    P.n_kv = a->n_kv_heads;
    P.dim = a->head_dim;
    P.causal = a->causal;
    P.scale = a->scale;
    P.scale_log2 = (float)((double)a->scale * 1.4426950408889634074);
    P.give_up = g_give_up.load(std::memory_order_relaxed);
}

// The driver's tensor-map encoder, looked up once.
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static std::atomic<void *> cache{nullptr};
    void *f = cache.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        cache.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// The map of a view's boxes: 64 elements x 1 head x 128 tokens, 128-byte
// swizzle.  Elements from head_dim on and tokens from n_tokens on read as 0,
// so narrower heads and the pack's end need no other code.
bool make_map(CUtensorMap *map, const dq_heads &h, int32_t n_heads, const dq_attention *a)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a->head_dim, (cuuint64_t)n_heads, (cuuint64_t)a->n_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)h.head_stride * 2, (cuuint64_t)h.token_stride * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)tc::kTile}, step[3] = {1, 1, 1};
    return encode(map, a->dtype == DQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, h.ptr,
                  dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One of a call's views: in, checked, to out.
struct ViewArg {
    const dq_heads *in;
    dq_heads *out;
    int32_t n_heads;
};

template <int N> dq_status check_views(const dq_attention *a, const ViewArg (&v)[N])
{
    for (const ViewArg &x : v) {
        const dq_status s = check_heads(x.in, a->n_tokens, x.n_heads, a->head_dim, 2, x.out);
        if (s != DQ_OK) return s;
    }
    return DQ_OK;
}

}  // namespace
}  // namespace dq

extern "C" dq_status dq_attention_forward(const dq_attention *a, const dq_heads *q, const dq_heads *k,
                                          const dq_heads *v, const dq_heads *out, float *lse, int32_t *status_dev,
                                          void *stream)
{
    using namespace dq;
    dq_status s = check(a);
    if (s != DQ_OK) return s;
    if (a->n_tokens == 0) return DQ_OK;
    if (!lse || !status_dev) return DQ_ERR_INVALID_ARG;
    AttentionParams P{};
    fill(P, a);
    const ViewArg views[] = {{q, &P.q, P.n_heads}, {k, &P.k, P.n_kv}, {v, &P.v, P.n_kv}, {out, &P.out, P.n_heads}};
    if ((s = check_views(a, views)) != DQ_OK) return s;
    if (((uintptr_t)lse | (uintptr_t)status_dev) & 3u) return DQ_ERR_ALIGNMENT;
    P.lse = lse;
    P.status = status_dev;
    if (!make_map(&P.map_q, P.q, P.n_heads, a) || !make_map(&P.map_k, P.k, P.n_kv, a) ||
        !make_map(&P.map_v, P.v, P.n_kv, a))
        return DQ_ERR_CUDA;
    return launch_attention_forward(P, a->dtype == DQ_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DQ_OK
               : DQ_ERR_CUDA;
}

extern "C" dq_status dq_attention_plan(const dq_attention *a, int32_t n_sms, dq_attention_launch *plan)
{
    using namespace dq;
    const dq_status s = check(a);
    if (s != DQ_OK) return s;
    if (n_sms < 1 || n_sms > 65535 || !plan) return DQ_ERR_INVALID_ARG;
    const Choice c[3] = {choose_forward(a->n_tokens, a->n_seqs, a->n_heads, a->n_kv_heads, n_sms),
                         choose_dq(a->n_tokens, a->n_seqs, a->n_heads, n_sms),
                         choose_dkv(a->n_tokens, a->n_seqs, a->n_heads, a->n_kv_heads, n_sms)};
    for (int i = 0; i < 3; ++i) plan[i] = dq_attention_launch{c[i].blocks, c[i].split, c[i].ordered};
    return DQ_OK;
}

extern "C" dq_status dq_attention_give_up_selftest(int32_t on)
{
    if (on != 0 && on != 1) return DQ_ERR_INVALID_ARG;
    dq::g_give_up.store(on, std::memory_order_relaxed);
    return DQ_OK;
}

extern "C" size_t dq_attention_backward_workspace_bytes(const dq_attention *a)
{
    using namespace dq;
    if (check(a) != DQ_OK) return 0;
    // delta of each row; fp16: its norms too
    const size_t arrays = a->dtype == DQ_FP16 ? 3 * (size_t)a->n_heads + (size_t)a->n_kv_heads : (size_t)a->n_heads;
    return (arrays * (size_t)a->n_tokens * sizeof(float) + 31) / 16 * 16;
}

extern "C" dq_status dq_attention_backward(const dq_attention *a, const dq_heads *dout, const dq_heads *q,
                                           const dq_heads *k, const dq_heads *v, const dq_heads *out, const float *lse,
                                           const dq_heads *dq_, const dq_heads *dk, const dq_heads *dv, void *ws,
                                           size_t ws_bytes, int32_t *status_dev, void *stream)
{
    using namespace dq;
    dq_status s = check(a);
    if (s != DQ_OK) return s;
    if (a->n_tokens == 0) return DQ_OK;
    if (!lse || !status_dev || !ws || ws_bytes < dq_attention_backward_workspace_bytes(a)) return DQ_ERR_INVALID_ARG;
    AttentionParams P{};
    fill(P, a);
    const ViewArg views[] = {{dout, &P.dout, P.n_heads}, {q, &P.q, P.n_heads}, {k, &P.k, P.n_kv}, {v, &P.v, P.n_kv},
                             {out, &P.out, P.n_heads},   {dq_, &P.dqv, P.n_heads}, {dk, &P.dk, P.n_kv},
                             {dv, &P.dv, P.n_kv}};
    if ((s = check_views(a, views)) != DQ_OK) return s;
    if (((uintptr_t)lse | (uintptr_t)status_dev) & 3u || (uintptr_t)ws & 15u) return DQ_ERR_ALIGNMENT;
    P.lse = const_cast<float *>(lse);
    P.delta = static_cast<float *>(ws);
    if (a->dtype == DQ_FP16) {
        P.row_norms = P.delta + (int64_t)P.n_heads * P.n_tokens;
        P.tile_norms = P.row_norms + (int64_t)P.n_heads * P.n_tokens;
    }
    P.status = status_dev;
    if (!make_map(&P.map_q, P.q, P.n_heads, a) || !make_map(&P.map_dout, P.dout, P.n_heads, a) ||
        !make_map(&P.map_k, P.k, P.n_kv, a) || !make_map(&P.map_v, P.v, P.n_kv, a))
        return DQ_ERR_CUDA;
    return launch_attention_backward(P, a->dtype == DQ_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DQ_OK
               : DQ_ERR_CUDA;
}
