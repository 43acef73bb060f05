// kv_append: a packed batch of new K/V rows into the bf16 / fp32 cache, at the
// slots that spec_page_plan gave them.
//
// A copy: every element is read once and written once, in 16-byte vectors.  A
// token's row of all heads is read as one run; within the cache it is a run of
// 64 elements (paged) or of a head (contiguous) at a fixed stride, so a
// vector's place is its token's plus a multiple of that stride.
//
// Bound by memory: 33 K tokens of 8 heads of 128 in bf16 (272 MB) take 43 us, 6.3
// TB/s, 92 % of a copy's rate; a few hundred 3.4 us, a launch and two dependent
// reads.
#include "common.cuh"
#include "kv8.cuh"

namespace sv {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyTokens = 64;      // most tokens of a CTA

struct AppendParams {
    const uint4 *k, *v;
    long long stride_k, stride_v;    // vectors between two tokens' rows
    uint4 *kc, *vc;
    const int64_t *slots;
    long long n_slots;
    long long block, row;            // vectors of a page (a request), of a token within a run's rows
    long long run_stride;            // vectors between two runs of a token
    int run_shift;                   // a run is 2^run_shift vectors
    int n, rows;                     // tokens, tokens per page (request)
    int vecs;                        // vectors of a token's row
    int tpc;                         // tokens of a CTA
    int *status;
};

__global__ void __launch_bounds__(kCopyThreads) kv_append_kernel(AppendParams P) {
    pdl_wait();
    __shared__ long long s_at[kCopyTokens];
    const int base = blockIdx.x * P.tpc, nt = min(P.tpc, P.n - base);
    if (threadIdx.x < nt) {
        const long long s = P.slots[base + threadIdx.x];
        long long at = -1;
        if (s >= P.n_slots) {
            if (blockIdx.y == 0) raise_status(P.status, SPEC_DEV_BAD_PAGE);
        } else if (s >= 0) {
            at = s / P.rows * P.block + s % P.rows * P.row;
        }
        s_at[threadIdx.x] = at;
    }
    __syncthreads();
    const uint4 *src = blockIdx.y ? P.v : P.k;
    uint4 *dst = blockIdx.y ? P.vc : P.kc;
    const long long stride = blockIdx.y ? P.stride_v : P.stride_k;
    const int total = nt * P.vecs, mask = (1 << P.run_shift) - 1;
    constexpr int U = 4;
    for (int f0 = threadIdx.x; f0 < total; f0 += U * kCopyThreads) {
        uint4 x[U];
        long long to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int f = f0 + u * kCopyThreads;
            to[u] = -1;
            if (f >= total) continue;
            const int t = f / P.vecs, i = f - t * P.vecs;
            const long long at = s_at[t];
            if (at < 0) continue;
            to[u] = at + (long long)(i >> P.run_shift) * P.run_stride + (i & mask);
            x[u] = __ldg(src + (long long)(base + t) * stride + i);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (to[u] >= 0) dst[to[u]] = x[u];
    }
}

}  // namespace
}  // namespace sv

extern "C" spec_status_t kv_append(const spec_kv_desc *cache, int n_tokens, const void *k,
                                   long long row_stride_k, const void *v, long long row_stride_v,
                                   const int64_t *slot_map, void *stream) {
    using namespace sv;
    if (!cache || n_tokens < 0) return SPEC_ERR_INVALID_ARG;
    const bool paged = cache->kind == SPEC_KV_PAGED;
    if (!paged && cache->kind != SPEC_KV_CONTIGUOUS) return SPEC_ERR_INVALID_ARG;
    if (cache->dtype != SPEC_F32 && cache->dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
    if (cache->n_kv_heads <= 0) return SPEC_ERR_INVALID_ARG;
    if (cache->head_dim != 64 && cache->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
    if (paged ? cache->n_pages <= 0 || cache->page_size <= 0 : cache->batch <= 0 || cache->max_seq <= 0)
        return SPEC_ERR_INVALID_ARG;
    if (paged && cache->page_size % 16 != 0) return SPEC_ERR_UNSUPPORTED;
    const long long width = (long long)cache->n_kv_heads * cache->head_dim;
    if (row_stride_k < width || row_stride_v < width) return SPEC_ERR_INVALID_ARG;
    const int es = cache->dtype == SPEC_BF16 ? 2 : 4, per = 16 / es;      // elements a vector
    if (width / per > (1 << 24)) return SPEC_ERR_UNSUPPORTED;
    if (n_tokens == 0) return SPEC_OK;
    if (!k || !v || !slot_map || !cache->k || !cache->v) return SPEC_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache->k) || !aligned16(cache->v) ||
        row_stride_k % per != 0 || row_stride_v % per != 0)
        return SPEC_ERR_INVALID_ARG;
    AppendParams P{};
    P.k = static_cast<const uint4 *>(k);
    P.v = static_cast<const uint4 *>(v);
    P.stride_k = row_stride_k / per;
    P.stride_v = row_stride_v / per;
    P.kc = static_cast<uint4 *>(cache->k);
    P.vc = static_cast<uint4 *>(cache->v);
    P.slots = slot_map;
    P.n = n_tokens;
    P.vecs = (int)(width / per);
    const int run = (paged ? 64 : cache->head_dim) / per;                 // 8, 16 or 32 vectors
    P.run_shift = run == 8 ? 3 : run == 16 ? 4 : 5;
    P.rows = paged ? cache->page_size : cache->max_seq;
    P.n_slots = (long long)(paged ? cache->n_pages : cache->batch) * P.rows;
    P.row = run;
    P.run_stride = (long long)P.rows * run;
    P.block = P.run_stride * (P.vecs / run);
    P.status = status_ptr();
    if (!P.status) return SPEC_ERR_CUDA;
    // tokens of a CTA: eight vectors a thread
    P.tpc = 8 * kCopyThreads / P.vecs;
    P.tpc = P.tpc < 1 ? 1 : P.tpc > kCopyTokens ? kCopyTokens : P.tpc;
    const dim3 grid((unsigned)ceil_div(n_tokens, P.tpc), 2);
    if (launch(kv_append_kernel, grid, dim3(kCopyThreads), 0, as_stream(stream), P) != SPEC_OK)
        return SPEC_ERR_CUDA;
    return launch_status();
}
