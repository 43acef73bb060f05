// spec_logits_adjust: penalties for repeated tokens, biases and grammar masks
// on the judged rows.
//
// A row's logits change at few tokens (those of the history, of the row's
// path in the draft tree, and those with a bias) but for its mask, so a CTA
// takes one request and one slice of the vocabulary for a group of its rows
// and works in two steps:
//   1. the rows' slices are copied in 16-byte vectors, tokens the mask does
//      not allow as -inf;
//   2. the slice's list of touched tokens -- counted once in shared memory,
//      the same for all of the request's rows -- is applied to every row from
//      the row's own logit, with the occurrences on that row's path found
//      from the ancestor bits of its node.
// Counts are integers and a token's biases are added in index order, so
// results do not depend on the order of the threads.  Bound by the rows'
// bytes, read and written once; one pass over the history per slice comes
// from L2.
#include <math.h>

#include "common.cuh"

namespace sv {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjSlice = 2048;              // vocabulary tokens a CTA takes
constexpr int kAdjMaxNodes = SPEC_MAX_ROWS;
constexpr int kAdjMaxBias = 1024;
constexpr uint32_t kAdjSeen = 0x80000000u;   // in the history (prompt or not)

struct AdjParams {
    const void *logits;
    void *out;
    const int32_t *history, *hist_len, *n_prompt, *tokens, *tree_parent, *row_node;
    const float *repetition, *presence, *frequency;
    const int32_t *bias_ids;
    const float *bias;
    const uint32_t *mask_bits;
    const int32_t *row_mask;
    int B, Rj, V, N, H, n_bias, n_masks;
    int slice, rows;                         // tokens and rows a CTA takes
    int *status;
};

// Copies n elements, element i allowed iff bit v0 + i of mask (mask NULL: all
// are); others become -inf.
template <typename T>
__device__ void copy_masked(T *dst, const T *src, int n, const uint32_t *mask, int v0) {
    constexpr int N = 16 / (int)sizeof(T);
    constexpr uint32_t kNegInf = sizeof(T) == 2 ? 0xff80u : 0xff800000u;
    const int tid = threadIdx.x;
    auto one = [&](int i) {
        T x = src[i];
        if (mask && !((mask[(v0 + i) >> 5] >> ((v0 + i) & 31)) & 1u)) store_f(&x, -INFINITY);
        dst[i] = x;
    };
    if (((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(src)) & 15) != 0) {
        for (int i = tid; i < n; i += kAdjThreads) one(i);
        return;
    }
    // up to the first 16-byte boundary, vectors, the rest
    const int off = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    const int lead = min(n, off ? N - off : 0);
    if (tid < lead) one(tid);
    const int nv = (n - lead) / N;
    const uint4 *sp = reinterpret_cast<const uint4 *>(src + lead);
    uint4 *dp = reinterpret_cast<uint4 *>(dst + lead);
    for (int i = tid; i < nv; i += kAdjThreads) {
        uint4 x = sp[i];
        if (mask) {
            // the vector's N mask bits, which may lie in two words
            const int v = v0 + lead + i * N;
            const int w = v >> 5, s = v & 31;
            uint64_t m = mask[w];
            if (s + N > 32) m |= (uint64_t)mask[w + 1] << 32;
            const uint32_t ok = (uint32_t)(m >> s);
            uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (N == 8) {
                    if (!((ok >> (2 * j)) & 1u)) e[j] = (e[j] & 0xffff0000u) | kNegInf;
                    if (!((ok >> (2 * j + 1)) & 1u)) e[j] = (e[j] & 0xffffu) | (kNegInf << 16);
                } else {
                    if (!((ok >> j) & 1u)) e[j] = kNegInf;
                }
            }
            x = make_uint4(e[0], e[1], e[2], e[3]);
        }
        dp[i] = x;
    }
    const int t0 = lead + nv * N;
    if (t0 + tid < n) one(t0 + tid);         // fewer than N <= kAdjThreads are left
}

template <typename T>
__global__ void __launch_bounds__(kAdjThreads) logits_adjust_kernel(AdjParams P) {
    pdl_wait();
    __shared__ uint32_t s_cnt[kAdjSlice];            // occurrences behind the prompt | kAdjSeen
    __shared__ float s_bias[kAdjSlice];
    __shared__ int16_t s_node[kAdjSlice];            // first node with the token, -1
    __shared__ uint16_t s_list[kAdjSlice];           // the touched tokens
    __shared__ uint32_t s_anc[kAdjMaxNodes][kAdjMaxNodes / 32];   // path of each node
    __shared__ int16_t s_par[kAdjMaxNodes], s_next[kAdjMaxNodes];
    __shared__ int s_tok[kAdjMaxNodes];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.y, v0 = blockIdx.x * P.slice, nv = min(P.slice, P.V - v0);
    const int j0 = blockIdx.z * P.rows, j1 = min(P.Rj, j0 + P.rows);
    int bits = 0;
    const T *in = static_cast<const T *>(P.logits) + (size_t)b * P.Rj * P.V + v0;
    T *out = static_cast<T *>(P.out) + (size_t)b * P.Rj * P.V + v0;

    for (int i = tid; i < nv; i += kAdjThreads) {
        s_cnt[i] = 0u;
        s_bias[i] = 0.f;
        s_node[i] = -1;
    }
    for (int x = tid; x < P.N; x += kAdjThreads) {
        const int p = P.tree_parent[(size_t)b * P.N + x];
        // -2: the path ends here for a bad parent (a node past the tree's end
        // may hold anything, so it is reported only where a row's path meets
        // it)
        s_par[x] = (int16_t)((p >= x || p < -1) ? -2 : p);
        s_tok[x] = P.tokens[(size_t)b * P.N + x];
    }
    if (tid == 0) s_n = 0;
    __syncthreads();

    // the history's tokens of this slice
    int hl = P.H > 0 ? P.hist_len[b] : 0;
    if (hl < 0 || hl > P.H) {
        bits |= SPEC_DEV_BAD_INDEX;
        hl = hl < 0 ? 0 : P.H;
    }
    const int np = P.n_prompt ? P.n_prompt[b] : 0;
    const int32_t *hist = P.history + (size_t)b * P.H;
    for (int i0 = tid; i0 < hl; i0 += 4 * kAdjThreads) {
        int t[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kAdjThreads;
            t[u] = i < hl ? hist[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (t[u] >= P.V) bits |= SPEC_DEV_BAD_INDEX;
            const int v = t[u] - v0;
            if (t[u] < 0 || v < 0 || v >= nv) continue;
            atomicOr(&s_cnt[v], kAdjSeen);
            if (i0 + u * kAdjThreads >= np) atomicAdd(&s_cnt[v], 1u);
        }
    }
    // the biases: the first entry of a token adds up all of them, in order
    const int32_t *ids = P.bias_ids + (size_t)b * P.n_bias;
    const float *bias = P.bias + (size_t)b * P.n_bias;
    for (int i = tid; i < P.n_bias; i += kAdjThreads) {
        const int t = ids[i], v = t - v0;
        if (t >= P.V) bits |= SPEC_DEV_BAD_INDEX;
        if (t < 0 || v < 0 || v >= nv) continue;
        bool leads = true;
        for (int k = 0; k < i && leads; ++k) leads = ids[k] != t;
        if (!leads) continue;
        float x = bias[i];
        for (int k = i + 1; k < P.n_bias; ++k)
            if (ids[k] == t) x += bias[k];
        s_bias[v] = x;
    }
    // the draft's paths, and its tokens of this slice
    for (int x = tid; x < P.N; x += kAdjThreads) {
        uint32_t w[kAdjMaxNodes / 32];
#pragma unroll
        for (int k = 0; k < kAdjMaxNodes / 32; ++k) w[k] = 0u;
        for (int y = x; y >= 0; y = s_par[y])
#pragma unroll
            for (int k = 0; k < kAdjMaxNodes / 32; ++k)
                if (k == (y >> 5)) w[k] |= 1u << (y & 31);
#pragma unroll
        for (int k = 0; k < kAdjMaxNodes / 32; ++k) s_anc[x][k] = w[k];
        const int t = s_tok[x], v = t - v0;
        if (t >= 0 && t < P.V && v >= 0 && v < nv) {
            int next = -1;
            for (int y = x + 1; y < P.N && next < 0; ++y)
                if (s_tok[y] == t) next = y;
            s_next[x] = (int16_t)next;
            bool leads = true;
            for (int y = 0; y < x && leads; ++y) leads = s_tok[y] != t;
            if (leads) s_node[v] = (int16_t)x;
        }
    }
    // step 1, which touches none of the above
    for (int j = j0; j < j1; ++j) {
        int m = P.n_masks > 0 ? P.row_mask[(size_t)b * P.Rj + j] : -1;
        if (m >= P.n_masks && P.n_masks > 0) {
            bits |= SPEC_DEV_BAD_INDEX;
            m = -1;
        }
        const uint32_t *mask = m >= 0 ? P.mask_bits + (size_t)m * ((P.V + 31) / 32) : nullptr;
        if (mask || in != out)
            copy_masked(out + (size_t)j * P.V, in + (size_t)j * P.V, nv, mask, v0);
    }
    __syncthreads();

    // the touched tokens
    for (int i = tid; i < kAdjSlice; i += kAdjThreads) {
        const bool on = i < nv && (s_cnt[i] != 0u || s_node[i] >= 0 || s_bias[i] != 0.f);
        const unsigned m = __ballot_sync(0xffffffffu, on);
        int at = 0;
        if (lane == 0 && m) at = atomicAdd(&s_n, __popc(m));
        at = __shfl_sync(0xffffffffu, at, 0);
        if (on) s_list[at + __popc(m & ((1u << lane) - 1u))] = (uint16_t)i;
    }
    __syncthreads();
    const int n = s_n;
    const float rep = P.repetition ? P.repetition[b] : 1.f;
    const float pres = P.presence ? P.presence[b] : 0.f;
    const float freq = P.frequency ? P.frequency[b] : 0.f;
    for (int j = j0 + (tid >> 5); j < j1; j += kAdjThreads / 32) {
        int node = -1;
        if (P.N > 0) node = P.row_node ? P.row_node[(size_t)b * P.Rj + j] : j;
        if (node >= P.N || node < -1) {
            bits |= SPEC_DEV_BAD_INDEX;
            node = -1;
        }
        if (blockIdx.x == 0) {            // this row's path: reported once
            for (int y = node; y != -1; y = s_par[y]) {
                if (y == -2) {
                    bits |= SPEC_DEV_BAD_TREE;
                    break;
                }
                if (s_tok[y] >= P.V) bits |= SPEC_DEV_BAD_INDEX;
            }
        }
        const int m = P.n_masks > 0 ? P.row_mask[(size_t)b * P.Rj + j] : -1;
        const uint32_t *mask =
            m >= 0 && m < P.n_masks ? P.mask_bits + (size_t)m * ((P.V + 31) / 32) : nullptr;
        for (int i = lane; i < n; i += 32) {
            const int v = s_list[i];
            if (mask && !((mask[(v0 + v) >> 5] >> ((v0 + v) & 31)) & 1u)) continue;
            const uint32_t c = s_cnt[v];
            int k = (int)(c & ~kAdjSeen);
            if (node >= 0)
                for (int y = s_node[v]; y >= 0; y = s_next[y])
                    k += (s_anc[node][y >> 5] >> (y & 31)) & 1u;
            float z = load_f(in + (size_t)j * P.V + v);
            if (k > 0 || (c & kAdjSeen)) z = z > 0.f ? z / rep : z * rep;
            z = z - freq * (float)k - (k > 0 ? pres : 0.f) + s_bias[v];
            store_f(out + (size_t)j * P.V + v, z);
        }
    }
    if (bits) raise_status(P.status, bits);
}

}  // namespace
}  // namespace sv

extern "C" spec_status_t spec_logits_adjust(
    const spec_logits_desc *d, const void *logits, void *out, const int32_t *history,
    const int32_t *hist_len, const int32_t *n_prompt, const int32_t *tokens,
    const int32_t *tree_parent, const int32_t *row_node, const float *repetition,
    const float *presence, const float *frequency, const int32_t *bias_ids, const float *bias,
    const uint32_t *mask_bits, const int32_t *row_mask, void *stream) {
    using namespace sv;
    if (!d || d->batch < 0 || d->n_judge_rows <= 0 || d->vocab <= 0 || d->max_nodes < 0 ||
        d->hist_cap < 0 || d->n_bias < 0 || d->n_masks < 0)
        return SPEC_ERR_INVALID_ARG;
    if (d->logit_dtype != SPEC_F32 && d->logit_dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
    if (d->max_nodes > kAdjMaxNodes || d->n_bias > kAdjMaxBias || d->batch > 65535)
        return SPEC_ERR_UNSUPPORTED;
    if (d->batch == 0) return SPEC_OK;
    if (!logits || !out || (d->hist_cap > 0 && (!history || !hist_len)) ||
        (d->max_nodes > 0 && (!tokens || !tree_parent)) ||
        (d->n_bias > 0 && (!bias_ids || !bias)) || (d->n_masks > 0 && (!mask_bits || !row_mask)))
        return SPEC_ERR_INVALID_ARG;
    AdjParams P{};
    P.logits = logits;
    P.out = out;
    P.history = history;
    P.hist_len = hist_len;
    P.n_prompt = n_prompt;
    P.tokens = tokens;
    P.tree_parent = tree_parent;
    P.row_node = row_node;
    P.repetition = repetition;
    P.presence = presence;
    P.frequency = frequency;
    P.bias_ids = bias_ids;
    P.bias = bias;
    P.mask_bits = mask_bits;
    P.row_mask = row_mask;
    P.B = d->batch;
    P.Rj = d->n_judge_rows;
    P.V = d->vocab;
    P.N = d->max_nodes;
    P.H = d->hist_cap;
    P.n_bias = d->n_bias;
    P.n_masks = d->n_masks;
    P.status = status_ptr();
    if (!P.status) return SPEC_ERR_CUDA;
    P.slice = kAdjSlice;
    P.rows = P.Rj;
    const int slices = ceil_div(P.V, P.slice);
    // rows split until every SM has two CTAs
    while (P.rows > 1 && (long long)slices * P.B * ceil_div(P.Rj, P.rows) < 2ll * num_sms())
        P.rows = ceil_div(P.rows, 2);
    const dim3 grid(slices, P.B, ceil_div(P.Rj, P.rows));
    if (grid.z > 65535) return SPEC_ERR_UNSUPPORTED;
    cudaStream_t s = as_stream(stream);
    const spec_status_t st =
        d->logit_dtype == SPEC_BF16
            ? launch(logits_adjust_kernel<__nv_bfloat16>, grid, dim3(kAdjThreads), 0, s, P)
            : launch(logits_adjust_kernel<float>, grid, dim3(kAdjThreads), 0, s, P);
    if (st != SPEC_OK) return st;
    return launch_status();
}
