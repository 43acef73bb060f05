// spec_logits_adjust: penalties for repeated tokens, biases and grammar masks
// on the judged rows.
//
// A row's logits change at few tokens (those of the history, of the row's
// path in the draft tree, and those with a bias) but for its mask.  A CTA
// takes one request, one slice of the vocabulary and a group of the request's
// rows:
//   1. the slice's tokens are counted once in shared memory, the same for all
//      of the rows, and a bit set for every touched one;
//   2. the rows' slices pass through registers in 16-byte vectors, several in
//      flight a thread; tokens that the row's mask does not allow become -inf;
//   3. the touched tokens take their penalties and biases, with the
//      occurrences on that row's path found from the ancestor bits of its
//      node.  Up to 256 of them are listed, and their logits written over
//      those of step 2, a thread a (token, row): done with the vectors, each
//      warp would run the adjustment for the one lane that needs it (7 us more
//      on 480 rows of 128256 logits).  In slices with more (the
//      first ones: low ids are the common tokens) it is done with the vectors
//      (11.5 us against 16 on 128 rows of 32000 logits).
// Counts are integers and a token's biases are added in index order, so
// results do not depend on the order of the threads.  Bound by the rows'
// bytes, read and written once (480 rows of 128256 logits: 57 us in bf16, 4.3
// TB/s, without masks 52; 99 us in fp32, 5.0 TB/s), and by the waits of a CTA's counting, ahead of which
// it asks for its first vectors (63 us without); the history is read once per
// CTA, from L2.
#include <math.h>

#include <type_traits>

#include "common.cuh"

namespace sv {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjRows = 16;                 // most rows a CTA takes
constexpr int kAdjResident = 4;              // CTAs an SM holds
constexpr int kAdjFlight = 4;                // vectors in flight a thread
constexpr int kAdjMaxNodes = SPEC_MAX_ROWS;
constexpr int kAdjMaxBias = 1024;
constexpr int kAdjListed = 256;              // touched tokens a slice lists
constexpr int kAdjMaxSlices = 65535;         // (the grid's limit)

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
    int rows;                                // rows a CTA takes
    int *status;
};

template <int kAdjSlice>
struct AdjShared {
    alignas(16) uint32_t cnt[kAdjSlice];     // occurrences behind the prompt
    alignas(16) float add[kAdjSlice];        // the biases, then what a row without the token on
                                             // its path adds
    alignas(16) int16_t node[kAdjSlice];     // first node with the token, -1
    uint32_t hit[kAdjSlice / 32 + 1];        // touched tokens,
    uint32_t old[kAdjSlice / 32 + 1];        // those in the history,
    uint32_t fresh[kAdjSlice / 32 + 1];      // and those of the draft
    uint32_t anc[kAdjMaxNodes][kAdjMaxNodes / 32];   // path of each node
    int draft[kAdjMaxNodes];                 // the slice's nodes in order: token within it << 16 | node
    int mask[kAdjRows], follow[kAdjRows];    // mask and node of each row
    float given[32];                         // biases on their way
    int n_draft, n_list;
    uint16_t list[kAdjListed];               // the touched tokens one after the other, where few
    int16_t up[kAdjMaxNodes], next[kAdjMaxNodes];
    uint8_t bad[kAdjMaxNodes];               // status bits of each node's path
};

// Bits [at, at + 8) of a bit string that has a byte behind its last.
__device__ __forceinline__ uint32_t bits8(const uint32_t *w, int at) {
    const uint8_t *p = reinterpret_cast<const uint8_t *>(w) + (at >> 3);
    return ((p[0] | (uint32_t)p[1] << 8) >> (at & 7)) & 0xffu;
}

// The bytes of x that kSel's digits name (8 + the byte), each replaced by its
// sign (prmt's sign form, which __byte_perm leaves out).
template <uint32_t kSel>
__device__ __forceinline__ uint32_t byte_signs(uint32_t x) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(x), "n"(kSel));
    return r;
}

template <typename T, int kAdjSlice>             // kAdjSlice: vocabulary tokens a CTA takes
__global__ void __launch_bounds__(kAdjThreads, kAdjResident) logits_adjust_kernel(AdjParams P) {
    pdl_wait();
    constexpr int N = 16 / (int)sizeof(T);           // logits a vector
    extern __shared__ __align__(16) uint8_t smem[];
    auto &sh = *reinterpret_cast<AdjShared<kAdjSlice> *>(smem);
    auto &s_cnt = sh.cnt;
    auto &s_add = sh.add;
    auto &s_node = sh.node;
    auto &s_hit = sh.hit;
    auto &s_old = sh.old;
    auto &s_new = sh.fresh;
    auto &s_list = sh.list;
    auto &s_anc = sh.anc;
    auto &s_up = sh.up;
    auto &s_next = sh.next;
    auto &s_bad = sh.bad;
    auto &s_draft = sh.draft;
    auto &s_mask = sh.mask;
    auto &s_follow = sh.follow;
    int &n_list = sh.n_list, &n_draft = sh.n_draft;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.y, v0 = blockIdx.z * kAdjSlice, nv = min(kAdjSlice, P.V - v0);
    const int j0 = blockIdx.x * P.rows, rows = min(P.Rj - j0, P.rows);
    int bits = 0;

    const T *in = static_cast<const T *>(P.logits) + ((size_t)b * P.Rj + j0) * P.V + v0;
    T *out = static_cast<T *>(P.out) + ((size_t)b * P.Rj + j0) * P.V + v0;
    // row j's logits up to its first 16-byte boundary, and its vectors
    auto lead_of = [&](int j) {
        const int off = (int)((reinterpret_cast<uintptr_t>(in + (size_t)j * P.V) & 15) / sizeof(T));
        return min(nv, off ? N - off : 0);
    };
    const bool vectors = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    // vector e0 of rows r0 .., the first ones ahead of everything else
    uint4 x[kAdjFlight];
    int at[kAdjFlight];                              // within the slice, -1 none
    auto load = [&](int e0, int r0) {
#pragma unroll
        for (int f = 0; f < kAdjFlight; ++f) {
            const int j = r0 + f;
            at[f] = -1;
            if (j >= rows || !vectors) continue;
            const int first = lead_of(j) + e0 * N;
            if (first + N > nv) continue;
            at[f] = first;
            x[f] = *reinterpret_cast<const uint4 *>(in + (size_t)j * P.V + first);
        }
    };
    load(tid, 0);

    // what every thread reads, asked for at once: its node, the request's
    // factors, and the first part of the history (whose entries past its
    // length are there, but unused)
    constexpr int kHist = 8;                         // entries in flight a thread
    const int32_t *hist = P.history + (size_t)b * P.H;
    int t[kHist];
#pragma unroll
    for (int u = 0; u < kHist; ++u) {
        const int i = tid + u * kAdjThreads;
        t[u] = i < P.H ? hist[i] : -1;
    }
    int hl = P.H > 0 ? P.hist_len[b] : 0;
    const int np = P.n_prompt ? P.n_prompt[b] : 0;
    const float rep = P.repetition ? P.repetition[b] : 1.f, inv_rep = 1.f / rep;
    const float pres = P.presence ? P.presence[b] : 0.f;
    const float freq = P.frequency ? P.frequency[b] : 0.f;
    int parent = -1, token = -1;
    static_assert(kAdjMaxNodes <= kAdjThreads, "one node a thread");
    if (tid < P.N) {
        parent = P.tree_parent[(size_t)b * P.N + tid];
        token = P.tokens[(size_t)b * P.N + tid];
    }
    constexpr uint32_t kNone = 0x80000000u;          // -0 leaves every x as it is, -0 too
    for (int i = tid; i < kAdjSlice / 4; i += kAdjThreads) {
        reinterpret_cast<uint4 *>(s_cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
        reinterpret_cast<uint4 *>(s_add)[i] = make_uint4(kNone, kNone, kNone, kNone);
        reinterpret_cast<uint2 *>(s_node)[i] = make_uint2(~0u, ~0u);
    }
    if (tid <= kAdjSlice / 32) s_hit[tid] = s_old[tid] = s_new[tid] = 0u;
    // the draft's tokens within the slice, in index order
    if (tid < 32) {
        const int32_t *ids = P.tokens + (size_t)b * P.N;
        int m = 0;
        for (int i0 = 0; i0 < P.N; i0 += 128) {
            int x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                x[u] = i < P.N ? ids[i] : -1;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int v = x[u] - v0;
                const bool mine = x[u] >= 0 && v >= 0 && v < nv;
                const unsigned w = __ballot_sync(0xffffffffu, mine);
                if (mine) s_draft[m + __popc(w & ((1u << lane) - 1u))] = v << 16 | (i0 + 32 * u + lane);
                m += __popc(w);
            }
        }
        if (lane == 0) n_draft = m;
    }
    for (int j = tid; j < rows; j += kAdjThreads) {
        const size_t at = (size_t)b * P.Rj + j0 + j;
        int m = P.n_masks > 0 ? P.row_mask[at] : -1;
        if (P.n_masks > 0 && m >= P.n_masks) {
            bits |= SPEC_DEV_BAD_INDEX;
            m = -1;
        }
        s_mask[j] = m;
        int node = -1;
        if (P.N > 0) node = P.row_node ? P.row_node[at] : j0 + j;
        if (node >= P.N || node < -1) {
            bits |= SPEC_DEV_BAD_INDEX;
            node = -1;
        }
        s_follow[j] = node;
    }
    __syncthreads();

    // the history's tokens of this slice
    if (hl < 0 || hl > P.H) {
        bits |= SPEC_DEV_BAD_INDEX;
        hl = hl < 0 ? 0 : P.H;
    }
    for (int i0 = tid;;) {
#pragma unroll
        for (int u = 0; u < kHist; ++u) {
            const int i = i0 + u * kAdjThreads, v = t[u] - v0;
            if (i >= hl) continue;
            if (t[u] >= P.V) bits |= SPEC_DEV_BAD_INDEX;
            if (t[u] < 0 || v < 0 || v >= nv) continue;
            atomicOr(&s_old[v >> 5], 1u << (v & 31));
            if (i >= np) atomicAdd(&s_cnt[v], 1u);
        }
        i0 += kHist * kAdjThreads;
        if (i0 >= hl) break;
#pragma unroll
        for (int u = 0; u < kHist; ++u) {
            const int i = i0 + u * kAdjThreads;
            t[u] = i < hl ? hist[i] : -1;
        }
    }
    // the biases, by one warp: 32 entries after the other, the first lane of
    // those with one token adds them up in index order
    if (tid >= 32 && tid < 64) {
        const int32_t *ids = P.bias_ids + (size_t)b * P.n_bias;
        const float *bias = P.bias + (size_t)b * P.n_bias;
        for (int i0 = 0; i0 < P.n_bias; i0 += 128) {
            int x[4];
            float y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                x[u] = i < P.n_bias ? ids[i] : -1;
                y[u] = i < P.n_bias ? bias[i] : 0.f;
                if (x[u] >= P.V) bits |= SPEC_DEV_BAD_INDEX;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int v = x[u] - v0;
                const bool mine = x[u] >= 0 && v >= 0 && v < nv;
                if (!__any_sync(0xffffffffu, mine)) continue;
                sh.given[lane] = y[u];
                unsigned peers = __match_any_sync(0xffffffffu, mine ? v : -1 - lane);
                __syncwarp();
                if (mine && lane == __ffs(peers) - 1) {
                    float sum = s_add[v];
                    for (; peers; peers &= peers - 1) sum += sh.given[__ffs(peers) - 1];
                    s_add[v] = sum;
                    atomicOr(&s_hit[v >> 5], 1u << (v & 31));
                }
                __syncwarp();
            }
        }
    }
    // the draft's tokens of this slice
    for (int i = tid; i < n_draft; i += kAdjThreads) {
        const int v = s_draft[i] >> 16, x = s_draft[i] & 0xffff;
        int next = -1;
        for (int k = i + 1; k < n_draft && next < 0; ++k)
            if ((s_draft[k] >> 16) == v) next = s_draft[k] & 0xffff;
        s_next[x] = (int16_t)next;
        bool leads = true;
        for (int k = 0; k < i && leads; ++k) leads = (s_draft[k] >> 16) != v;
        if (!leads) continue;
        s_node[v] = (int16_t)x;
        atomicOr(&s_new[v >> 5], 1u << (v & 31));
    }
    // its paths, where one is looked at (and reported, by the first slice):
    // each node takes on what its ancestor knows, 1, 2, 4, ... levels up
    if (P.N > 0 && (n_draft > 0 || blockIdx.z == 0)) {
        const int x = tid;
        constexpr int kWords = kAdjMaxNodes / 32;
        uint32_t w[kWords];
        int up = -1;
        uint8_t bad = 0;
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = k == (x >> 5) ? 1u << (x & 31) : 0u;
        if (x < P.N) {
            // a node past the tree's end may hold anything, so a bad one is
            // reported only where a row's path meets it, and ends that path
            if (parent >= x || parent < -1) bad |= SPEC_DEV_BAD_TREE;
            else up = parent;
            if (token >= P.V) bad |= SPEC_DEV_BAD_INDEX;
        }
        bool changed;
        do {
            changed = false;
            if (x < P.N) {
                s_up[x] = (int16_t)up;
                s_bad[x] = bad;
#pragma unroll
                for (int k = 0; k < kWords; ++k)
                    if (32 * k < P.N) s_anc[x][k] = w[k];
            }
            __syncthreads();
            if (up >= 0) {
#pragma unroll
                for (int k = 0; k < kWords; ++k)
                    if (32 * k < P.N) w[k] |= s_anc[up][k];
                bad |= s_bad[up];
                up = s_up[up];
                changed = true;
            }
        } while (__syncthreads_or(changed));
        if (blockIdx.z == 0)
            for (int j = tid; j < rows; j += kAdjThreads)
                if (s_follow[j] >= 0) bits |= s_bad[s_follow[j]];
    }
    __syncthreads();
    // what the history's tokens add; the touched ones, listed by one warp
    constexpr int kOwn = kAdjSlice / kAdjThreads, kWords = kAdjSlice / 1024;    // tokens a thread, words a lane
    static_assert(kOwn == 8 || kOwn == 16, "a byte or two of s_old a thread");
    for (uint32_t m = kOwn == 8 ? reinterpret_cast<const uint8_t *>(s_old)[tid]
                                : reinterpret_cast<const uint16_t *>(s_old)[tid]; m; m &= m - 1) {
        const int v = kOwn * tid + __ffs(m) - 1;
        if (s_cnt[v]) s_add[v] -= fmaf(freq, (float)s_cnt[v], pres);
    }
    if (tid < 32) {
        uint32_t m[kWords];
        int n = 0;
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
            const int w = kWords * lane + q;
            m[q] = s_hit[w] | s_old[w] | s_new[w];
            s_hit[w] = m[q];
            n += __popc(m[q]);
        }
        int at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += x;
        }
        const int total = __shfl_sync(0xffffffffu, at, 31);
        if (lane == 0) n_list = total;
        if (total <= kAdjListed) {
            at -= n;
#pragma unroll
            for (int q = 0; q < kWords; ++q)
                for (; m[q]; m[q] &= m[q] - 1)
                    s_list[at++] = (uint16_t)(32 * (kWords * lane + q) + __ffs(m[q]) - 1);
        }
    }
    __syncthreads();
    const bool listed = n_list <= kAdjListed;
    const int words = (P.V + 31) / 32;
    // a touched token's logit, in the row that follows `node`
    auto adjust = [&](float z, int v, int node) {
        float add = s_add[v];
        bool seen = (s_old[v >> 5] >> (v & 31)) & 1u;
        int y = s_node[v];
        if (y >= 0 && node >= 0) {
            int k = 0;                               // occurrences on the path
            for (; y >= 0; y = s_next[y]) k += (s_anc[node][y >> 5] >> (y & 31)) & 1u;
            if (k > 0) {
                seen = true;
                add -= freq * (float)k + (s_cnt[v] == 0u ? pres : 0.f);
            }
        }
        return fmaf(z, !seen ? 1.f : z > 0.f ? inv_rep : rep, add);
    };
    auto allowed = [&](int j, int i) {
        return s_mask[j] < 0 ||
               ((P.mask_bits[(size_t)s_mask[j] * words + ((v0 + i) >> 5)] >> ((v0 + i) & 31)) & 1u);
    };
    // one logit at a time: `n` of row j from `first`; listed tokens are
    // adjusted later
    auto singles = [&](int j, int first, int n) {
#pragma unroll 1
        for (int i = first; i < first + n; ++i) {
            T x = in[(size_t)j * P.V + i];
            if (!allowed(j, i)) store_f(&x, -INFINITY);
            else if (!listed && ((s_hit[i >> 5] >> (i & 31)) & 1u))
                store_f(&x, adjust(load_f(&x), i, s_follow[j]));
            out[(size_t)j * P.V + i] = x;
        }
    };
    if (!vectors)
        for (int i = tid; i < rows * nv; i += kAdjThreads) singles(i / nv, i % nv, 1);
    // A thread takes the same vectors in every row; where the rows begin alike
    // (their length a multiple of 16 bytes) these are the same tokens, and what
    // it knows of them stays in registers.
    constexpr int kVecs = kAdjSlice / N;             // at most, a row
    constexpr uint32_t kAll = (1u << N) - 1u;
    auto pass = [&](auto lists) {
        constexpr bool kLists = decltype(lists)::value;
        for (int e0 = tid; e0 < kVecs && vectors; e0 += kAdjThreads) {
            int known_at = -1;
            uint32_t hit = 0, old = 0, fresh = 0;
            float add[N];
            for (int r0 = 0; r0 < rows; r0 += kAdjFlight) {
                if (r0 > 0 || e0 != tid) load(e0, r0);
                uint32_t ok[kAdjFlight];
#pragma unroll
                for (int f = 0; f < kAdjFlight; ++f) {
                    const int j = r0 + f;
                    ok[f] = kAll;
                    if (at[f] < 0) continue;
                    if (s_mask[j] >= 0) {
                        const int v = v0 + at[f], w = v >> 5, sft = v & 31;
                        const uint32_t *mw = P.mask_bits + (size_t)s_mask[j] * words;
                        uint64_t m = mw[w];
                        if (sft + N > 32) m |= (uint64_t)mw[w + 1] << 32;
                        ok[f] = (uint32_t)(m >> sft) & kAll;
                    }
                }
#pragma unroll
                for (int f = 0; f < kAdjFlight; ++f) {
                    if (at[f] < 0) continue;
                    if (!kLists && at[f] != known_at) {
                        known_at = at[f];
                        hit = bits8(s_hit, known_at) & kAll;
                        if (hit) {
                            old = bits8(s_old, known_at);
                            fresh = bits8(s_new, known_at) & kAll;
#pragma unroll
                            for (int q = 0; q < N; ++q) add[q] = s_add[known_at + q];
                        }
                    }
                    uint32_t e[4] = {x[f].x, x[f].y, x[f].z, x[f].w};
                    if (!kLists && (hit & ok[f])) {
                        auto known = [&](float z, int q) {
                            return fmaf(z, !((old >> q) & 1u) ? 1.f : z > 0.f ? inv_rep : rep, add[q]);
                        };
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if constexpr (N == 8) {
                                const __nv_bfloat162 r = __floats2bfloat162_rn(
                                    known(__uint_as_float(e[q] << 16), 2 * q),
                                    known(__uint_as_float(e[q] & 0xffff0000u), 2 * q + 1));
                                e[q] = *reinterpret_cast<const uint32_t *>(&r);
                            } else {
                                e[q] = __float_as_uint(known(__uint_as_float(e[q]), q));
                            }
                        }
                        // the draft's tokens anew, for this row's path
                        for (uint32_t m = fresh; m; m &= m - 1) {
                            const int q = __ffs(m) - 1, h = q * 4 / N;
                            const uint32_t word = h < 2 ? (h == 0 ? x[f].x : x[f].y) : (h == 2 ? x[f].z : x[f].w);
                            uint32_t keep = 0, z = word;
                            if constexpr (N == 8) {
                                keep = q & 1 ? 0xffffu : 0xffff0000u;
                                z = q & 1 ? word & 0xffff0000u : word << 16;
                            }
                            const float y = adjust(__uint_as_float(z), at[f] + q, s_follow[r0 + f]);
                            z = __float_as_uint(y);
                            if constexpr (N == 8) {
                                z = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y));
                                z = q & 1 ? z << 16 : z;
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k == h) e[k] = (e[k] & keep) | z;
                        }
                    }
                    if (ok[f] != kAll) {
                        if constexpr (N == 8) {
#pragma unroll
                            for (int q = 0; q < 4; q += 2) {
                                // four bits, each at a byte's top, whose sign fills a logit's halves
                                const uint32_t t = (((ok[f] >> 2 * q) & 15u) * 0x00204081u & 0x01010101u) << 7;
                                const uint32_t k0 = byte_signs<0x9988>(t), k1 = byte_signs<0xbbaa>(t);
                                e[q] = (e[q] & k0) | (0xff80ff80u & ~k0);
                                e[q + 1] = (e[q + 1] & k1) | (0xff80ff80u & ~k1);
                            }
                        } else {
#pragma unroll
                            for (int q = 0; q < 4; ++q) e[q] = (ok[f] >> q) & 1u ? e[q] : 0xff800000u;
                        }
                    }
                    *reinterpret_cast<uint4 *>(out + (size_t)(r0 + f) * P.V + at[f]) =
                        make_uint4(e[0], e[1], e[2], e[3]);
                }
            }
        }
    };
    if (listed) pass(std::true_type{});
    else pass(std::false_type{});
    // (the rows' ends outside the vectors: fewer than N logits each)
    for (int i = tid; i < 2 * rows && vectors; i += kAdjThreads) {
        const int j = i >> 1, lead = lead_of(j), tail = (nv - lead) % N;
        if (i & 1) singles(j, nv - tail, tail);
        else singles(j, 0, lead);
    }
    if (!listed) {
        if (bits) raise_status(P.status, bits);
        return;
    }
    __syncthreads();
    // the listed tokens that the row allows, over what was written there
    // (in place, an allowed token's logit is still as it was given)
    int shift = 0;
    while ((1 << shift) < rows) ++shift;
    const int j = tid & ((1 << shift) - 1);
    if (j < rows)
        for (int i0 = tid >> shift; i0 < n_list; i0 += kAdjFlight * (kAdjThreads >> shift)) {
            int v[kAdjFlight];
            float z[kAdjFlight];
            uint32_t w[kAdjFlight];
#pragma unroll
            for (int f = 0; f < kAdjFlight; ++f) {
                const int i = i0 + f * (kAdjThreads >> shift);
                v[f] = i < n_list ? s_list[i] : -1;
                w[f] = ~0u;
                if (v[f] < 0) continue;
                z[f] = load_f(in + (size_t)j * P.V + v[f]);
                if (s_mask[j] >= 0) w[f] = P.mask_bits[(size_t)s_mask[j] * words + ((v0 + v[f]) >> 5)];
            }
#pragma unroll
            for (int f = 0; f < kAdjFlight; ++f)
                if (v[f] >= 0 && ((w[f] >> ((v0 + v[f]) & 31)) & 1u))
                    store_f(out + (size_t)j * P.V + v[f], adjust(z[f], v[f], s_follow[j]));
        }
    if (bits) raise_status(P.status, bits);
}

template <typename T, int kAdjSlice>
spec_status_t launch_adjust(const AdjParams &P, dim3 grid, cudaStream_t s) {
    constexpr size_t kSmem = sizeof(AdjShared<kAdjSlice>);
    const spec_status_t st = set_smem_limit((const void *)logits_adjust_kernel<T, kAdjSlice>, kSmem);
    if (st != SPEC_OK) return st;
    return launch(logits_adjust_kernel<T, kAdjSlice>, grid, dim3(kAdjThreads), kSmem, s, P);
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
    if (d->max_nodes > kAdjMaxNodes || d->n_bias > kAdjMaxBias || d->batch > 65535 ||
        d->vocab > kAdjMaxSlices * 4096)
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
    // Slices of 2048 tokens, or of 4096 for a few rows a request in more CTAs
    // than there are places on the SMs: then the counting is the larger part
    // (199 rows of 73557 logits: 59 us with 2048, 39 with 4096; 17 rows of
    // 28523: 12.7 and 14.1; 60 rows a request: 58 and 69).
    const long long places = (long long)kAdjResident * num_sms();
    const bool wide = P.Rj <= 4 && ceil_div_ll(P.V, 2048) * P.B > places;
    // Rows a CTA: as many as leave one CTA for every place, since each counts
    // the request's history anew, but no more than 16: slices with many touched
    // tokens (often the first: low ids are the common tokens) take longer, so
    // they start first and further CTAs even them out
    const long long slices = ceil_div_ll(P.V, wide ? 4096 : 2048);
    if (slices > kAdjMaxSlices) return SPEC_ERR_UNSUPPORTED;
    const long long parts = places / (slices * P.B);
    const long long rows = ceil_div_ll(P.Rj, parts < 1 ? 1 : parts > P.Rj ? P.Rj : parts);
    P.rows = (int)(rows > kAdjRows ? kAdjRows : rows);
    const dim3 grid((unsigned)ceil_div_ll(P.Rj, P.rows), P.B, (unsigned)slices);
    cudaStream_t s = as_stream(stream);
    const bool bf16 = d->logit_dtype == SPEC_BF16;
    const spec_status_t st = wide ? (bf16 ? launch_adjust<__nv_bfloat16, 4096>(P, grid, s)
                                          : launch_adjust<float, 4096>(P, grid, s))
                                  : (bf16 ? launch_adjust<__nv_bfloat16, 2048>(P, grid, s)
                                          : launch_adjust<float, 2048>(P, grid, s));
    if (st != SPEC_OK) return st;
    return launch_status();
}
