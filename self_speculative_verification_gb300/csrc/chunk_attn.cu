// spec_chunk_attn and spec_chunk_attn_kv8: attention of new tokens that the
// cache already holds, each over everything up to itself.
//
//   o_i = sum_t exp(q_i . k_t scale - lse_i) v_t,  lse_i = ln sum_t exp(q_i . k_t scale),
//   t = 0 .. seq_len + i
//
// This file holds the entry points, the CUDA-core kernel (fp32 rows) and the
// kernel that merges the parts of units that several CTAs shared.
#include <math.h>

#include "chunk_attn.cuh"
#include "kv8_common.cuh"

namespace sv {
namespace {

constexpr int kRows = 32;        // packed rows of a CUDA-core unit
constexpr int kKeys = 64;        // keys of a step
constexpr int kSimtThreads = 128;
constexpr int kSimtPerSm = 2;

enum { kCacheRows = 0, kCache8 = 1 };

template <int D>
struct ChunkSimtShared {
    float q[kRows][D];
    float k[kKeys][D + 4];       // (a quarter warp's rows start in different banks)
    float v[kKeys][D];
    float p[kRows][kKeys + 4];
    ChunkShare share;
};

// Where token t of (request b, head h) has its key and value rows, and an 8-bit
// block's scales; null for a page id outside the cache (SPEC_DEV_BAD_PAGE),
// whose tokens count as zeros.
struct ChunkRow {
    const uint8_t *k, *v;
    float ks, vs;
};

template <int D, int kCache>
__device__ __forceinline__ ChunkRow chunk_row(const ChunkParams &P, int b, int h, int t) {
    ChunkRow r{nullptr, nullptr, 1.f, 1.f};
    const uint8_t *kc = static_cast<const uint8_t *>(P.kc), *vc = static_cast<const uint8_t *>(P.vc);
    if (kCache == kCacheRows && !P.paged) {
        const size_t at = (((size_t)b * P.Hkv + h) * P.capacity + t) * D * 4;
        r.k = kc + at;
        r.v = vc + at;
        return r;
    }
    const int page = __ldg(P.page_table + (size_t)b * P.max_pages + t / P.ps), off = t % P.ps;
    if (page < 0 || page >= P.n_pages) {
        raise_status(P.status, SPEC_DEV_BAD_PAGE);
        return r;
    }
    if (kCache == kCache8) {
        const size_t at = kv8_block(page, h, P.Hkv, P.ps, D);
        r.k = kc + at + kv8_row(off, 0, D);
        r.v = kc + at + kv8_row(off, 1, D);
        const float *s = P.scales + ((size_t)page * P.Hkv + h) * 2;
        r.ks = kv8_read_scale(__ldg(s));
        r.vs = kv8_read_scale(__ldg(s + 1));
    } else {
        const size_t at = (((size_t)page * P.Hkv + h) * (D / 64) * P.ps + off) * 256;
        r.k = kc + at;
        r.v = vc + at;
    }
    return r;
}

// Elements c .. c + 3 of such a row.
template <int D, int kCache>
__device__ __forceinline__ float4 chunk_elems(const ChunkParams &P, const uint8_t *row, float scale, int c) {
    if (kCache == kCache8) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(row + c));
        const float2 lo = from_e4m3x2(w & 0xffffu), hi = from_e4m3x2(w >> 16);
        return make_float4(lo.x * scale, lo.y * scale, hi.x * scale, hi.y * scale);
    }
    // (paged: the 64-element blocks of a head are a page's rows apart)
    const size_t at = P.paged ? (size_t)(c / 64) * P.ps * 256 + (c % 64) * 4 : (size_t)c * 4;
    return __ldg(reinterpret_cast<const float4 *>(row + at));
}

// The CUDA-core kernel, everything in fp32: the tensor cores have no fp32 product.
// 128 threads: thread (ty, tx) has the scores of rows 4 ty .. + 3 and keys tx + 16
// i, and the outputs of the same rows and dimensions 4 tx + 64 i .. + 3, so that a
// 16-byte read of shared memory feeds eight FMAs and more.  Long calls are bound by
// those; the smallest (two chunks of 8 tokens behind 200: 14 us with the merging launch)
// by a few steps' chains -- page id, loads, products -- after the share of the
// work is found.
template <int D, int kCache>
__global__ void __launch_bounds__(kSimtThreads, kSimtPerSm) chunk_simt_kernel(ChunkParams P) {
    pdl_wait();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    ChunkSimtShared<D> &sh = *reinterpret_cast<ChunkSimtShared<D> *>(smem_raw);
    constexpr int NC = D / 64;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    chunk_share<kSimtThreads>(P, sh.share);
    ChunkWalk walk(P, sh.share);
    ChunkPart u;
    while (walk.next(P, u)) {
        const long long rows = (long long)u.n * P.G, r0 = (long long)u.j * kRows;
        const int nr = (int)min((long long)kRows, rows - r0);
        __syncthreads();
        for (int i = tid; i < kRows * (D / 4); i += kSimtThreads) {
            const int r = i / (D / 4), c = (i % (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < nr) {
                const long long p = r0 + r;
                const float *src = static_cast<const float *>(P.q) + (u.first + p / P.G) * P.stride_q +
                               ((long long)u.h * P.G + p % P.G) * D + c;
                x = *reinterpret_cast<const float4 *>(src);
            }
            *reinterpret_cast<float4 *>(&sh.q[r][c]) = x;
        }
        int seen[4];                                     // tokens this thread's rows see
        float m[4], l[4], acc[4][NC][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            seen[i] = r < nr ? u.S + (int)((r0 + r) / P.G) + 1 : 0;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][c][e] = 0.f;
        }
        const int last = u.S + (int)((r0 + nr - 1) / P.G) + 1;
        for (int s = u.s0; s < u.s1; ++s) {
            const int t0 = s * kKeys, nk = min(kKeys, last - t0);
            __syncthreads();
            bool odd = false;                            // a non-finite value among them
            // a thread's vectors are of one column, every kStep-th token: their rows
            // are found first, then all loads are in flight at once
            constexpr int kStep = kSimtThreads / (D / 4), kBatch = 8;
            const int c = (tid % (D / 4)) * 4, tr = tid / (D / 4);
            for (int i0 = 0; i0 < kKeys; i0 += kStep * kBatch) {
                ChunkRow row[kBatch];
                float4 k[kBatch], v[kBatch];
#pragma unroll
                for (int e = 0; e < kBatch; ++e) {
                    const int t = i0 + e * kStep + tr;
                    row[e] = ChunkRow{nullptr, nullptr, 1.f, 1.f};
                    if (t < nk) row[e] = chunk_row<D, kCache>(P, u.b, u.h, t0 + t);
                }
#pragma unroll
                for (int e = 0; e < kBatch; ++e) {
                    k[e] = v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (row[e].k) {
                        k[e] = chunk_elems<D, kCache>(P, row[e].k, row[e].ks, c);
                        v[e] = chunk_elems<D, kCache>(P, row[e].v, row[e].vs, c);
                    }
                }
#pragma unroll
                for (int e = 0; e < kBatch; ++e) {
                    const int t = i0 + e * kStep + tr;
                    odd = odd || !(fabsf(v[e].x) < INFINITY && fabsf(v[e].y) < INFINITY && fabsf(v[e].z) < INFINITY &&
                                   fabsf(v[e].w) < INFINITY);
                    *reinterpret_cast<float4 *>(&sh.k[t][c]) = k[e];
                    *reinterpret_cast<float4 *>(&sh.v[t][c]) = v[e];
                }
            }
            odd = __syncthreads_or(odd);
            if (tid / 32 * 8 >= nr) continue;            // (a warp's eight rows: none)
            float x[4][4] = {};
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 a[4], k[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(&sh.q[ty * 4 + i][c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) k[i] = *reinterpret_cast<const float4 *>(&sh.k[tx + 16 * i][c]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[i][j] = fmaf(a[i].w, k[j].w, fmaf(a[i].z, k[j].z, fmaf(a[i].y, k[j].y, fmaf(a[i].x, k[j].x, x[i][j]))));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float top = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = t0 + tx + 16 * j < seen[i] ? x[i][j] * P.scale_log2 : -INFINITY;
                    top = fmaxf(top, x[i][j]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float base = top == -INFINITY ? 0.f : top;
                const float alpha = m[i] == -INFINITY ? (l[i] == 0.f ? 0.f : 1.f) : exp2f(m[i] - base);
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = t0 + tx + 16 * j < seen[i] ? exp2f(x[i][j] - base) : 0.f;
                    sum += p;
                    sh.p[ty * 4 + i][tx + 16 * j] = p;
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                l[i] = l[i] * alpha + sum;
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][c][e] *= alpha;
            }
            __syncwarp();
            if (!odd) {
#pragma unroll 2
                for (int t = 0; t < kKeys; t += 4) {
                    float4 p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(&sh.p[ty * 4 + i][t]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            const float4 v = *reinterpret_cast<const float4 *>(&sh.v[t + k][tx * 4 + 64 * c]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float w = k == 0 ? p[i].x : k == 1 ? p[i].y : k == 2 ? p[i].z : p[i].w;
                                acc[i][c][0] = fmaf(w, v.x, acc[i][c][0]);
                                acc[i][c][1] = fmaf(w, v.y, acc[i][c][1]);
                                acc[i][c][2] = fmaf(w, v.z, acc[i][c][2]);
                                acc[i][c][3] = fmaf(w, v.w, acc[i][c][3]);
                            }
                        }
                }
            } else {                                     // (0 * NaN: only what a row sees)
                for (int t = 0; t < kKeys; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (t0 + t >= seen[i]) continue;
                        const float w = sh.p[ty * 4 + i][t];
#pragma unroll
                        for (int c = 0; c < NC; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[i][c][e] = fmaf(w, sh.v[t][tx * 4 + 64 * c + e], acc[i][c][e]);
                    }
            }
        }
        const bool whole = u.s0 == 0 && u.s1 == u.steps;
        const int slot = chunk_slot(u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= nr) continue;
            if (whole) {
                const long long p = r0 + r, row = u.first + p / P.G, hq = (long long)u.h * P.G + p % P.G;
                float *o = static_cast<float *>(P.o) + (row * P.Hq + hq) * D;
                const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    *reinterpret_cast<float4 *>(o + tx * 4 + 64 * c) =
                        make_float4(acc[i][c][0] * inv, acc[i][c][1] * inv, acc[i][c][2] * inv, acc[i][c][3] * inv);
                if (tx == 0)
                    P.lse[row * P.Hq + hq] = l[i] == 0.f ? -INFINITY
                                             : l[i] != l[i] ? l[i]
                                                            : (m[i] + log2f(l[i])) * kLn2;
            } else {
                float *o = P.part_o + ((size_t)slot * kRows + r) * D;
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    *reinterpret_cast<float4 *>(o + tx * 4 + 64 * c) =
                        make_float4(acc[i][c][0], acc[i][c][1], acc[i][c][2], acc[i][c][3]);
                if (tx == 0) P.part_ml[(size_t)slot * kRows + r] = make_float2(m[i], l[i]);
            }
        }
    }
}

constexpr int kMergeWarps = 8;
// rows of a warp, and parts of them, in flight (64 registers: 2 x 3 of D = 128; a
// unit of the fp32 kernel has more parts, its steps being shorter)
template <typename T> constexpr int kMergeRows = sizeof(T) == 2 ? 2 : 1;
template <typename T> constexpr int kMergeParts = sizeof(T) == 2 ? 3 : 4;

// Merges the parts of the unit that is first cut where CTA blockIdx.x + 1
// begins, in the parts' order; no read depends on more
// than the records, since the call's end waits for them (four rows of a warp after
// each other, each behind three more reads: mixed batch 226 -> 222 us, whole prompts
// 380 -> 372, the smallest calls 20.6 -> 17.4).
template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32, 4) chunk_merge_kernel(ChunkParams P, int n_cta) {
    pdl_wait();
    constexpr int R = kMergeRows<T>, U = kMergeParts<T>, E = D / 32;      // E: elements of a lane
    const int i = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ int s_slot[1024];
    __shared__ int4 s_at, s_unit;
    __shared__ int s_n;
    // the unit's parts: the one that begins it, then every CTA's that begins
    // inside it and has a step of it
    if (warp == 0) {
        const ChunkRecord x = P.records[min(i - 1 + lane, n_cta)];
        int4 c, m;
        c.x = __shfl_sync(0xffffffffu, x.at.x, 1);
        c.y = __shfl_sync(0xffffffffu, x.at.y, 1);
        c.z = __shfl_sync(0xffffffffu, x.at.z, 1);
        c.w = __shfl_sync(0xffffffffu, x.at.w, 1);
        m.x = __shfl_sync(0xffffffffu, x.unit.x, 1);
        m.y = __shfl_sync(0xffffffffu, x.unit.y, 1);
        m.z = __shfl_sync(0xffffffffu, x.unit.z, 1);
        const bool in = x.at.x == c.x && x.at.y == c.y && x.at.z == c.z && x.at.w > 0;
        unsigned inside = __ballot_sync(0xffffffffu, in);
        int n = 0;
        if (c.x < P.B && c.w > 0 && !(inside & 1u)) {    // (else no unit, or one that is cut earlier)
            n = 1;
            // CTA i - 1 + lane has steps of the unit up to where the next one begins
            const int next = __shfl_down_sync(0xffffffffu, x.at.w, 1);
            const bool on = (inside >> min(lane + 1, 31)) & 1u;
            const bool some = lane > 0 && lane < 31 && in && i - 1 + lane < n_cta && x.at.w < (on ? next : m.z);
            unsigned w = __ballot_sync(0xffffffffu, some);
            if (lane == 0) s_slot[0] = 2 * (i - 1) + 1;
            if (some) s_slot[n + __popc(w & ((1u << lane) - 1u))] = 2 * (i - 1 + lane);
            n += __popc(w);
            // (more than 30)
            for (int k0 = i + 30; (inside >> 31) && k0 < n_cta; k0 += 31) {
                const int k = min(k0 + lane, n_cta);
                const int4 y = P.records[k].at;
                const bool in2 = k < n_cta && y.x == c.x && y.y == c.y && y.z == c.z && y.w > 0;
                inside = __ballot_sync(0xffffffffu, in2);
                const int next2 = __shfl_down_sync(0xffffffffu, y.w, 1);
                const bool on2 = (inside >> min(lane + 1, 31)) & 1u;
                const bool some2 = lane < 31 && in2 && y.w < (on2 ? next2 : m.z);
                w = __ballot_sync(0xffffffffu, some2);
                if (some2) s_slot[n + __popc(w & ((1u << lane) - 1u))] = 2 * k;
                n += __popc(w);
            }
        }
        if (lane == 0) {
            s_n = n;
            s_at = c;
            s_unit = m;
        }
    }
    __syncthreads();
    const int n = s_n;
    if (n == 0) return;
    const int4 c = s_at, unit = s_unit;
    const ChunkReq r{unit.x, unit.y, 0};
    const bool paired = chunk_paired(P, r);
    const long long r0 = (long long)c.z * P.ru;
    for (int row0 = (blockIdx.y * kMergeWarps + warp) * R; row0 < P.ru; row0 += gridDim.y * kMergeWarps * R) {
        // each row's place in o (in heads), or -1; the second tile of a pair is the
        // other head
        long long to[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int row = row0 + q;
            const int x = paired && 2 * row >= P.ru ? 1 : 0;
            const long long p = paired ? row - x * (P.ru / 2) : r0 + row;
            const int h = paired ? 2 * c.y + x : c.y;
            to[q] = -1;
            if (row < P.ru && p < (long long)r.n * P.G && h < P.Hkv)
                to[q] = (r.first + p / P.G) * P.Hq + (long long)h * P.G + p % P.G;
        }
        float2 ml[R][U];
        float x[R][U][E];
        auto load = [&](int k0) {
#pragma unroll
            for (int v = 0; v < U; ++v)
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    ml[q][v] = make_float2(-INFINITY, kUnwritten);
                    if (k0 + v >= n || to[q] < 0) continue;
                    const size_t at = (size_t)s_slot[k0 + v] * P.ru + row0 + q;
                    ml[q][v] = P.part_ml[at];
                    const float *o = P.part_o + at * D + lane * E;
                    if constexpr (E == 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(o);
                        x[q][v][0] = f.x; x[q][v][1] = f.y; x[q][v][2] = f.z; x[q][v][3] = f.w;
                    } else {
                        const float2 f = *reinterpret_cast<const float2 *>(o);
                        x[q][v][0] = f.x; x[q][v][1] = f.y;
                    }
                }
        };
        load(0);
        // the largest maximum, a part a lane
        float top[R], l[R], acc[R][E];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            top[q] = -INFINITY;
            l[q] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[q][e] = 0.f;
        }
        if (n <= U) {
#pragma unroll
            for (int q = 0; q < R; ++q)
#pragma unroll
                for (int v = 0; v < U; ++v) top[q] = fmaxf(top[q], ml[q][v].x);
        } else {
            for (int k = lane; k < n; k += 32)
#pragma unroll
                for (int q = 0; q < R; ++q)
                    if (to[q] >= 0) top[q] = fmaxf(top[q], P.part_ml[(size_t)s_slot[k] * P.ru + row0 + q].x);
#pragma unroll
            for (int q = 0; q < R; ++q) top[q] = warp_max(top[q]);
        }
        for (int k0 = 0; k0 < n; k0 += U) {
            if (k0 > 0) load(k0);
#pragma unroll
            for (int v = 0; v < U; ++v)
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    // (one whose scores are all -inf has no weight and an output of 0, or
                    // NaN from a value; one of NaN has its maximum from the other scores,
                    // or none)
                    if (ml[q][v].y == kUnwritten) continue;
                    const float w = ml[q][v].x == -INFINITY ? 1.f : exp2f(ml[q][v].x - top[q]);
                    l[q] = fmaf(w, ml[q][v].y, l[q]);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[q][e] = fmaf(w, x[q][v][e], acc[q][e]);
                }
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (to[q] < 0) continue;
            T *o = static_cast<T *>(P.o) + to[q] * D + lane * E;
            const float inv = l[q] == 0.f ? 0.f : 1.f / l[q];
            if constexpr (sizeof(T) == 2) {
                uint32_t w[E / 2];
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(acc[q][2 * e] * inv, acc[q][2 * e + 1] * inv);
                    w[e] = *reinterpret_cast<const uint32_t *>(&h);
                }
                if constexpr (E == 4) *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint32_t *>(o) = w[0];
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) store_f(o + e, acc[q][e] * inv);
            }
            if (lane == 0)
                P.lse[to[q]] = l[q] == 0.f ? -INFINITY : l[q] != l[q] ? l[q] : (top[q] + log2f(l[q])) * kLn2;
        }
    }
}

// ------------------------------------------------------------- host side

ChunkPlan simt_plan() {
    // (a step is worth a CTA: the smallest calls 21 -> 17 us)
    return ChunkPlan{kRows, 0, kKeys, 2 * kKeys, 8, kKeys, kSimtPerSm * num_sms()};
}

ChunkPlan plan_of(const ChunkParams &P, int dtype, bool kv8) {
    return dtype == SPEC_BF16 ? chunk_tc_plan(P, kv8) : simt_plan();
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// What the workspace holds, in this order.
struct ChunkSpace {
    size_t o, ml, rec, bytes;
};
ChunkSpace space_of(const ChunkPlan &pl, int d) {
    ChunkSpace w{};
    const size_t rows = 2 * (size_t)pl.n_cta * pl.ru;
    w.ml = round256(rows * d * sizeof(float));
    w.rec = w.ml + round256(rows * sizeof(float2));
    w.bytes = w.rec + round256((size_t)(pl.n_cta + 1) * sizeof(ChunkRecord));
    return w;
}

// Checks a call's shape, and fills in what follows from it.
spec_status_t chunk_shape(const spec_chunk_desc *a, int n_kv_heads, int head_dim, int batch,
                          long long capacity, ChunkParams &P) {
    if (a->batch < 0 || a->n_tokens < 0 || a->n_q_heads <= 0 || a->n_kv_heads <= 0 ||
        a->n_q_heads % a->n_kv_heads != 0 || !(a->scale >= 0.f) || !(a->scale < INFINITY))
        return SPEC_ERR_INVALID_ARG;
    if (a->dtype != SPEC_BF16 && a->dtype != SPEC_F32) return SPEC_ERR_UNSUPPORTED;
    if (a->head_dim != 64 && a->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
    if (n_kv_heads != a->n_kv_heads || head_dim != a->head_dim || batch < a->batch || capacity <= 0)
        return SPEC_ERR_INVALID_ARG;
    if (capacity > (1ll << 30) || a->n_q_heads / a->n_kv_heads > 128) return SPEC_ERR_UNSUPPORTED;
    P.B = a->batch;
    P.n_tokens = a->n_tokens;
    P.Hq = a->n_q_heads;
    P.Hkv = a->n_kv_heads;
    P.G = P.Hq / P.Hkv;
    P.d = a->head_dim;
    P.capacity = (int)capacity;
    const float scale = a->scale > 0.f ? a->scale : 1.f / sqrtf((float)P.d);
    P.scale_log2 = scale * kLog2e;
    return SPEC_OK;
}

spec_status_t chunk_cache(const spec_chunk_desc *a, const spec_kv_desc *c, ChunkParams &P) {
    if (!a || !c) return SPEC_ERR_INVALID_ARG;
    P.paged = c->kind == SPEC_KV_PAGED;
    if (!P.paged && c->kind != SPEC_KV_CONTIGUOUS) return SPEC_ERR_INVALID_ARG;
    long long capacity = c->max_seq;
    if (P.paged) {
        if (c->n_pages <= 0 || c->page_size <= 0 || c->max_pages_per_seq <= 0) return SPEC_ERR_INVALID_ARG;
        if (c->page_size % 16 != 0) return SPEC_ERR_UNSUPPORTED;
        capacity = (long long)c->max_pages_per_seq * c->page_size;
        P.ps = c->page_size;
        P.max_pages = c->max_pages_per_seq;
        P.n_pages = c->n_pages;
    }
    const spec_status_t st = chunk_shape(a, c->n_kv_heads, c->head_dim, c->batch, capacity, P);
    if (st != SPEC_OK) return st;
    if (c->dtype != a->dtype) return SPEC_ERR_INVALID_ARG;
    // (tensor copies count rows of 64 elements, and heads, in 32 bits)
    const long long tiles = P.paged ? (long long)c->n_pages * P.Hkv * (P.d / 64) : (long long)c->batch * P.Hkv;
    if (tiles > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
    P.cache_heads = tiles;
    P.kc = c->k;
    P.vc = c->v;
    P.page_table = c->page_table;
    return SPEC_OK;
}

spec_status_t chunk_cache8(const spec_chunk_desc *a, const spec_kv8_desc *c, ChunkParams &P) {
    if (!a || !c) return SPEC_ERR_INVALID_ARG;
    spec_status_t st = check_kv8(c);
    if (st != SPEC_OK) return st;
    if (c->max_pages_per_seq <= 0) return SPEC_ERR_INVALID_ARG;
    st = chunk_shape(a, c->n_kv_heads, c->head_dim, c->batch, (long long)c->max_pages_per_seq * c->page_size, P);
    if (st != SPEC_OK) return st;
    P.paged = 1;
    P.ps = c->page_size;
    P.max_pages = c->max_pages_per_seq;
    P.n_pages = c->n_pages;
    P.kc = c->kv;
    P.vc = c->kv;
    P.scales = c->scales;
    P.page_table = c->page_table;
    return SPEC_OK;
}

// Fills in the plan; the whole call's cost has to be countable in 64 bits.
spec_status_t chunk_plan(const ChunkParams &P, int dtype, bool kv8, ChunkPlan &pl) {
    pl = plan_of(P, dtype, kv8);
    const double units = (double)P.n_tokens * P.G / pl.ru + P.B;
    if (units * P.Hkv > 2147483647.0 ||
        units * P.Hkv * P.G * ((double)pl.fixed_cost + P.capacity + pl.ru) > 1e18)
        return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

template <int kCache>
spec_status_t launch_simt(const ChunkParams &P, int n_cta, cudaStream_t s) {
    const bool wide = P.d == 128;
    const size_t smem = wide ? sizeof(ChunkSimtShared<128>) : sizeof(ChunkSimtShared<64>);
    auto *f = wide ? chunk_simt_kernel<128, kCache> : chunk_simt_kernel<64, kCache>;
    if (set_smem_limit(reinterpret_cast<const void *>(f), smem) != SPEC_OK) return SPEC_ERR_CUDA;
    return launch(f, dim3(n_cta), dim3(kSimtThreads), smem, s, P);
}

template <typename T, int D>
spec_status_t launch_merge(const ChunkParams &P, int n_cta, cudaStream_t s) {
    const dim3 grid(n_cta - 1, ceil_div(P.ru, kMergeRows<T> * kMergeWarps));
    return launch(chunk_merge_kernel<T, D>, grid, dim3(kMergeWarps * 32), 0, s, P, n_cta);
}

spec_status_t run_chunk(ChunkParams &P, int dtype, bool kv8, const void *q, long long stride_q,
                        const int32_t *seq_len, const int32_t *cu_new, void *o, float *lse,
                        void *workspace, size_t workspace_bytes, void *stream) {
    ChunkPlan pl;
    spec_status_t st = chunk_plan(P, dtype, kv8, pl);
    if (st != SPEC_OK) return st;
    const long long width = (long long)P.Hq * P.d;
    if (stride_q < width) return SPEC_ERR_INVALID_ARG;
    if (P.B == 0 || P.n_tokens == 0) return SPEC_OK;
    if (!q || !P.kc || !P.vc || !seq_len || !cu_new || !o || !lse || !workspace ||
        (P.paged && !P.page_table) || (kv8 && !P.scales))
        return SPEC_ERR_INVALID_ARG;
    const int es = dtype == SPEC_BF16 ? 2 : 4;
    if (!aligned16(q) || !aligned16(o) || !aligned16(P.kc) || !aligned16(P.vc) || stride_q * es % 16 != 0 ||
        reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return SPEC_ERR_INVALID_ARG;
    // (rows of q are read while others' results are written)
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(o);
    const uintptr_t q1 = q0 + (uintptr_t)((P.n_tokens - 1ll) * stride_q + width) * es;
    const uintptr_t o1 = o0 + (uintptr_t)(P.n_tokens * width) * es;
    if (q0 < o1 && o0 < q1) return SPEC_ERR_INVALID_ARG;
    const ChunkSpace w = space_of(pl, P.d);
    if (workspace_bytes < w.bytes) return SPEC_ERR_CAPACITY;
    P.q = q;
    P.stride_q = stride_q;
    P.seq_len = seq_len;
    P.cu_new = cu_new;
    P.o = o;
    P.lse = lse;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    P.part_o = reinterpret_cast<float *>(base + w.o);
    P.part_ml = reinterpret_cast<float2 *>(base + w.ml);
    P.records = reinterpret_cast<ChunkRecord *>(base + w.rec);
    P.ru = pl.ru;
    P.tu = pl.tu;
    P.ks = pl.ks;
    P.fixed_cost = pl.fixed_cost;
    P.pair_cost = pl.pair_cost;
    P.min_share = pl.min_share;
    P.wait = wait_limit();
    P.status = status_ptr();
    if (!P.status) return SPEC_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    if (dtype == SPEC_BF16) st = launch_chunk_tc(P, kv8, pl.n_cta, s);
    else st = kv8 ? launch_simt<kCache8>(P, pl.n_cta, s) : launch_simt<kCacheRows>(P, pl.n_cta, s);
    if (st != SPEC_OK) return st;
    if (dtype == SPEC_BF16)
        st = P.d == 128 ? launch_merge<__nv_bfloat16, 128>(P, pl.n_cta, s) : launch_merge<__nv_bfloat16, 64>(P, pl.n_cta, s);
    else
        st = P.d == 128 ? launch_merge<float, 128>(P, pl.n_cta, s) : launch_merge<float, 64>(P, pl.n_cta, s);
    if (st != SPEC_OK) return st;
    return launch_status();
}

spec_status_t size_of(const ChunkParams &P, int dtype, bool kv8, size_t *bytes) {
    ChunkPlan pl;
    const spec_status_t st = chunk_plan(P, dtype, kv8, pl);
    if (st != SPEC_OK) return st;
    *bytes = space_of(pl, P.d).bytes;
    return SPEC_OK;
}

}  // namespace
}  // namespace sv

extern "C" spec_status_t spec_chunk_attn_workspace_size(const spec_chunk_desc *desc,
                                                        const spec_kv_desc *cache, size_t *bytes) {
    using namespace sv;
    if (!bytes) return SPEC_ERR_INVALID_ARG;
    ChunkParams P{};
    const spec_status_t st = chunk_cache(desc, cache, P);
    return st == SPEC_OK ? size_of(P, desc->dtype, false, bytes) : st;
}

extern "C" spec_status_t spec_chunk_attn(const spec_chunk_desc *desc, const void *q, long long row_stride_q,
                                         const spec_kv_desc *cache, const int32_t *seq_len,
                                         const int32_t *cu_new, void *o, float *lse, void *workspace,
                                         size_t workspace_bytes, void *stream) {
    using namespace sv;
    ChunkParams P{};
    const spec_status_t st = chunk_cache(desc, cache, P);
    if (st != SPEC_OK) return st;
    return run_chunk(P, desc->dtype, false, q, row_stride_q, seq_len, cu_new, o, lse, workspace,
                     workspace_bytes, stream);
}

extern "C" spec_status_t spec_chunk_attn_kv8_workspace_size(const spec_chunk_desc *desc,
                                                            const spec_kv8_desc *cache, size_t *bytes) {
    using namespace sv;
    if (!bytes) return SPEC_ERR_INVALID_ARG;
    ChunkParams P{};
    const spec_status_t st = chunk_cache8(desc, cache, P);
    return st == SPEC_OK ? size_of(P, desc->dtype, true, bytes) : st;
}

extern "C" spec_status_t spec_chunk_attn_kv8(const spec_chunk_desc *desc, const void *q,
                                             long long row_stride_q, const spec_kv8_desc *cache,
                                             const int32_t *seq_len, const int32_t *cu_new, void *o,
                                             float *lse, void *workspace, size_t workspace_bytes,
                                             void *stream) {
    using namespace sv;
    ChunkParams P{};
    const spec_status_t st = chunk_cache8(desc, cache, P);
    if (st != SPEC_OK) return st;
    return run_chunk(P, desc->dtype, true, q, row_stride_q, seq_len, cu_new, o, lse, workspace,
                     workspace_bytes, stream);
}
