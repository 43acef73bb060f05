// spec_verify_attn_kv8: masked attention of the speculative rows over
// (committed prefix in 8 bits || soft prompt || block).
//
// O = softmax(q K^T * scale + mask) V and LSE = ln sum exp(q k * scale) with
// K and V of the prefix read as code * scale(page, head).
//
// The smallest calls (two requests of 128-200 tokens) take 10 us, two
// launches whose reads wait for each other (page, codes and scale, sums).
//
// This file holds the host planning, the CUDA-core kernel (fp32 inputs, whose
// products the tensor cores' 8- and 16-bit operands cannot hold) and its
// combine kernel.
#include <math.h>

#include <type_traits>

#include "attn_kv8.cuh"
#include "kv8_common.cuh"
#include "ptx_sm103.cuh"

namespace sv {
namespace {

constexpr int kCols = 32;    // columns per tile

enum { kColPrefix = 0, kColSoft = 1, kColBlock = 2 };

// Shared memory of a CTA of RB packed rows.
template <int D, int RB>
struct SimtShared {
    // (row pitches: eight rows' 16-byte reads, or eight columns' P, spread over the banks)
    alignas(16) float q[RB][D + 4];
    alignas(16) float k[kCols][D + 4];
    alignas(16) float v[kCols][D];
    alignas(16) float p[kCols][RB + 4];    // a row's -0: the column is not seen
    float alpha[RB];                       // what the rows' O is scaled by
    uint32_t vis[RB][SPEC_MAX_ROWS / 32];
    uint32_t any[SPEC_MAX_ROWS / 32];      // block columns that one of the rows sees
    uint8_t flags[RB];
};

// CTAs that share an SM (fewer registers a thread than the compiler takes
// when not asked: single token 130 -> 113 us, 300 rows a head 226 -> 153 us).
constexpr int simt_ctas(int d, int rb) { return d == 128 ? (rb == 32 ? 4 : 5) : (rb == 32 ? 5 : 8); }

// CTA (split, KV head x row block, request): a running softmax over its
// columns, 32 at a time through shared memory.  Scores: a thread takes RB / 8
// rows and every 16th column, two dimensions to a packed fma; O: RB / 4
// (d = 128) or RB / 8 (d = 64) rows and four head dimensions.  With 32 rows and
// d = 128 a warp's shared-memory wavefront feeds four (scores) and five (O)
// fused multiply-adds a thread, about what the SM does in its time; 28 rows
// over 30 K tokens, 16 heads, take 762 us, 27 TFLOP/s (64 columns at a time,
// half of the CTAs an SM: 15 % slower).
template <int D, int RB>
__global__ void __launch_bounds__(128, simt_ctas(D, RB))
attn_kv8_simt_kernel(Kv8Params Q) {
    pdl_wait();
    const AttnParams &P = Q.a;
    extern __shared__ __align__(16) uint8_t smem[];
    auto &sh = *reinterpret_cast<SimtShared<D, RB> *>(smem);
    constexpr int RT = RB / 8, CT = kCols / 16;          // scores: rows and columns a thread
    constexpr int DG = D / 4, RP = RB * DG / 128;        // O: groups of dimensions, rows a thread

    const int split = blockIdx.x;
    const int h = blockIdx.y / P.n_rb, rb = blockIdx.y % P.n_rb;
    const int b = blockIdx.z;
    const int tid = threadIdx.x;
    const int rg = tid / 16, cg = tid % 16;              // scores: rows rg RT .., columns cg + 16 c
    const int pg = tid / DG, dg = tid % DG;              // O: rows pg RP .., dimensions 4 dg ..

    const int S = clamp_seq(P, b, split == 0 && blockIdx.y == 0 && tid == 0);
    const int nsp = n_splits_of(P, S);
    if (split >= nsp) return;
    const int t0 = split * P.chunk, t1 = min(S, t0 + P.chunk);
    const bool last = split == nsp - 1;
    const int row0 = rb * RB;

    const float *q = static_cast<const float *>(P.q);
    for (int i = tid; i < RB * DG; i += 128) {
        const int p = row0 + i / DG, c = i % DG * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < P.M) {
            const int r = p / P.G, hq = h * P.G + p % P.G;
            x = *reinterpret_cast<const float4 *>(q + (((size_t)b * P.R + r) * P.Hq + hq) * D + c);
            x.x *= P.scale_log2;
            x.y *= P.scale_log2;
            x.z *= P.scale_log2;
            x.w *= P.scale_log2;
        }
        *reinterpret_cast<float4 *>(&sh.q[i / DG][c]) = x;
    }
    if (last) {
        if (tid < SPEC_MAX_ROWS / 32) sh.any[tid] = 0u;
        __syncthreads();
        for (int i = tid; i < RB * P.W; i += 128) {
            const int pr = i / P.W, w = i % P.W, p = row0 + pr;
            const uint32_t x = p < P.M ? P.vis[((size_t)b * P.R + p / P.G) * P.W + w] : 0u;
            sh.vis[pr][w] = x;
            if (x) atomicOr(&sh.any[w], x);
        }
        __syncthreads();
    }
    if (tid < RB) {
        const int p = row0 + tid;
        sh.flags[tid] = p < P.M ? P.row_flags[(size_t)b * P.R + p / P.G] : 0;
    }

    float m[RT], l[RT];                                  // (l: of this thread's columns)
    uint64_t acc[RP][2];                                 // dimensions 0, 1 and 2, 3
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < RP; ++i) acc[i][0] = acc[i][1] = 0ull;

    const uint8_t *kv = static_cast<const uint8_t *>(P.kc);
    const int n_prefix_tiles = ceil_div(t1 - t0, kCols);
    const int n_soft_tiles = last ? ceil_div(P.n_soft, kCols) : 0;
    const int n_block_tiles = last ? ceil_div(P.R, kCols) : 0;
    const int n_tiles = n_prefix_tiles + n_soft_tiles + n_block_tiles;
    bool bad_page = false;

    // a prefix tile's K and V, 16 codes a vector, and their scales, in
    // registers a tile ahead
    constexpr int VPR = D / 16;
    constexpr int kPer = 2 * kCols * VPR / 128;
    uint4 w[kPer];
    float sc[kPer];
    auto fetch = [&](int tile) {
        if (tile >= n_prefix_tiles) return;
        const int base = t0 + tile * kCols, ncols = min(kCols, t1 - base);
        int page[kPer];
#pragma unroll
        for (int it = 0; it < kPer; ++it) {
            const int j = ((tid + it * 128) / VPR) % kCols, t = base + j;
            page[it] = j < ncols ? P.page_table[(size_t)b * P.max_pages + t / P.page_size] : 0;
        }
#pragma unroll
        for (int it = 0; it < kPer; ++it) {
            const int i = tid + it * 128, x = i / (kCols * VPR), j = (i / VPR) % kCols, c = i % VPR;
            w[it] = make_uint4(0u, 0u, 0u, 0u);
            sc[it] = 0.f;
            if (j >= ncols) continue;
            if (page[it] < 0 || page[it] >= P.n_pages) {
                bad_page = true;
                continue;
            }
            w[it] = *reinterpret_cast<const uint4 *>(
                kv + kv8_block(page[it], h, P.Hkv, P.page_size, D) +
                kv8_row((base + j) % P.page_size, x, D) + c * 16);
            sc[it] = Q.scales[((size_t)page[it] * P.Hkv + h) * 2 + x];
        }
    };
    fetch(0);

    for (int tile = 0; tile < n_tiles; ++tile) {
        int kind, base, ncols;
        if (tile < n_prefix_tiles) {
            kind = kColPrefix;
            base = t0 + tile * kCols;
            ncols = min(kCols, t1 - base);
        } else if (tile < n_prefix_tiles + n_soft_tiles) {
            kind = kColSoft;
            base = (tile - n_prefix_tiles) * kCols;
            ncols = min(kCols, P.n_soft - base);
        } else {
            kind = kColBlock;
            base = (tile - n_prefix_tiles - n_soft_tiles) * kCols;
            ncols = min(kCols, P.R - base);
            static_assert(kCols == 32, "a tile's columns are a word of vis");
            if (sh.any[base / 32] == 0u) continue;
        }
        __syncthreads();             // previous tile consumed (and q, vis, flags ready)
        if (kind == kColPrefix) {
#pragma unroll
            for (int it = 0; it < kPer; ++it) {
                const int i = tid + it * 128, x = i / (kCols * VPR), j = (i / VPR) % kCols, c = i % VPR;
                float *dst = x ? &sh.v[j][c * 16] : &sh.k[j][c * 16];
                // its four groups from the (c / 2)-th on, so that a row's eight
                // threads write to different banks
                const bool r1 = (c >> 1) & 1, r2 = (c >> 2) & 1;
                const uint32_t a0 = r1 ? w[it].y : w[it].x, a1 = r1 ? w[it].z : w[it].y;
                const uint32_t a2 = r1 ? w[it].w : w[it].z, a3 = r1 ? w[it].x : w[it].w;
                const uint32_t u[4] = {r2 ? a2 : a0, r2 ? a3 : a1, r2 ? a0 : a2, r2 ? a1 : a3};
                const float f = kv8_read_scale(sc[it]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 lo = from_e4m3x2(u[e] & 0xffffu), hi = from_e4m3x2(u[e] >> 16);
                    *reinterpret_cast<float4 *>(dst + 4 * ((e + (c >> 1)) & 3)) =
                        make_float4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
                }
            }
        } else {
            const size_t first = kind == kColSoft ? (size_t)h * P.n_soft
                                                  : ((size_t)b * P.Hkv + h) * P.R;
            const float *kp = static_cast<const float *>(kind == kColSoft ? P.soft_k : P.kb) + (first + base) * D;
            const float *vp = static_cast<const float *>(kind == kColSoft ? P.soft_v : P.vb) + (first + base) * D;
            for (int i = tid; i < kCols * DG; i += 128) {
                const int j = i / DG, c = i % DG * 4;
                const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4 *>(&sh.k[j][c]) =
                    j < ncols ? *reinterpret_cast<const float4 *>(kp + 4 * i) : z;
                *reinterpret_cast<float4 *>(&sh.v[j][c]) =
                    j < ncols ? *reinterpret_cast<const float4 *>(vp + 4 * i) : z;
            }
        }
        __syncthreads();
        fetch(tile + 1);

        // (sums of the even and of the odd dimensions, side by side)
        uint64_t s2[RT][CT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int c = 0; c < CT; ++c) s2[i][c] = 0ull;
#pragma unroll 4
        for (int k = 0; k < D; k += 4) {
            ulonglong2 kk[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) kk[c] = *reinterpret_cast<const ulonglong2 *>(&sh.k[cg + 16 * c][k]);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const ulonglong2 qq = *reinterpret_cast<const ulonglong2 *>(&sh.q[rg * RT + i][k]);
#pragma unroll
                for (int c = 0; c < CT; ++c) s2[i][c] = fma2(qq.y, kk[c].y, fma2(qq.x, kk[c].x, s2[i][c]));
            }
        }
        float s[RT][CT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                float x, y;
                unpair(s2[i][c], x, y);
                s[i][c] = x + y;
            }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int pr = rg * RT + i;
            const uint8_t fl = sh.flags[pr];
            unsigned seen = 0;
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int j = cg + 16 * c;
                bool visible = false;
                if (j < ncols && (fl & SPEC_ROW_VALID)) {
                    if (kind == kColPrefix) visible = true;
                    else if (kind == kColSoft) visible = (fl & SPEC_ROW_SEES_SOFT) != 0;
                    else visible = (sh.vis[pr][(base + j) >> 5] >> ((base + j) & 31)) & 1u;
                }
                seen |= (unsigned)visible << c;
                if (visible) top = fmaxf(top, s[i][c]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float mn = fmaxf(m[i], top);
            const float mr = mn == -INFINITY ? 0.f : mn;    // (nothing but masked, -inf or NaN scores)
            const float alpha = exp2f(m[i] - mr);
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const float p = (seen >> c) & 1u ? exp2f(s[i][c] - mr) : -0.f;
                sum += p;
                s[i][c] = p;
            }
            l[i] = fmaf(l[i], alpha, sum);
            m[i] = mn;
            if (cg == 0) sh.alpha[pr] = alpha;
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            float *dst = &sh.p[cg + 16 * c][rg * RT];
            if constexpr (RT == 4) *reinterpret_cast<float4 *>(dst) = make_float4(s[0][c], s[1][c], s[2][c], s[3][c]);
            else dst[0] = s[0][c];
        }
        __syncthreads();

#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const float f = sh.alpha[pg * RP + i];
            const uint64_t ff = pair(f, f), z = pair(-0.f, -0.f);
            acc[i][0] = fma2(acc[i][0], ff, z);
            acc[i][1] = fma2(acc[i][1], ff, z);
        }
        // O.  Outside the prefix, columns that a row does not see are left out:
        // their values may be anything.
        auto add = [&](auto all) {
            constexpr bool kAll = decltype(all)::value;
#pragma unroll 4
            for (int j = 0; j < ncols; ++j) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&sh.v[j][4 * dg]);
                float pj[RP];
                if constexpr (RP % 4 == 0) {
#pragma unroll
                    for (int i = 0; i < RP; i += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(&sh.p[j][pg * RP + i]);
                        pj[i] = x.x;
                        pj[i + 1] = x.y;
                        pj[i + 2] = x.z;
                        pj[i + 3] = x.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < RP; ++i) pj[i] = sh.p[j][pg * RP + i];
                }
#pragma unroll
                for (int i = 0; i < RP; ++i) {
                    if (!kAll && __float_as_int(pj[i]) == (int)0x80000000u) continue;
                    const uint64_t pp = pair(pj[i], pj[i]);
                    acc[i][0] = fma2(pp, v.x, acc[i][0]);
                    acc[i][1] = fma2(pp, v.y, acc[i][1]);
                }
            }
        };
        if (kind == kColPrefix) add(std::true_type{});
        else add(std::false_type{});
    }
    if (bad_page) raise_status(P.status, SPEC_DEV_BAD_PAGE);

#pragma unroll
    for (int i = 0; i < RP; ++i) {
        const int pr = pg * RP + i, p = row0 + pr;
        if (p >= P.M) continue;
        // (a row that is not valid sees nothing, but its O may have met a NaN)
        const bool valid = (sh.flags[pr] & SPEC_ROW_VALID) != 0;
        *reinterpret_cast<ulonglong2 *>(P.part_o + part_index(P, b, h, split, p) * D + 4 * dg) =
            valid ? make_ulonglong2(acc[i][0], acc[i][1]) : make_ulonglong2(0ull, 0ull);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int p = row0 + rg * RT + i;
        float sum = l[i];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (cg == 0 && p < P.M)
            *reinterpret_cast<float2 *>(P.part_ml + part_index(P, b, h, split, p) * 2) = make_float2(m[i], sum);
    }
}

// Merge the splits of every packed row, one warp each.
template <int D>
__global__ void __launch_bounds__(128) attn_kv8_combine_kernel(AttnParams P) {
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int p = blockIdx.x * 4 + warp;
    const int h = blockIdx.y, b = blockIdx.z;
    if (p >= P.M) return;
    const int nsp = n_splits_of(P, clamp_seq(P, b, false));
    float mstar = -INFINITY;
    for (int s = 0; s < nsp; ++s) mstar = fmaxf(mstar, P.part_ml[part_index(P, b, h, s, p) * 2]);
    const float mr = mstar == -INFINITY ? 0.f : mstar;
    float out[D / 32], L = 0.f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) out[j] = 0.f;
    for (int s = 0; s < nsp; ++s) {
        const size_t idx = part_index(P, b, h, s, p);
        // (a split without visible columns has sums 0, or NaN that must stay)
        const float ms = P.part_ml[idx * 2];
        const float w = ms == -INFINITY ? 1.f : exp2f(ms - mr);
        L = fmaf(w, P.part_ml[idx * 2 + 1], L);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) out[j] = fmaf(w, P.part_o[idx * D + lane + 32 * j], out[j]);
    }
    const int r = p / P.G, hq = h * P.G + p % P.G;
    float *o = static_cast<float *>(P.o) + (((size_t)b * P.R + r) * P.Hq + hq) * D;
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) store_f(o + lane + 32 * j, out[j] * inv);
    if (lane == 0)
        P.lse[((size_t)b * P.Hq + hq) * P.R + r] = L == 0.f ? -INFINITY : (mr + log2f(L)) * kLn2;
}

// ---------------------------------------------------------------- planning

struct Plan8 {
    Kv8Params Q;
    size_t off_ml;      // byte offset of part_ml in the workspace
    size_t ws_bytes;
    bool use_tc;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

spec_status_t make_plan8(const spec_attn_desc *a, const spec_kv8_desc *c, Plan8 *out) {
    if (!a || !c) return SPEC_ERR_INVALID_ARG;
    if (a->batch < 0 || a->n_rows <= 0 || a->n_q_heads <= 0 || a->n_kv_heads <= 0 ||
        a->n_q_heads % a->n_kv_heads != 0 || a->n_soft < 0 || a->split_tokens < 0)
        return SPEC_ERR_INVALID_ARG;
    if (a->n_rows > SPEC_MAX_ROWS || a->n_soft > 64) return SPEC_ERR_UNSUPPORTED;
    if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
    const spec_status_t st = check_kv8(c);
    if (st != SPEC_OK) return st;
    if (c->n_kv_heads != a->n_kv_heads || c->head_dim != a->head_dim || c->batch < a->batch ||
        c->max_pages_per_seq <= 0 || a->split_tokens % 64 != 0)
        return SPEC_ERR_INVALID_ARG;
    if (a->batch > 65535 || (long long)c->max_pages_per_seq * c->page_size > (1ll << 30))
        return SPEC_ERR_UNSUPPORTED;
    Plan8 plan{};
    AttnParams &P = plan.Q.a;
    P.B = a->batch;
    P.R = a->n_rows;
    P.Hq = a->n_q_heads;
    P.Hkv = a->n_kv_heads;
    P.G = a->n_q_heads / a->n_kv_heads;
    P.d = a->head_dim;
    if ((long long)P.R * P.G > (1 << 20)) return SPEC_ERR_UNSUPPORTED;
    P.M = P.R * P.G;
    P.W = ceil_div(P.R, 32);
    P.n_soft = a->n_soft;
    P.paged = 1;
    P.page_size = c->page_size;
    P.max_pages = c->max_pages_per_seq;
    P.n_pages = c->n_pages;
    P.capacity = c->max_pages_per_seq * c->page_size;
    const float scale = a->scale != 0.f ? a->scale : 1.f / sqrtf((float)a->head_dim);
    P.scale_log2 = scale * kLog2e;
    P.rb_rows = P.M <= 8 ? 8 : 32;
    P.n_rb = ceil_div(P.M, P.rb_rows);
    if ((long long)P.Hkv * P.n_rb > 65535) return SPEC_ERR_UNSUPPORTED;
    if (a->split_tokens > 0) {
        // (no longer than the longest prefix, rounded up to a tile)
        const int most = (P.capacity + 63) / 64 * 64;
        P.chunk = a->split_tokens < most ? a->split_tokens : most;
    } else {
        // about eight CTAs per SM for prefixes at half the capacity
        const long long units = (long long)P.B * P.Hkv * P.n_rb;
        const long long half = P.capacity / 2 > 64 ? P.capacity / 2 : 64;
        const long long target = 8ll * num_sms();
        long long chunk = (units * half + target - 1) / target;
        chunk = (chunk + 63) / 64 * 64;
        if (chunk < 64) chunk = 64;
        if (chunk > 16384) chunk = 16384;
        P.chunk = (int)chunk;
    }
    P.max_splits = ceil_div(P.capacity, P.chunk);
    plan.use_tc = a->dtype == SPEC_BF16;
    if (plan.use_tc) {
        if (!kv8_tc_supported(P)) return SPEC_ERR_UNSUPPORTED;
        plan.ws_bytes = kv8_tc_workspace_bytes(P);
        *out = plan;
        return SPEC_OK;
    }
    const size_t nrow = (size_t)P.B * P.Hkv * P.max_splits * P.M;
    plan.off_ml = align256(nrow * P.d * sizeof(float));
    plan.ws_bytes = plan.off_ml + align256(nrow * 2 * sizeof(float));
    *out = plan;
    return SPEC_OK;
}

template <int D, int RB>
spec_status_t launch_simt8(const Kv8Params &Q, cudaStream_t s) {
    const AttnParams &P = Q.a;
    constexpr size_t kSmem = sizeof(SimtShared<D, RB>);
    spec_status_t st = set_smem_limit((const void *)attn_kv8_simt_kernel<D, RB>, kSmem);
    if (st != SPEC_OK) return st;
    st = launch(attn_kv8_simt_kernel<D, RB>, dim3(P.max_splits, P.Hkv * P.n_rb, P.B), dim3(128), kSmem, s, Q);
    if (st != SPEC_OK) return st;
    st = launch(attn_kv8_combine_kernel<D>, dim3(ceil_div(P.M, 4), P.Hkv, P.B), dim3(128), 0, s, P);
    return st != SPEC_OK ? st : launch_status();
}

}  // namespace
}  // namespace sv

extern "C" spec_status_t spec_verify_attn_kv8_workspace_size(const spec_attn_desc *attn,
                                                             const spec_kv8_desc *cache,
                                                             size_t *bytes) {
    if (!bytes) return SPEC_ERR_INVALID_ARG;
    sv::Plan8 plan;
    const spec_status_t st = sv::make_plan8(attn, cache, &plan);
    if (st != SPEC_OK) return st;
    *bytes = plan.ws_bytes;
    return SPEC_OK;
}

extern "C" spec_status_t spec_verify_attn_kv8(const spec_attn_desc *attn, const void *q,
                                              const spec_kv8_desc *cache, const void *kb,
                                              const void *vb, const void *soft_k,
                                              const void *soft_v, const int32_t *seq_len,
                                              const uint32_t *vis, const uint8_t *row_flags,
                                              void *o, float *lse, void *workspace,
                                              size_t workspace_bytes, void *stream) {
    using namespace sv;
    Plan8 plan;
    const spec_status_t st = make_plan8(attn, cache, &plan);
    if (st != SPEC_OK) return st;
    AttnParams &P = plan.Q.a;
    if (P.B == 0) return SPEC_OK;
    if (!q || !kb || !vb || !seq_len || !vis || !row_flags || !o || !lse || !workspace ||
        !cache->kv || !cache->scales || !cache->page_table ||
        (P.n_soft > 0 && (!soft_k || !soft_v)))
        return SPEC_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(kb) || !aligned16(vb) || !aligned16(o) ||
        !aligned16(cache->kv) || (P.n_soft > 0 && (!aligned16(soft_k) || !aligned16(soft_v))) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
        return SPEC_ERR_INVALID_ARG;
    if (workspace_bytes < plan.ws_bytes) return SPEC_ERR_CAPACITY;
    P.status = status_ptr();
    if (!P.status) return SPEC_ERR_CUDA;
    P.q = q;
    P.kc = cache->kv;
    P.page_table = cache->page_table;
    P.kb = kb;
    P.vb = vb;
    P.soft_k = soft_k;
    P.soft_v = soft_v;
    P.seq_len = seq_len;
    P.vis = vis;
    P.row_flags = row_flags;
    P.o = o;
    P.lse = lse;
    P.part_o = static_cast<float *>(workspace);
    P.part_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.off_ml);
    plan.Q.scales = cache->scales;
    cudaStream_t s = as_stream(stream);
    if (plan.use_tc) return launch_attn_kv8_tc(plan.Q, s);
    if (P.rb_rows == 8) return P.d == 128 ? launch_simt8<128, 8>(plan.Q, s) : launch_simt8<64, 8>(plan.Q, s);
    return P.d == 128 ? launch_simt8<128, 32>(plan.Q, s) : launch_simt8<64, 32>(plan.Q, s);
}
