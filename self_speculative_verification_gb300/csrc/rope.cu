// spec_rope: rotary positions of queries and keys.
//
// Pair i of a head's first rot_dim elements, (x, y), becomes a (x cos t - y sin
// t, y cos t + x sin t) with t = position * freqs[i].  The angle is taken in
// turns: freqs[i] / 2 pi is held as a 64-bit binary fraction, so position *
// fraction modulo 2^64 is the angle modulo a turn without any rounding but the
// fraction's own (2^-52 of it, for 2 pi and the division, or 2^-64), at any
// position; the remainder becomes a float, and sin and cos of pi times it are
// taken in fp32.
//
// Bound by memory: 33 K tokens of 40 heads of 128 (bf16, halves; 680 MB) take 118
// us, 5.8 TB/s, 85 % of a copy's rate; 6 K tokens of 10 heads of 64 in fp32 (31 MB)
// 7.0; a block of 128 rows of 64 heads 3.4, its launch and three dependent reads.
#include <math.h>

#include "common.cuh"
#include "kv8.cuh"
#include "ptx_sm103.cuh"

namespace sv {
namespace {

constexpr int kRopeTokens = 4;       // most tokens of a CTA
constexpr int kMaxPairs = 128;       // rot_dim <= 256

struct RopeParams {
    const void *q, *k;
    void *q_out, *k_out;
    long long sq, sqo, sk, sko;      // elements between two tokens' rows
    const int32_t *positions, *seq_len, *cu_new;
    int n, B, Hq, H, d, rot;         // H: query and key heads
    int tpc;                         // tokens of a CTA (of the gridDim.y that share their heads)
    int items;                       // a head's parts, a thread each
    bool keep_q, keep_k;             // in place: what is not rotated stays
    float attention;
    int *status;
    uint64_t turn[kMaxPairs];        // 2^64 turns a position, by pair
};

enum { kPairs = 0, kHalves = 1, kHalvesScalar = 2 };

// Threads of a CTA: at least a head's parts (by vectors 64 at most, by elements
// 255).  Small CTAs of few tokens: 128 threads and 4 tokens take 118 us for 33 K
// tokens of 40 heads of 128 (680 MB, 5.8 TB/s), 256 and 16 take 127.
__host__ __device__ constexpr int rope_threads(int layout) { return layout == kHalvesScalar ? 256 : 128; }

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

// Pairs of one part, and where pair i's cosine and sine lie in shared memory: the
// k-th pairs of all parts side by side, so that a row's threads, a part each, read
// one run.
template <typename T, int kLayout>
__host__ __device__ constexpr int part_pairs() {
    return kLayout == kPairs ? kVec<T> / 2 : kLayout == kHalves ? kVec<T> : 1;
}

// The position of packed token i, which no request before b0 holds; false for a
// row that is left as it is.
__device__ __forceinline__ bool rope_position(const RopeParams &P, int i, int b0, long long *pos) {
    if (P.positions) {
        *pos = P.positions[i];
        return *pos >= 0;
    }
    int b = b0;
    while (b < P.B && __ldg(P.cu_new + b + 1) <= i) ++b;
    if (b >= P.B) return false;
    const int first = __ldg(P.cu_new + b), S = __ldg(P.seq_len + b);
    if (i < first) return false;
    if (S < 0) {
        raise_status(P.status, SPEC_DEV_SEQ_OVERFLOW);
        return false;
    }
    *pos = (long long)S + (i - first);
    return true;
}

template <typename T>
__device__ __forceinline__ void unpack_vec(const uint4 &v, float (&x)[kVec<T>]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            x[i] = __uint_as_float(w[i]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void store_vec(T *p, const float (&x)[kVec<T>]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        else w[i] = __float_as_uint(x[i]);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void rotate(float &x, float &y, float2 cs) {
    const float a = x * cs.x - y * cs.y, b = y * cs.x + x * cs.y;
    x = a;
    y = b;
}

// Part `it` of one head: src -> dst.
//   kPairs         vector it of the head, pairs (2i, 2i + 1)
//   kHalvesScalar  elements it and it + rot / 2 of the rotated part; behind them
//                  the rest, an element a part
// (kHalves, where rot / 2 is a multiple of a vector: the same by vectors, in the
// kernel.)
template <typename T, int kLayout>
__device__ __forceinline__ void rope_item(const RopeParams &P, const T *src, T *dst, int it,
                                          const float2 *cs, int parts, bool keep) {
    constexpr int V = kVec<T>;
    const int half = P.rot / 2;
    if constexpr (kLayout == kPairs) {
        const int c = it * V;
        if (c >= P.rot && keep) return;
        const uint4 v = *reinterpret_cast<const uint4 *>(src + c);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < V; e += 2) {                 // (what does not turn keeps its bits)
            if (c + e >= P.rot) continue;
            float2 x;
            if constexpr (sizeof(T) == 2) x = make_float2(__uint_as_float(w[e / 2] << 16), __uint_as_float(w[e / 2] & 0xffff0000u));
            else x = make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]));
            rotate(x.x, x.y, cs[e / 2 * parts + it]);
            if constexpr (sizeof(T) == 2) {
                w[e / 2] = pack_bf16(x.x, x.y);
            } else {
                w[e] = __float_as_uint(x.x);
                w[e + 1] = __float_as_uint(x.y);
            }
        }
        *reinterpret_cast<uint4 *>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        if (it < half) {
            float x = load_f(src + it), y = load_f(src + it + half);
            rotate(x, y, cs[it]);
            store_f(dst + it, x);
            store_f(dst + it + half, y);
        } else if (!keep) {
            dst[it + half] = src[it + half];
        }
    }
}

// (32 registers a thread, so that an SM is full)
template <typename T, int kLayout>
__global__ void __launch_bounds__(rope_threads(kLayout), 2048 / rope_threads(kLayout)) rope_kernel(const __grid_constant__ RopeParams P) {
    constexpr int kThreads = rope_threads(kLayout);
    pdl_wait();
    __shared__ long long s_pos[kRopeTokens];
    __shared__ bool s_in[kRopeTokens];
    constexpr int kPer = part_pairs<T, kLayout>();
    __shared__ float2 s_cs[kRopeTokens][kMaxPairs + kPer];
    const int tid = threadIdx.x, base = blockIdx.x * P.tpc, nt = min(P.tpc, P.n - base);
    // the requests that end before this CTA's tokens, counted by all threads at once
    int b0 = 0;
    if (!P.positions)
        for (int b = 0; b < P.B; b += kThreads)
            b0 += __syncthreads_count(b + tid < P.B && __ldg(P.cu_new + b + tid + 1) <= base);
    if (tid < nt) {
        long long pos = 0;
        s_in[tid] = rope_position(P, base + tid, b0, &pos);
        s_pos[tid] = pos;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && !P.positions) {
        bool bad = tid == 0 && P.cu_new[0] < 0;
        for (int b = tid; b < P.B; b += kThreads)
            bad = bad || P.cu_new[b + 1] < P.cu_new[b] || P.cu_new[b + 1] > P.n;
        if (bad) raise_status(P.status, SPEC_DEV_BAD_INDEX);
    }
    __syncthreads();
    const int half = P.rot / 2, parts = (half + kPer - 1) / kPer;    // parts that turn
    for (int f = tid; f < nt * half; f += kThreads) {
        const int t = f / half, i = f - t * half;
        const float x = __ll2float_rn((long long)((uint64_t)s_pos[t] * P.turn[i])) * 0x1p-63f;
        float s, c;
        sincospif(x, &s, &c);
        s_cs[t][i % kPer * parts + i / kPer] = make_float2(c * P.attention, s * P.attention);
    }
    __syncthreads();
    const int slots = kThreads / P.items;            // rows at a time
    const int slot = tid / P.items, it = tid - slot * P.items;
    if (slot >= slots) return;
    const int row0 = blockIdx.y * slots + slot, stride = slots * gridDim.y;
    auto find = [&](int row, const T *&src, T *&dst, const float2 *&cs, bool &keep) -> bool {
        const int t = row / P.H, h = row - t * P.H;
        if (!s_in[t]) return false;
        const long long i = base + t;
        const bool key = h >= P.Hq;
        const int hh = key ? h - P.Hq : h;
        src = static_cast<const T *>(key ? P.k : P.q) + i * (key ? P.sk : P.sq) + (long long)hh * P.d;
        dst = static_cast<T *>(key ? P.k_out : P.q_out) + i * (key ? P.sko : P.sqo) + (long long)hh * P.d;
        cs = s_cs[t];
        keep = key ? P.keep_k : P.keep_q;
        return true;
    };
    if constexpr (kLayout == kHalves) {
        constexpr int V = kVec<T>;
        const int half = P.rot / 2, c = it * V;
        const bool turns = c < half;
        const int second = turns ? c + half : half + c;  // (behind: the vector that is copied)
        for (int row = row0; row < nt * P.H; row += stride) {
            const T *src;
            T *dst;
            const float2 *cs;
            bool keep;
            if (!find(row, src, dst, cs, keep) || (!turns && keep)) continue;
            const uint4 b = *reinterpret_cast<const uint4 *>(src + second);
            if (!turns) {
                *reinterpret_cast<uint4 *>(dst + second) = b;
                continue;
            }
            float x[V], y[V];
            unpack_vec<T>(*reinterpret_cast<const uint4 *>(src + c), x);
            unpack_vec<T>(b, y);
#pragma unroll
            for (int e = 0; e < V; ++e) rotate(x[e], y[e], cs[e * parts + it]);
            store_vec(dst + c, x);
            store_vec(dst + second, y);
        }
    } else {
#pragma unroll 2
        for (int row = row0; row < nt * P.H; row += stride) {
            const T *src;
            T *dst;
            const float2 *cs;
            bool keep;
            if (find(row, src, dst, cs, keep)) rope_item<T, kLayout>(P, src, dst, it, cs, parts, keep);
        }
    }
}

// Whether n rows of wa bytes from a on, sa bytes apart, may meet n rows of wb
// bytes from b on, sb bytes apart (with unlike strides: whether the spans do).
bool rows_meet(const void *pa, long long sa, long long wa, const void *pb, long long sb, long long wb, int n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(pa), b = reinterpret_cast<uintptr_t>(pb);
    if (a >= b + (uintptr_t)((n - 1) * sb + wb) || b >= a + (uintptr_t)((n - 1) * sa + wa)) return false;
    if (sa != sb) return true;
    const long long off = (long long)((b - a) % (uintptr_t)sa);          // (b below a: wraps)
    const long long at = b >= a ? off : (long long)((sa - (long long)((a - b) % (uintptr_t)sa)) % sa);
    return at < wa || at + wb > sa;
}

}  // namespace
}  // namespace sv

extern "C" spec_status_t spec_rope_freqs(int rot_dim, double base, int scaling, double factor,
                                         double trained_len, double low, double high, double *freqs) {
    using namespace sv;
    if (rot_dim <= 0 || rot_dim % 2 != 0 || !freqs || !(base > 0.0) || !(base < INFINITY))
        return SPEC_ERR_INVALID_ARG;
    if (rot_dim > 2 * kMaxPairs) return SPEC_ERR_UNSUPPORTED;
    if (scaling != SPEC_ROPE_PLAIN && scaling != SPEC_ROPE_LINEAR && scaling != SPEC_ROPE_RAMP)
        return SPEC_ERR_UNSUPPORTED;
    if (scaling != SPEC_ROPE_PLAIN && (!(factor > 0.0) || !(factor < INFINITY))) return SPEC_ERR_INVALID_ARG;
    if (scaling == SPEC_ROPE_RAMP && (!(trained_len > 0.0) || !(trained_len < INFINITY) || !(low < high) ||
                                      !(low > -INFINITY) || !(high < INFINITY)))
        return SPEC_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot_dim);
        double w = scaling == SPEC_ROPE_PLAIN ? 1.0 : 0.0;               // share of the plain one
        if (scaling == SPEC_ROPE_RAMP) {
            w = (trained_len * f / (2.0 * M_PI) - low) / (high - low);
            w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
        }
        freqs[i] = w == 1.0 ? f : f * (w + (1.0 - w) / factor);
    }
    return SPEC_OK;
}

extern "C" spec_status_t spec_rope(const spec_rope_desc *desc, const double *freqs, const void *q,
                                   long long row_stride_q, void *q_out, long long row_stride_q_out,
                                   const void *k, long long row_stride_k, void *k_out,
                                   long long row_stride_k_out, const int32_t *positions, int batch,
                                   const int32_t *seq_len, const int32_t *cu_new, void *stream) {
    using namespace sv;
    if (!desc || !freqs) return SPEC_ERR_INVALID_ARG;
    const int n = desc->n_tokens, Hq = desc->n_q_heads, Hk = desc->n_k_heads, d = desc->head_dim;
    const int rot = desc->rot_dim;
    if (n < 0 || Hq < 0 || Hk < 0 || d <= 0 || rot <= 0 || rot > d || rot % 2 != 0 || batch < 0 ||
        !(fabsf(desc->attention) < INFINITY))
        return SPEC_ERR_INVALID_ARG;
    if (desc->dtype != SPEC_BF16 && desc->dtype != SPEC_F32) return SPEC_ERR_UNSUPPORTED;
    if (desc->layout != SPEC_ROPE_PAIRS && desc->layout != SPEC_ROPE_HALVES) return SPEC_ERR_UNSUPPORTED;
    if (d % 8 != 0 || d > 256 || (long long)Hq + Hk > 65536) return SPEC_ERR_UNSUPPORTED;
    for (int i = 0; i < rot / 2; ++i)
        if (!(fabs(freqs[i]) < INFINITY)) return SPEC_ERR_INVALID_ARG;
    const long long wq = (long long)Hq * d, wk = (long long)Hk * d;
    if (row_stride_q < wq || row_stride_q_out < wq || row_stride_k < wk || row_stride_k_out < wk)
        return SPEC_ERR_INVALID_ARG;
    if (n == 0 || Hq + Hk == 0) return SPEC_OK;
    // (the stride of a single row is not used; of more, all rows' bytes are counted
    // in 64 bits)
    for (long long *s : {&row_stride_q, &row_stride_q_out})
        if (n == 1) *s = wq;
        else if (Hq && *s > (1ll << 59) / n) return SPEC_ERR_INVALID_ARG;
    for (long long *s : {&row_stride_k, &row_stride_k_out})
        if (n == 1) *s = wk;
        else if (Hk && *s > (1ll << 59) / n) return SPEC_ERR_INVALID_ARG;
    if ((Hq && (!q || !q_out)) || (Hk && (!k || !k_out))) return SPEC_ERR_INVALID_ARG;
    if (!positions && (!seq_len || !cu_new || batch == 0)) return SPEC_ERR_INVALID_ARG;
    const int es = desc->dtype == SPEC_BF16 ? 2 : 4, per = 16 / es;
    if (Hq && (!aligned16(q) || !aligned16(q_out) || row_stride_q % per != 0 || row_stride_q_out % per != 0))
        return SPEC_ERR_INVALID_ARG;
    if (Hk && (!aligned16(k) || !aligned16(k_out) || row_stride_k % per != 0 || row_stride_k_out % per != 0))
        return SPEC_ERR_INVALID_ARG;
    // what a call writes meets nothing else that it reads or writes, but for
    // rows in place
    struct Rows { const void *p; long long s, w; };
    const Rows in[2] = {{q, row_stride_q * es, wq * es}, {k, row_stride_k * es, wk * es}};
    const Rows out[2] = {{q_out, row_stride_q_out * es, wq * es}, {k_out, row_stride_k_out * es, wk * es}};
    bool keep[2] = {false, false};
    for (int x = 0; x < 2; ++x) {
        if (in[x].w == 0) continue;
        keep[x] = in[x].p == out[x].p && in[x].s == out[x].s;
        for (int y = 0; y < 2; ++y) {
            if (in[y].w == 0) continue;
            if (!(x == y && keep[x]) && rows_meet(out[x].p, out[x].s, out[x].w, in[y].p, in[y].s, in[y].w, n))
                return SPEC_ERR_INVALID_ARG;
            if (y > x && rows_meet(out[x].p, out[x].s, out[x].w, out[y].p, out[y].s, out[y].w, n))
                return SPEC_ERR_INVALID_ARG;
        }
    }
    RopeParams P{};
    P.q = q;
    P.k = k;
    P.q_out = q_out;
    P.k_out = k_out;
    P.sq = row_stride_q;
    P.sqo = row_stride_q_out;
    P.sk = row_stride_k;
    P.sko = row_stride_k_out;
    P.positions = positions;
    P.seq_len = seq_len;
    P.cu_new = cu_new;
    P.n = n;
    P.B = batch;
    P.Hq = Hq;
    P.H = Hq + Hk;
    P.d = d;
    P.rot = rot;
    P.keep_q = keep[0];
    P.keep_k = keep[1];
    P.attention = desc->attention != 0.f ? desc->attention : 1.f;
    for (int i = 0; i < rot / 2; ++i) {
        // (of the magnitude, which loses nothing; a negative one is its complement)
        const double t = fabs(freqs[i]) / (2.0 * M_PI);
        const uint64_t u = (uint64_t)((t - floor(t)) * 0x1p64);
        P.turn[i] = freqs[i] < 0.0 ? 0u - u : u;
    }
    P.status = status_ptr();
    if (!P.status) return SPEC_ERR_CUDA;
    // tokens of a CTA: up to 4, fewer while the GPU has room for more CTAs
    P.tpc = kRopeTokens;
    while (P.tpc > 1 && ceil_div(n, P.tpc) < 4 * num_sms()) P.tpc /= 2;
    const int layout = desc->layout == SPEC_ROPE_PAIRS ? kPairs : rot / 2 % per == 0 ? kHalves : kHalvesScalar;
    P.items = layout == kPairs ? d / per : layout == kHalves ? rot / 2 / per + (d - rot) / per : d - rot / 2;
    // and CTAs that share a token's heads while a thread has more than one part of
    // them (128 rows of 64 heads: 6.5 -> 3.4 us)
    const int at_once = rope_threads(layout) / P.items;
    int share = 1;
    while (ceil_div(n, P.tpc) * share < 4 * num_sms() && ceil_div(P.H, share) > at_once) share *= 2;
    const dim3 grid((unsigned)ceil_div(n, P.tpc), (unsigned)share), block(rope_threads(layout));
    cudaStream_t s = as_stream(stream);
    spec_status_t st;
#define SV_ROPE(T)                                                                        \
    (layout == kPairs    ? launch(rope_kernel<T, kPairs>, grid, block, 0, s, P)           \
     : layout == kHalves ? launch(rope_kernel<T, kHalves>, grid, block, 0, s, P)          \
                         : launch(rope_kernel<T, kHalvesScalar>, grid, block, 0, s, P))
    if (desc->dtype == SPEC_BF16) st = SV_ROPE(__nv_bfloat16);
    else st = SV_ROPE(float);
#undef SV_ROPE
    if (st != SPEC_OK) return SPEC_ERR_CUDA;
    return launch_status();
}
