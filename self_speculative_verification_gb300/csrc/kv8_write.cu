// kv8_commit and kv8_append: new K/V rows into a cache of e4m3 codes with a
// power-of-two scale per (page, KV head).
//
// A block (one page, one head, keys or values) takes the scale 2^e with the
// smallest e for which its largest new |x| is at most 448 * 2^e, or keeps a
// larger one that it has; where a partly used block's scale grows, the rows
// it holds are rounded to the new one.  code = rn(x * 2^-e): the product is
// exact, so the code is the one rounding.
//
// One warp writes one block: its rows come in as 16-byte vectors (a bf16 row
// of 128 is half a warp's), the maximum is a bit-pattern maximum over the
// warp, and they leave as 8- or 4-byte groups of codes.  Prompts of 36 K
// tokens (8 heads of 128) take 41.5 us in bf16, 5.1 TB/s, and 74.6 in fp32, 4.7
// TB/s, bound by the search for runs ahead of the rows' reads and by the ALU
// (bf16: 51 %, unpacking and maxima); a commit is bound by its two launches and
// their dependent reads (8 rows of 16 requests, 32 heads: 6.7 us of GPU time;
// up to 24 fp32 rows of 64 requests, 8 heads: 11.8, bf16 9.0).
#include "commit_common.cuh"
#include "kv8.cuh"
#include "kv8_common.cuh"

namespace sv {
namespace {

// One 16-byte vector of new values: its floats, and the largest |x| of it as
// fp32 bits (which order as the values do; a non-finite one is the largest).
template <typename T> struct RowVec;
template <> struct RowVec<float> {
    static constexpr int N = 4;
    __device__ static void get(const uint4 &v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    // the running maximum m of |x|, and its value's bits
    __device__ static uint32_t amax(uint32_t m, const uint4 &v) {
        return max(max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu)), m);
    }
    __device__ static uint32_t bits(uint32_t m) { return m; }
};
template <> struct RowVec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void get(const uint4 &v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    // the running maxima m of the even and the odd values' |x|, and the larger one's bits
    __device__ static uint32_t amax(uint32_t m, const uint4 &v) {
        m = max2(max2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), m);
        return max2(max2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu), m);
    }
    __device__ static uint32_t bits(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
};

// N values as codes, x * r; `odd`: among non-finite ones, which become NaN.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *dst, float (&x)[N], float r, bool odd) {
    if (odd) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fabsf(x[i]) < INFINITY ? x[i] : __uint_as_float(0x7fffffffu);
    }
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        w[i] = e4m3x2(x[4 * i] * r, x[4 * i + 1] * r) | (e4m3x2(x[4 * i + 2] * r, x[4 * i + 3] * r) << 16);
    if constexpr (N == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(dst) = w[0];
}

// One warp: rows `n` of one block, at offsets first .. first + n - 1 of its
// page; row(i) is the i-th row's first element or, unless kDense, nullptr
// (not written).
// Sixteen rows pass through registers at a time; a block of more is read
// twice, the second time from L1 / L2 (at most 128 KB).
template <typename T, int D, bool kDense, typename Row>
__device__ void write_block(uint8_t *tile, float *scale, int x, int first, int n, const Row &row) {
    constexpr int N = RowVec<T>::N, LPR = D / N;     // lanes per row
    constexpr int RPI = 32 / LPR, kHeld = 16 / RPI;  // rows per round, rounds held
    const int lane = threadIdx.x & 31, sub = lane / LPR, col = (lane % LPR) * N;
    uint4 held[kHeld];
    uint32_t have = 0;       // rounds of `held` that hold a row
    auto fetch = [&](int i0) {
        have = 0;
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            const int i = i0 + u * RPI + sub;
            held[u] = make_uint4(0u, 0u, 0u, 0u);
            if (i >= n) continue;
            const T *p = row(i);
            if (!kDense && !p) continue;
            have |= 1u << u;
            held[u] = *reinterpret_cast<const uint4 *>(p + col);
        }
    };
    constexpr uint32_t kInf = 0x7f800000u;
    const int last = (n - 1) / 16 * 16;
    uint32_t amax = 0, any = 0;
    for (int i0 = 0; i0 <= last; i0 += 16) {
        fetch(i0);
        any |= have;
#pragma unroll
        for (int u = 0; u < kHeld; ++u) amax = RowVec<T>::amax(amax, held[u]);
    }
    if (!kDense && !__any_sync(0xffffffffu, any != 0u)) return;
    amax = __reduce_max_sync(0xffffffffu, RowVec<T>::bits(amax));
    const bool bad = amax >= kInf;
    if (bad) {               // the largest finite one, value by value
        amax = 0;
        for (int i0 = 0; i0 <= last; i0 += 16) {
            if (last > 0) fetch(i0);
#pragma unroll
            for (int u = 0; u < kHeld; ++u) {
                float v[N];
                RowVec<T>::get(held[u], v);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const uint32_t a = __float_as_uint(v[j]) & 0x7fffffffu;
                    if (a < kInf) amax = max(amax, a);
                }
            }
        }
        amax = __reduce_max_sync(0xffffffffu, amax);
    }
    const float need = exp2_int(kv8_exponent(__uint_as_float(amax)));
    // a partly used block keeps the larger scale (the present one as readers
    // take it, for its codes mean that); NaN stays NaN
    const float was = first > 0 ? kv8_read_scale(*scale) : 0.f;
    const bool was_nan = was != was;
    const float s = fmaxf(was, need);                // (fmaxf drops a NaN)
    if (first > 0 && !was_nan && s > was) {
        const float r = was / s;
        constexpr int VPR = D / 16;                  // 16-code vectors a row
        for (int i = lane; i < first * VPR; i += 32) {
            uint4 *p = reinterpret_cast<uint4 *>(tile + kv8_row(i / VPR, x, D) + (i % VPR) * 16);
            uint4 v = *p;
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 a = from_e4m3x2(w[j] & 0xffffu), b = from_e4m3x2(w[j] >> 16);
                w[j] = e4m3x2(a.x * r, a.y * r) | (e4m3x2(b.x * r, b.y * r) << 16);
            }
            *p = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    const float r = 1.f / s;                         // exact for a power of two
    for (int i0 = last; i0 >= 0; i0 -= 16) {         // (the last rows are still held)
        if (i0 != last) fetch(i0);
        // (from a multiple of eight on, the rows' places are constants apart)
        const bool even = ((first + i0) & 7) == 0;
        uint8_t *at = tile + kv8_row(first + i0, x, D) + sub * D + col;
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            if (kDense ? i0 + u * RPI + sub >= n : !((have >> u) & 1u)) continue;
            float v[N];
            RowVec<T>::get(held[u], v);
            store_codes<N>(even ? at + kv8_row(u * RPI, 0, D)
                                : tile + kv8_row(first + i0 + u * RPI + sub, x, D) + col, v, r, bad);
        }
    }
    __syncwarp();
    if (lane == 0) *scale = (bad || was_nan) ? __uint_as_float(0x7fffffffu) : s;
}

constexpr int kWriteWarps = 8;

struct Commit8Params {
    CommitParams c;
    uint8_t *kv;
    float *scales;
    const void *kb, *vb;
};

// CTA (request b, eight of its (page, head, K / V) blocks).
template <typename T, int D>
__global__ void __launch_bounds__(kWriteWarps * 32) kv8_commit_kernel(Commit8Params Q, int units,
                                                                      int ctas_per_req) {
    pdl_wait();
    const CommitParams &P = Q.c;
    const int b = blockIdx.x / ctas_per_req, part = blockIdx.x % ctas_per_req;
    int before = 0, total = 0;
    page_prefix(P, b, &before, &total);
    const int head = *P.free_head;
    if (head < 0 || (long long)head + total > P.n_free) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_status(P.status, SPEC_DEV_CAPACITY);
        return;
    }
    int bits = 0;
    const int a = effective_acc(P, b, &bits);
    if (bits && part == 0 && threadIdx.x == 0) raise_status(P.status, bits);
    if (a == 0) return;
    const int S = P.seq_len[b], ps = P.page_size;
    const int used = pages_for(S, ps);
    const int u = part * kWriteWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int j = S / ps + u / (2 * P.Hkv);          // the page, within the request
    if (u >= units || j * ps >= S + a) return;
    const int h = (u >> 1) % P.Hkv, x = u & 1;
    const int t0 = max(S, j * ps), t1 = min(S + a, (j + 1) * ps);
    const int page = j < used ? P.page_table[(size_t)b * P.max_pages + j]
                              : P.free_pages[head + before + (j - used)];
    if (page < 0 || page >= P.n_pages) {
        if (lane == 0) raise_status(P.status, SPEC_DEV_BAD_PAGE);
        return;
    }
    const T *src = static_cast<const T *>(x ? Q.vb : Q.kb) + ((size_t)b * P.Hkv + h) * P.R * D;
    const int32_t *path = P.path + (size_t)b * P.path_cap + (t0 - S);
    bool bad_row = false;
    auto row = [&](int i) -> const T * {
        const int r = path[i];
        if (r < 0 || r >= P.R) {
            bad_row = true;
            return nullptr;
        }
        return src + (size_t)r * D;
    };
    write_block<T, D, false>(Q.kv + kv8_block(page, h, P.Hkv, ps, D),
                      Q.scales + ((size_t)page * P.Hkv + h) * 2 + x, x, t0 - j * ps, t1 - t0, row);
    if (bad_row) raise_status(P.status, SPEC_DEV_BAD_INDEX);
}

struct Append8Params {
    uint8_t *kv;
    float *scales;
    const void *k, *v;
    long long stride_k, stride_v;
    const int64_t *slots;
    int n, Hkv, ps, n_pages;
    int hpc;                 // heads per CTA
    int *status;
};

constexpr int kAppendTokens = 64;

// CTA (64 packed tokens, hpc heads): the runs that begin among its tokens (a
// run: consecutive tokens in consecutive slots of one page, tokens that are
// not written in between), one warp per (run, head, K / V).
template <typename T, int D>
__global__ void __launch_bounds__(kWriteWarps * 32, sizeof(T) == 2 ? 4 : 2)
kv8_append_kernel(Append8Params P) {
    pdl_wait();
    __shared__ int s_start[kAppendTokens], s_len[kAppendTokens];    // len < 0: with gaps
    __shared__ int s_page[kAppendTokens], s_first[kAppendTokens];
    __shared__ int s_runs[kAppendTokens / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int base = blockIdx.x * kAppendTokens, h0 = blockIdx.y * P.hpc;
    const long long n_slots = (long long)P.n_pages * P.ps;
    if (threadIdx.x < kAppendTokens) {
        const int i = base + threadIdx.x;
        bool start = false;
        long long s = -1;
        if (i < P.n) {
            s = P.slots[i];
            if (s >= n_slots) {
                if (blockIdx.y == 0) raise_status(P.status, SPEC_DEV_BAD_PAGE);
            } else if (s >= 0) {
                // it goes on with a run when the nearest written token before
                // it lies as far back as that one's slot
                int m = 1;
                const int off = (int)(s % P.ps);
                while (m <= off && m <= i && P.slots[i - m] < 0) ++m;
                start = m > off || m > i || P.slots[i - m] != s - m;
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, start);
        if (lane == 0) s_runs[warp] = __popc(m);
        if (start) {
            const int at = warp * 32 + __popc(m & ((1u << lane) - 1u));
            s_start[at] = i;
            s_page[at] = (int)(s / P.ps);
            s_first[at] = (int)(s % P.ps);
        }
    }
    __syncthreads();
    const int n0 = s_runs[0], n_runs = n0 + s_runs[1];
    // the runs' lengths, one warp each
    for (int r = warp; r < n_runs; r += kWriteWarps) {
        const int at = r < n0 ? r : 32 + r - n0, i = s_start[at], first = s_first[at];
        const long long slot = (long long)s_page[at] * P.ps + first;
        int n = 0;
        bool gaps = false;
        for (int k = 0; first + k < P.ps; k += 32) {
            const bool in = first + k + lane < P.ps && k + lane < P.n - i;
            const long long s = in ? P.slots[i + k + lane] : 0;
            const unsigned end = __ballot_sync(0xffffffffu, !in || (s >= 0 && s != slot + k + lane));
            const int here = end ? __ffs(end) - 1 : 32;
            gaps = gaps || __any_sync(0xffffffffu, lane < here && s < 0);
            n = k + here;
            if (end) break;
        }
        if (lane == 0) s_len[at] = gaps ? -n : n;
    }
    __syncthreads();
    const int heads = min(P.hpc, P.Hkv - h0);
    for (int u = warp; u < n_runs * heads * 2; u += kWriteWarps) {
        const int r = u / (heads * 2), h = h0 + (u >> 1) % heads, x = u & 1;
        const int at = r < n0 ? r : 32 + r - n0;
        const int i = s_start[at], page = s_page[at], first = s_first[at], len = s_len[at];
        const T *src = x ? static_cast<const T *>(P.v) + (size_t)i * P.stride_v + (size_t)h * D
                         : static_cast<const T *>(P.k) + (size_t)i * P.stride_k + (size_t)h * D;
        const long long stride = x ? P.stride_v : P.stride_k;
        uint8_t *tile = P.kv + kv8_block(page, h, P.Hkv, P.ps, D);
        float *scale = P.scales + ((size_t)page * P.Hkv + h) * 2 + x;
        if (len > 0)
            write_block<T, D, true>(tile, scale, x, first, len, [&](int t) { return src + (size_t)t * stride; });
        else
            write_block<T, D, false>(tile, scale, x, first, -len, [&](int t) -> const T * {
                return P.slots[i + t] < 0 ? nullptr : src + (size_t)t * stride;
            });
    }
}

}  // namespace

spec_status_t check_kv8(const spec_kv8_desc *c) {
    if (c->n_kv_heads <= 0 || c->n_pages <= 0 || c->page_size <= 0) return SPEC_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
    if (c->page_size % 16 != 0 || c->page_size > kKv8MaxPage) return SPEC_ERR_UNSUPPORTED;
    if ((long long)c->n_pages * c->n_kv_heads > 2147483647ll) return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

}  // namespace sv

extern "C" spec_status_t kv8_commit(const spec_kv8_desc *cache, int dtype, int batch, int n_rows,
                                    const void *kb, const void *vb, int path_cap,
                                    const int32_t *path, const int32_t *acc_len, int32_t *seq_len,
                                    const int32_t *free_pages, int n_free, int32_t *free_head,
                                    void *stream) {
    using namespace sv;
    if (!cache || batch < 0 || n_rows <= 0 || path_cap < 0 || n_free < 0) return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
    spec_status_t st = check_kv8(cache);
    if (st != SPEC_OK) return st;
    if (cache->batch < batch || cache->max_pages_per_seq <= 0) return SPEC_ERR_INVALID_ARG;
    if ((long long)cache->max_pages_per_seq * cache->page_size > (1ll << 30))
        return SPEC_ERR_UNSUPPORTED;
    if (batch == 0) return SPEC_OK;
    if (!kb || !vb || !path || !acc_len || !seq_len || !cache->kv || !cache->scales ||
        !cache->page_table || !free_pages || !free_head)
        return SPEC_ERR_INVALID_ARG;
    if (!aligned16(kb) || !aligned16(vb) || !aligned16(cache->kv)) return SPEC_ERR_INVALID_ARG;
    // the pages that path_cap rows can touch
    const long long pages = ((long long)path_cap + cache->page_size - 2) / cache->page_size + 1;
    const long long units = pages * cache->n_kv_heads * 2;
    const long long ctas = (units + kWriteWarps - 1) / kWriteWarps;
    if (units > 2147483647ll || ctas * batch > 2147483647ll) return SPEC_ERR_UNSUPPORTED;
    Commit8Params Q{};
    Q.kv = static_cast<uint8_t *>(cache->kv);
    Q.scales = cache->scales;
    Q.kb = kb;
    Q.vb = vb;
    CommitParams &P = Q.c;
    P.page_table = cache->page_table;
    P.path = path;
    P.acc_len = acc_len;
    P.seq_len = seq_len;
    P.free_pages = free_pages;
    P.free_head = free_head;
    P.n_free = n_free;
    P.B = batch;
    P.Hkv = cache->n_kv_heads;
    P.R = n_rows;
    P.path_cap = path_cap;
    P.paged = 1;
    P.page_size = cache->page_size;
    P.max_pages = cache->max_pages_per_seq;
    P.n_pages = cache->n_pages;
    P.capacity = cache->max_pages_per_seq * cache->page_size;
    P.status = status_ptr();
    if (!P.status) return SPEC_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    const dim3 grid((unsigned)(ctas * batch)), block(kWriteWarps * 32);
    const int u = (int)units, c = (int)ctas;
    if (dtype == SPEC_BF16)
        st = cache->head_dim == 128
                 ? launch(kv8_commit_kernel<__nv_bfloat16, 128>, grid, block, 0, s, Q, u, c)
                 : launch(kv8_commit_kernel<__nv_bfloat16, 64>, grid, block, 0, s, Q, u, c);
    else
        st = cache->head_dim == 128 ? launch(kv8_commit_kernel<float, 128>, grid, block, 0, s, Q, u, c)
                                    : launch(kv8_commit_kernel<float, 64>, grid, block, 0, s, Q, u, c);
    if (st != SPEC_OK) return st;
    if (launch(kv_commit_finalize_kernel, dim3(1), dim3(256), 0, s, P) != SPEC_OK)
        return SPEC_ERR_CUDA;
    return launch_status();
}

extern "C" spec_status_t kv8_append(const spec_kv8_desc *cache, int dtype, int n_tokens,
                                    const void *k, long long row_stride_k, const void *v,
                                    long long row_stride_v, const int64_t *slot_map, void *stream) {
    using namespace sv;
    if (!cache || n_tokens < 0) return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
    spec_status_t st = check_kv8(cache);
    if (st != SPEC_OK) return st;
    const long long width = (long long)cache->n_kv_heads * cache->head_dim;
    if (row_stride_k < width || row_stride_v < width) return SPEC_ERR_INVALID_ARG;
    if (n_tokens == 0) return SPEC_OK;
    if (!k || !v || !slot_map || !cache->kv || !cache->scales) return SPEC_ERR_INVALID_ARG;
    const int es = dtype == SPEC_BF16 ? 2 : 4;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache->kv) || row_stride_k * es % 16 != 0 ||
        row_stride_v * es % 16 != 0)
        return SPEC_ERR_INVALID_ARG;
    Append8Params P{};
    P.kv = static_cast<uint8_t *>(cache->kv);
    P.scales = cache->scales;
    P.k = k;
    P.v = v;
    P.stride_k = row_stride_k;
    P.stride_v = row_stride_v;
    P.slots = slot_map;
    P.n = n_tokens;
    P.Hkv = cache->n_kv_heads;
    P.ps = cache->page_size;
    P.n_pages = cache->n_pages;
    P.status = status_ptr();
    if (!P.status) return SPEC_ERR_CUDA;
    // heads split over CTAs until every SM has eight: each finds the runs anew
    // (sixteen: 54 us instead of 48 on 36 K tokens of 8 heads)
    const int gx = (int)ceil_div_ll(n_tokens, kAppendTokens);
    int split = 1;
    while (split < P.Hkv && split < 32768 && (long long)gx * split < 8ll * num_sms()) split *= 2;
    P.hpc = ceil_div(P.Hkv, split);
    const int gy = ceil_div(P.Hkv, P.hpc);
    if (gy > 65535) return SPEC_ERR_UNSUPPORTED;
    cudaStream_t s = as_stream(stream);
    const dim3 grid(gx, gy), block(kWriteWarps * 32);
    if (dtype == SPEC_BF16)
        st = cache->head_dim == 128 ? launch(kv8_append_kernel<__nv_bfloat16, 128>, grid, block, 0, s, P)
                                    : launch(kv8_append_kernel<__nv_bfloat16, 64>, grid, block, 0, s, P);
    else
        st = cache->head_dim == 128 ? launch(kv8_append_kernel<float, 128>, grid, block, 0, s, P)
                                    : launch(kv8_append_kernel<float, 64>, grid, block, 0, s, P);
    if (st != SPEC_OK) return st;
    return launch_status();
}
