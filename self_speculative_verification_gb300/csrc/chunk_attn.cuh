// Work decomposition shared by the chunk-attention kernels: attention of a
// packed batch of new tokens over a KV cache that already holds them.
//
// Packed rows: for KV head h, the G = Hq / Hkv query heads h*G .. h*G+G-1 of
// new token i of a request are its packed rows i*G .. i*G+G-1; row p sees the
// cache's tokens 0 .. S + p / G (S: tokens held before), itself the last one.
//
// Unit: `ru` consecutive packed rows of one (request, KV head), cut along the
// keys into steps of `ks` tokens up to the last one its last row sees.  Units
// are numbered request by request, head by head, rows ascending.  On the
// tensor cores a unit is two query tiles; a request whose rows all fit one has
// units of two heads instead, a tile each.
//
// Ranges: every unit has a cost in closed form -- a fixed one, and the tokens
// its last row sees -- so the sum over any number of units is closed too, and
// a CTA finds its equal share of the whole call's cost from one scan of the
// requests and two searches, whatever the lengths.  A share that begins or
// ends inside a unit begins or ends at a step of it: the CTA then writes the
// rows' running maximum, sum and unnormalised output (fp32) to one of its two
// slots, and the merging kernel puts the parts together in order.
#pragma once

#include "common.cuh"
#include "kv8.cuh"

namespace sv {

// Where a CTA's share begins (ChunkPos; a request past the last: nowhere), and of
// that unit its request's first packed token, new tokens, and its steps.
struct ChunkRecord {
    int4 at, unit;
};

struct ChunkParams {
    const void *q;
    long long stride_q;      // elements between two tokens' rows of q
    const void *kc, *vc;     // cache; 8 bits: kc the tiles
    const float *scales;     // 8 bits: [n_pages][Hkv][2]
    const int32_t *page_table, *seq_len, *cu_new;
    void *o;
    float *lse;
    float *part_o;           // [2 n_cta][ru][d]
    float2 *part_ml;         // [2 n_cta][ru] (log2 domain)
    ChunkRecord *records;    // [n_cta + 1]
    int *status;
    int B, n_tokens, Hq, Hkv, G, d;
    int paged, ps, max_pages, n_pages;
    int capacity;            // tokens per request
    long long cache_heads;   // contiguous: requests * heads of the cache
    int ru, ks;              // rows of a unit, keys of a step
    int tu;                  // tokens of a unit (two tiles: ru / G), or 0: units end inside a token's rows
    int fixed_cost;          // of a unit, in keys
    int pair_cost;           // of a key behind a pair of heads, in eighths
    int min_share;           // least cost (keys) worth a CTA
    float scale_log2;        // softmax scale * log2(e)
    long long wait;          // limit of every pipeline wait, in SM cycles
};

// The tensor-core path: rows and CTAs of a call, its kernel's launch.
struct ChunkPlan {
    int ru, tu, ks, fixed_cost, pair_cost, min_share, n_cta;
};
ChunkPlan chunk_tc_plan(const ChunkParams &P, bool kv8);
spec_status_t launch_chunk_tc(const ChunkParams &P, bool kv8, int n_cta, cudaStream_t s);

namespace {

// The sum of a part whose row has no output in part_o.
constexpr float kUnwritten = -1.f;

// A request's new tokens: n of them, packed from row `first` on, S held
// before; n = 0 for one without any, or with lengths out of range.
struct ChunkReq {
    int first, n, S;
};

__device__ __forceinline__ ChunkReq chunk_request(const ChunkParams &P, int b, int *bits) {
    ChunkReq r{__ldg(P.cu_new + b), 0, __ldg(P.seq_len + b)};
    const int end = __ldg(P.cu_new + b + 1);
    if (r.first < 0 || end < r.first || end > P.n_tokens) {
        if (bits) *bits |= SPEC_DEV_BAD_INDEX;
    } else if (end == r.first) {
    } else if (r.S < 0 || r.S > P.capacity - (end - r.first)) {
        if (bits) *bits |= SPEC_DEV_SEQ_OVERFLOW;
    } else {
        r.n = end - r.first;
    }
    return r;
}

// Whether the request's units are pairs of heads, and how many heads or pairs.
__device__ __forceinline__ bool chunk_paired(const ChunkParams &P, const ChunkReq &r) { return 2 * r.n <= P.tu; }
__device__ __forceinline__ int chunk_heads(const ChunkParams &P, const ChunkReq &r) {
    return chunk_paired(P, r) ? (P.Hkv + 1) / 2 : P.Hkv;
}

__device__ __forceinline__ int chunk_units(const ChunkParams &P, const ChunkReq &r) {
    if (P.tu) return (int)(((uint32_t)r.n + P.tu - 1) / (uint32_t)P.tu);
    return (int)(((long long)r.n * P.G + P.ru - 1) / P.ru);
}

// Cost of a head's (a pair's) first j units (in keys * G): unit i costs G (fixed
// + S) + (i + 1) ru; for a pair, whose steps are each head's own, the S counts
// pair_cost / 8 times.
__device__ __forceinline__ long long chunk_cost(const ChunkParams &P, const ChunkReq &r, long long j) {
    const long long S = chunk_paired(P, r) ? (long long)r.S * P.pair_cost >> 3 : r.S;
    return j * P.G * (P.fixed_cost + S) + P.ru * (j * (j + 1) / 2);
}

// A place in the call's work: unit j of head h of request b, from step s on.
struct ChunkPos {
    int b, h, j, s;
};

// Steps of unit j: up to the last token its last row sees.
__device__ __forceinline__ int chunk_steps(const ChunkParams &P, const ChunkReq &r, int j) {
    int last;                                            // that token, within the new ones
    if (P.tu) {
        last = (int)min((long long)r.n, (long long)(j + 1) * P.tu) - 1;
    } else {
        const long long rows = min((long long)r.n * P.G, (long long)(j + 1) * P.ru);
        last = (int)((rows - 1) / P.G);
    }
    return (int)((uint32_t)(r.S + last + P.ks) / (uint32_t)P.ks);   // (S + last + 1 tokens)
}

// Where cost `at` of request b's lies.  Quotients and the root are taken in
// fp32 and put right by comparisons: 64-bit divisions and fp64 cost the start
// of a call microseconds.  (The same place comes out for the CTA that ends
// there and for the one that begins.)
__device__ __forceinline__ ChunkPos chunk_find(const ChunkParams &P, int b, const ChunkReq &r,
                                               long long at) {
    const int nu = chunk_units(P, r);
    const long long head = chunk_cost(P, r, nu);
    ChunkPos p{b, 0, 0, 0};
    const int heads = chunk_heads(P, r);
    p.h = min((int)(__ll2float_rn(at) / __ll2float_rn(head)), heads - 1);
    while (p.h > 0 && p.h * head > at) --p.h;
    while (p.h < heads - 1 && (p.h + 1) * head <= at) ++p.h;
    at -= p.h * head;
    // the last j with cost(j) <= at: cost(j) = (ru j^2 + (2 a + ru) j) / 2
    const float a = __ll2float_rn(chunk_cost(P, r, 1)) - (float)P.ru, ru = (float)P.ru;
    const float half = a / ru + 0.5f, x = __ll2float_rn(at) / ru;
    p.j = min((int)(2.f * x / (half + sqrtf(half * half + 2.f * x))), nu - 1);
    while (p.j > 0 && chunk_cost(P, r, p.j) > at) --p.j;
    while (p.j < nu - 1 && chunk_cost(P, r, p.j + 1) <= at) ++p.j;
    const long long f = at - chunk_cost(P, r, p.j), w = chunk_cost(P, r, p.j + 1) - chunk_cost(P, r, p.j);
    const int steps = chunk_steps(P, r, p.j);
    p.s = min((int)(__ll2float_rn(f) / __ll2float_rn(w) * (float)steps), steps - 1);
    return p;
}

struct ChunkShare {
    long long warp_sum[32];
    ChunkPos begin, end;     // begin.b == B: nothing to do
};

// The share of CTA blockIdx.x, by all T threads of the CTA; records where it
// begins.  Ends with a barrier.
template <int T>
__device__ void chunk_share(const ChunkParams &P, ChunkShare &sh) {
    static_assert(T % 32 == 0 && T <= 1024, "threads");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (P.B + T - 1) / T, b0 = min(P.B, tid * per), b1 = min(P.B, b0 + per);
    if (tid == 0) sh.begin = sh.end = ChunkPos{P.B, 0, 0, 0};
    long long mine = 0;
    int bits = 0;
    ChunkReq r{0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        r = chunk_request(P, b, &bits);
        mine += chunk_heads(P, r) * chunk_cost(P, r, chunk_units(P, r));
    }
    if (bits && blockIdx.x == 0) raise_status(P.status, bits);
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31) sh.warp_sum[warp] = sum;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < T / 32; ++w) {
        const long long x = sh.warp_sum[w];
        before += w < warp ? x : 0;
        total += x;
    }
    before += sum - mine;
    // n shares of `share` each, the last one with what fp32 left over (at most
    // n 2^-23 of the total)
    const float all = __ll2float_rn(total);
    const int n = max(1, (int)fminf(all / ((float)P.min_share * (float)P.G), (float)gridDim.x));
    const long long share = (long long)(all / (float)n);
    for (int e = 0; e < 2; ++e) {
        const int i = (int)blockIdx.x + e;
        if (i >= n) break;
        const long long at = share * i;
        if (at < before || at >= before + mine) continue;
        long long c = before;
        for (int b = b0; b < b1; ++b) {
            if (per > 1) r = chunk_request(P, b, nullptr);
            const long long w = chunk_heads(P, r) * chunk_cost(P, r, chunk_units(P, r));
            if (at < c + w) {
                (e ? sh.end : sh.begin) = chunk_find(P, b, r, at - c);
                break;
            }
            c += w;
        }
    }
    __syncthreads();
    if (tid == 0) {
        const ChunkPos p = sh.begin;
        ChunkRecord c{make_int4(p.b, p.h, p.j, p.s), make_int4(0, 0, 0, 0)};
        if (p.s > 0) {                                   // (what the merging kernel asks for)
            const ChunkReq q = chunk_request(P, p.b, nullptr);
            c.unit = make_int4(q.first, q.n, chunk_steps(P, q, p.j), 0);
        }
        P.records[blockIdx.x] = c;
        if (blockIdx.x == gridDim.x - 1)
            P.records[gridDim.x] = ChunkRecord{make_int4(P.B, 0, 0, 0), make_int4(0, 0, 0, 0)};
    }
}

// What a CTA does of one unit: steps s0 .. s1 - 1 of `steps`.
struct ChunkPart {
    int b, h, j;
    int first, S;            // request: its first packed token, tokens held before
    int n;                   // request: new tokens
    int steps, s0, s1;
    bool paired;             // h: pair of heads 2 h, 2 h + 1
};

// Walks a CTA's share part by part.
struct ChunkWalk {
    ChunkPos at, end;
    ChunkReq r;
    int nu;
    bool fresh;

    __device__ __forceinline__ ChunkWalk(const ChunkParams &P, const ChunkShare &sh)
        : at(sh.begin), end(sh.end), r{0, 0, 0}, nu(0), fresh(true) {}

    __device__ __forceinline__ bool next(const ChunkParams &P, ChunkPart &u) {
        while (at.b < P.B) {
            if (fresh) {
                r = chunk_request(P, at.b, nullptr);
                nu = chunk_units(P, r);
                fresh = false;
            }
            if (at.b > end.b) return false;
            if (r.n == 0) {
                at = ChunkPos{at.b + 1, 0, 0, 0};
                fresh = true;
                continue;
            }
            const bool last = at.b == end.b && at.h == end.h && at.j == end.j;
            u.b = at.b;
            u.h = at.h;
            u.j = at.j;
            u.first = r.first;
            u.S = r.S;
            u.n = r.n;
            u.paired = chunk_paired(P, r);
            u.steps = chunk_steps(P, r, at.j);
            u.s0 = at.s;
            u.s1 = last ? end.s : u.steps;
            if (last) {
                at.b = P.B;
            } else {
                at.s = 0;
                if (++at.j == nu) {
                    at.j = 0;
                    if (++at.h == chunk_heads(P, r)) {
                        at.h = 0;
                        ++at.b;
                        fresh = true;
                    }
                }
            }
            if (u.s0 < u.s1) return true;
        }
        return false;
    }
};

// The slot of a part that is not a whole unit: a CTA has at most one that
// begins inside its unit and one that begins with it.
__device__ __forceinline__ int chunk_slot(const ChunkPart &u) {
    return 2 * (int)blockIdx.x + (u.s0 > 0 ? 0 : 1);
}

}  // namespace
}  // namespace sv
