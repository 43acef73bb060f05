// The tensor-core path of spec_verify_attn_kv8 (bf16 rows).
//
// The cache's codes go to the tensor cores as they are: a step takes 128
// tokens of one (request, KV head) and computes, with kind::f8f6f4 (e4m3 x
// e4m3 and e4m3 x e5m2, fp32 sums),
//   S^T [128 tokens x rows] = K (A, K-major) . Q^T (B),
//   O^T [head dims x rows] += V^T (A, MN-major) . P^T (B, MN-major),
// so the keys and values are the M = 128 operands whatever the number of
// query rows, both read straight from the tile the tensor copy left in shared
// memory (its eight-row key and value groups alternate, i.e. either lies at a
// fixed stride), and a thread of the softmax owns one token: the block's two
// scales are a scalar each to it.
//
// What is not 8 bits wide is made so.  A bf16 value has 8 significant bits, an
// e4m3 value 4: a query (and a block or soft-prompt key or value) is the sum
// of two e4m3 values under one power-of-two scale per row, exact but for
// elements under 2^-9 of the row's largest (there: half of e4m3's smallest
// step, 2^-17.8 of the largest).  P needs range more than bits, for a long
// prefix of small weights beside a large one adds up: it is the sum of three
// e5m2 values (3 significant bits, 30 binades of normal numbers; kind::f8f6f4
// takes e4m3 x e5m2), the second raised by 2^3 and the third by 2^6, so that
// what is left of a p lies in their range wherever p does.  That is p to 2^-9
// of itself (bf16: 2^-8) down to 2^-26 of the row's largest, and to 2^-35 of
// the largest below.  The parts of Q are columns of one product (or, at 64
// rows, summed in it), the parts of P columns of the other.
//
// Softmax: p = 2^(s + log2(v_scale) - M), M per row, raised only when a value
// would pass e5m2's 57344; so the tile needs no maximum, only a vote (and
// every row's sum is a register of each token's thread until the unit ends).
// l adds p / v_scale.
//
// A persistent grid takes equal parts of the linear step space (attn_tc_sched;
// a unit's start counted as four steps, 2700-6800 cycles by a fit over the
// CTAs: tree 96 us, 100 with two and 98 with six):
// a unit is a (request, KV head, block of R packed rows), its steps the prefix
// in 128-token tiles, then the tail -- soft prompt and block, which a first
// kernel has split into two e4m3 tiles -- in the same form, two ring slots a
// step.  Units split between CTAs leave fp32 partials for a combine kernel.
//
// Bound by the cache's bytes up to 32 packed rows per KV head (8 MMAs of
// about 50 cycles against ~1400 cycles to stream a tile at d = 128): 64
// requests of 16-32 K tokens, 8 KV heads, 32 rows take 508 us, 6.4 TB/s.  By
// the softmax's chain from 64 rows on (~2900 cycles a step), where the row
// blocks of a head read the cache through L2: 8 requests of 256-2048 tokens
// with 120-node trees, 480 rows a head, take 95 us, 195 TFLOP/s.  Small calls
// wait for the preparing kernel and the first copies, then for the combine:
// one token over 32 K takes 21 us, over 300 tokens 12 us; many short prefixes
// pay a unit's chain each (1200 units of two steps: 37 us).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "attn_kv8.cuh"
#include "attn_tc_sched.cuh"
#include "kv8_common.cuh"

namespace sv {
namespace {

using namespace tc5;

constexpr int kStep = 128;                  // tokens a step
constexpr float kTop = 15.75f;              // log2 of the largest P allowed (57344 = 2^15.807)
constexpr float kAim = 12.f;                // log2 P of a row's maximum when M is raised: 2^3.75 of
                                            // room before the next raise, which takes a step twice
                                            // as long (2^1.75: tree 96 -> 109 us; 2^5.75 gains
                                            // nothing), and 2^26 of P's normal range below it
constexpr float kNoRef = -1e30f;            // M of a row that has seen nothing
constexpr int kParts = 3;                   // e5m2 values that P is the sum of,
constexpr float kPartUp = 8.f;              // each raised by this over the one before

// A unit's row, as the preparing kernel leaves it.
struct alignas(8) RowMeta {
    float scale;             // softmax scale (log2) x the row's power of two
    int out;                 // (row * Hq + head) * 2 + valid, within the request; -1 past the last
};

// A CTA's range of the schedule, as the preparing kernel leaves it: its steps,
// and where the first one is.
struct alignas(16) CtaPlan {
    int n_steps, b, h, rb;
    int S, n_tiles, tile, unused;
};

struct Tc8Params {
    TcParams t;              // schedule, split, partials (t.a: the call)
    const CtaPlan *plan;     // [n_ctas]
    const float *scales;     // the cache's
    const RowMeta *q_meta;   // [units][RB]
    const float2 *tail_scale;    // [B][Hkv][tail_pad]: scales of the tail's tokens
    int tail_len, tail_pad;  // n_soft + R, rounded up to 16
    int n_tail;              // its 128-token tiles
    int box_log2;            // log2 of the tokens per cache box
    int ps16;                // page_size / 16, and ceil(2^32 / it): a page index is a product
    uint64_t ps16_inv;       // (exact for 26-bit token / 16: the error is under 16 * 2^26 / 2^32)
};

// The softmax's warpgroups.  Up to 32 rows two take alternate steps, each with
// all of the unit's rows and a running softmax (M, l, O) of its own, merged at
// the unit's end: a step's chain (wait, tensor memory, vote, exponentials, P,
// arrive: ~2000 cycles, most of it latency) then costs half.  With 64 rows, whose
// arithmetic is the larger part, they take half of the rows of every step (four
// with a quarter each repeat what a step costs a thread: tree 105 -> 111 us,
// with P in two parts).
template <int D, int RB>
struct Cfg {
    static constexpr bool kAlt = RB <= 32;
    static constexpr int NA = kAlt ? 2 : 1;             // steps in the softmax at a time
    static constexpr int NR = kAlt ? 1 : 2;             // warpgroups that share a step's rows
    static constexpr int NG = NA * NR;                  // softmax warpgroups
    static constexpr int RW = RB / NR;                  // rows of a warpgroup
    static constexpr int kThreads = NG * 128 + 128;
    static constexpr int CH = kAlt ? RW : 16;           // rows taken from tensor memory at a time
    static constexpr int NB = kAlt ? 4 : 3;             // S buffers: S runs ahead of the softmax
    static constexpr int kSlot = 2 * kStep * D;         // K and V of a step
    static constexpr int kQ = 2 * RB * D;               // a unit's queries, both parts
    static constexpr int QB = RB == 32 ? 1 : 2;         // query buffers (32 rows: no room for two)
    // P^T: tiles of PW columns, tokens PW bytes apart; the parts follow one
    // another, RB columns each (up to 16 rows all of them in one tile)
    static constexpr int PW = RB == 32 ? 32 : 64;
    static constexpr int kPTile = kStep * PW;
    static constexpr int kP = (RB <= 16 ? 1 : kParts) * kPTile;
    static constexpr int PN = RB == 8 ? 32 : kParts * RB;   // columns of the product (8 rows: 24 and 8 idle)
    static constexpr int NS = (kAlt ? 6 : 4) * (128 / D);   // ring slots
    // the two parts of Q in columns of their own, or (64 rows, for which
    // tensor memory has no room) as two products into the same ones
    static constexpr bool kSumQ = RB == 64;
    static constexpr int SN = kSumQ ? RB : 2 * RB;
    // TMEM: part q of warpgroup g's O at O(g) + QS q, S buffer b at kColS + SN b
    static constexpr int QS = RB;                       // (RB = RW where the groups alternate)
    static constexpr int kOStep = kAlt ? (PN + RB) / (2 * RB) * (2 * RB) : RW;
    static constexpr uint32_t kColS = kAlt ? 2 * kOStep : 256;
    static constexpr int kUsed = (int)kColS + NB * SN;
    static constexpr int kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static_assert(kUsed <= 512 && kOStep >= (kAlt ? PN : RW) && PN % 16 == 0 && PN <= 256, "tensor memory");
};

template <int D, int RB>
struct Shared8 {
    using C = Cfg<D, RB>;
    uint64_t full[C::NS], empty[C::NS];
    uint64_t q_full[C::QB], q_empty[C::QB];
    uint64_t s_full[C::NB], s_free[C::NB];
    uint64_t p_full[2], o_upd[2];
    uint64_t drain[2];
    float4 scale[C::NS][8];              // token_scale of each box of a slot
    alignas(16) float qs[C::NG][C::RW];      // a row's q_scale
    alignas(16) float neg_m[C::NG][C::RW];   // and its -M
    alignas(16) float fac[C::NG][C::RW];     // what its O is scaled by
    alignas(16) float red[C::NG][4][C::RW];  // the warps' maxima, or sums; what M is raised by
    alignas(16) int out[C::NG][C::RW];       // RowMeta::out
    uint32_t tmem_base;
};

template <int D, int RB>
constexpr size_t smem8() {
    using C = Cfg<D, RB>;
    return (size_t)C::NS * C::kSlot + C::QB * C::kQ + 2 * C::kP + sizeof(Shared8<D, RB>);
}
static_assert(smem8<128, 64>() <= 227 * 1024 && smem8<128, 32>() <= 227 * 1024 &&
                  smem8<64, 64>() <= 227 * 1024 && smem8<64, 32>() <= 227 * 1024,
              "shared memory of the 8-bit attention kernel");

constexpr int kAllBar = 8;               // all softmax warpgroups

// OR over the N threads at named barrier `id` (1 + g: a warpgroup).
template <int N>
__device__ __forceinline__ bool group_or(int id, bool x) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "barrier.cta.red.or.pred p, %1, %3, q;\n\tselp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((int)x), "n"(N)
        : "memory");
    return r != 0;
}
template <int N>
__device__ __forceinline__ void group_sync(int id) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}

// Largest of the warp's values (a NaN counts only where all are).
__device__ __forceinline__ float warp_redux_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// What a token's thread needs of its two scales: (key scale, log2 of the value
// scale, 1 / value scale, NaN if the value scale is NaN else 0).
__device__ __forceinline__ float4 token_scale(float k, float v) {
    const bool bad = v != v;
    v = bad ? 1.f : v;
    return make_float4(k, log2f(v), 1.f / v, bad ? __uint_as_float(0x7fffffffu) : 0.f);
}

// Sums over the warp of HR values a lane: lane i * (32 / HR) holds the i-th
// (each round halves the values a lane carries).
template <int HR>
__device__ __forceinline__ float warp_sums(const float (&x)[HR]) {
    const int lane = threadIdx.x & 31;
    float r[HR];
#pragma unroll
    for (int i = 0; i < HR; ++i) r[i] = x[i];
    int n = HR;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int j = 0; j < HR / 2; ++j) {
                if (j >= n) break;
                const float send = up ? r[j] : r[j + n], keep = up ? r[j + n] : r[j];
                r[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        } else {
            r[0] += __shfl_xor_sync(0xffffffffu, r[0], o);
        }
    }
    return r[0];
}

// Two values of P as three e5m2 pairs (by way of f16, of which e5m2 is the upper
// byte): the nearest, and the ones nearest to 8 and 64 times what is left.
__device__ __forceinline__ void split_p(float p0, float p1, uint32_t (&part)[kParts]) {
    uint32_t x;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(p1), "f"(p0));
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        uint16_t e;
        asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(e) : "r"(x));
        part[i] = e;
        if (i + 1 == kParts) break;
        // exact, both: what is left has fewer bits, and 8 times it is in range
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(__byte_perm(part[i], 0u, 0x1404)));
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(0x48004800u));   // 8, 8
    }
}

// Clears token tok's value row of a slot (a function of its own: inlined, tree
// 96.3 -> 97.6 us, short prefixes 39.1 -> 38.3).  A row's groups are taken from
// the (tok)-th on, so that eight rows' writes go to different banks.
template <int D>
__device__ __noinline__ void clear_row(uint8_t *slot, int tok) {
    uint4 *row = reinterpret_cast<uint4 *>(slot + kv8_row(tok, 1, D));
#pragma unroll
    for (int e = 0; e < D / 16; ++e) row[(e + (D == 128 ? tok : tok >> 1)) & (D / 16 - 1)] = make_uint4(0u, 0u, 0u, 0u);
}

template <int D, int RB>
__global__ void __launch_bounds__((Cfg<D, RB>::kThreads), 1)
attn_kv8_tc_kernel(const __grid_constant__ Tc8Params P, const __grid_constant__ CUtensorMap m_kv,
                   const __grid_constant__ CUtensorMap m_tail,
                   const __grid_constant__ CUtensorMap m_q) {
    using C = Cfg<D, RB>;
    constexpr int RW = C::RW, NS = C::NS, NG = C::NG, NR = C::NR;
    // warps: the softmax's, then the producers and the two that issue MMAs
    constexpr int kProducerWarp = 4 * NG, kScoreWarp = 4 * NG + 1, kValueWarp = 4 * NG + 2,
                  kProducerWarp2 = 4 * NG + 3;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem;
    uint8_t *qbuf = ring + NS * C::kSlot;
    uint8_t *pbuf = qbuf + C::QB * C::kQ;
    auto &sh = *reinterpret_cast<Shared8<D, RB> *>(pbuf + 2 * C::kP);

    // (warp numbers and step counts are broadcast: the compiler then keeps what
    // follows from them, the descriptors of copies and MMAs among it, in uniform
    // registers)
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const TcParams &T = P.t;
    const AttnParams &A = T.a;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < C::QB; ++b) {
            mbar_init(&sh.q_full[b], 1);
            mbar_init(&sh.q_empty[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.p_full[b], 4 * NR);
            mbar_init(&sh.o_upd[b], 1);
        }
        for (int b = 0; b < C::NB; ++b) {
            mbar_init(&sh.s_full[b], 1);
            mbar_init(&sh.s_free[b], 4 * NR);
        }
        mbar_init(&sh.drain[0], 1);
        mbar_init(&sh.drain[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == kScoreWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem_base)),
                     "r"(C::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem_base;
    // (the preparing kernel's range, queries and tail; it began after every
    // kernel before it had ended)
    pdl_wait();
    const int cta = blockIdx.x;
    const int4 r0 = __ldcg(reinterpret_cast<const int4 *>(P.plan + cta));
    const int4 r1 = __ldcg(reinterpret_cast<const int4 *>(P.plan + cta) + 1);
    auto unit_of = [&](const Cursor &c) { return (c.b * T.seg_h + c.h) * T.seg_rb + c.rb; };

    const int n_steps = __shfl_sync(0xffffffffu, r0.x, 0);
    auto range_begin = [&] {
        Cursor c;
        c.b = r0.y;
        c.h = r0.z;
        c.rb = r0.w;
        c.S = r1.x;
        c.n_prefix = ceil_div(c.S, kTile);
        c.n_tiles = r1.y;
        c.tile = r1.z;
        return c;
    };

    if (n_steps > 0 && (warp == kProducerWarp || warp == kProducerWarp2)) {
        // ------------------------------------------------------ producers
        // Two warps take alternate ring slots (a slot's copies keep their
        // issuing warp for most of the time the tile takes to stream, and
        // the other warp gets its next slot ready meanwhile): its copies and
        // its scales.  They walk the range in groups of up to eight prefix
        // steps of a unit (or one tail step, two slots): lane 8 u + i owns
        // box i of the warp's u-th step of the group, so a page id costs one
        // load per lane, issued two groups ahead of its copy, and a scale
        // one, issued a group ahead.
        const int w = warp == kProducerWarp ? 0 : 1;
        const uint64_t keep = policy_evict_last();
        const uint64_t stream = T.seg_rb == 1 ? policy_evict_first() : keep;
        const int bt = 1 << P.box_log2, boxes = kStep >> P.box_log2;
        const int u = lane >> 3, box = lane & 7;
        struct Group {
            Cursor c;            // its first step
            int k, n;            // that step's number, steps (0: past the range)
            int at;              // its first slot, counted from the range's first
            bool tail;
            int pg, row;         // this lane's page (-1 no box, -2 a bad page), row of its tile
        };
        auto group_at = [&](const Cursor &c, int k, int at) {
            Group g;
            g.c = c;
            g.k = k;
            g.n = 0;
            g.at = at;
            g.tail = false;
            g.pg = -1;
            g.row = 0;
            if (k >= n_steps) return g;
            const int np = (c.S + kStep - 1) / kStep;
            g.tail = c.tile >= np;
            g.n = g.tail ? 1 : min(min(8, np - c.tile), n_steps - k);
            const int i = 2 * u + ((at ^ w) & 1);            // this lane's step of the group
            const int tok = (c.tile + i) * kStep + (box << P.box_log2);
            if (!g.tail && i < g.n && box < boxes && tok < c.S) {
                const int t16 = tok >> 4, j = (int)((t16 * P.ps16_inv) >> 32);
                g.row = (t16 - j * P.ps16) * 32;
                const int pg = A.page_table[(size_t)c.b * A.max_pages + j];
                g.pg = pg < 0 || pg >= A.n_pages ? -2 : pg;
            }
            return g;
        };
        auto after = [&](const Group &g) {          // the group that follows
            Cursor c = g.c;
            if (g.n > 0 && g.k + g.n < n_steps) {
                c.tile += g.n - 1;
                cursor_next(T, c);
            }
            return group_at(c, g.n > 0 ? g.k + g.n : n_steps, g.at + (g.tail ? 2 : g.n));
        };
        auto scale_of = [&](const Group &g) {
            if (g.pg < 0) return make_float2(1.f, 1.f);
            const float *at = P.scales + ((size_t)g.pg * A.Hkv + g.c.h) * 2;   // (4-byte aligned)
            return make_float2(at[0], at[1]);
        };
        Group cur = group_at(range_begin(), 0, 0), next = after(cur);
        float2 sc = scale_of(cur);
        int slot = w, phase = 0, used = 0;   // used: slots filled by this warp
        static_assert(NS % 2 == 0, "a warp's slots have one parity");
        bool ok = true;
        while (cur.n > 0 && ok) {
            const Group far = after(next);
            const float2 sc1 = scale_of(next);
            const float4 ts = token_scale(kv8_read_scale(sc.x), kv8_read_scale(sc.y));
            if (cur.pg == -2) raise_status(A.status, SPEC_DEV_BAD_PAGE);
            const unsigned boxed = __ballot_sync(0xffffffffu, cur.pg >= 0);
            const bool tail = __shfl_sync(0xffffffffu, (int)cur.tail, 0) != 0;
            // (tail) its tile and its boxes of 16 tokens
            const int tile0 = __shfl_sync(0xffffffffu, cur.c.tile - (cur.c.S + kStep - 1) / kStep, 0);
            const int bh = __shfl_sync(0xffffffffu, cur.c.b * A.Hkv + cur.c.h, 0);
            const int nb = (min(kStep, P.tail_len - tile0 * kStep) + 15) >> 4;
            const int first = (__shfl_sync(0xffffffffu, cur.at, 0) ^ w) & 1;
            const int slots = __shfl_sync(0xffffffffu, cur.tail ? 2 : cur.n, 0);
            const int tile_of = cur.pg * A.Hkv + cur.c.h;
            for (int i = first, v = 0; i < slots; i += 2, ++v) {
                // (everything a copy needs, before its slot is waited for)
                int z[8], row[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    z[x] = __shfl_sync(0xffffffffu, tile_of, (8 * v + x) & 31);
                    row[x] = __shfl_sync(0xffffffffu, cur.row, (8 * v + x) & 31);
                }
                const unsigned mine = (boxed >> (8 * v)) & 0xffu;
                if (!__all_sync(0xffffffffu, mbar_wait(&sh.empty[slot], (uint32_t)(phase ^ 1), T.wait))) {
                    ok = false;
                    break;
                }
                uint8_t *dst = ring + slot * C::kSlot;
                if (u == v && box < boxes && !tail) sh.scale[slot][box] = ts;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_expect_tx(&sh.full[slot], tail ? (uint32_t)(nb * 32 * D)
                                                               : (uint32_t)__popc(mine) * (uint32_t)(2 * bt * D));
                __syncwarp();
                if (tail) {
                    const int r0 = (bh * 2 + i) * (2 * P.tail_pad) + tile0 * (2 * kStep);
                    for (int x = 0; x < nb; ++x)
                        if (lane == 0)
                            tma_load_2d(dst + x * 32 * D, &m_tail, 0, r0 + x * 32, &sh.full[slot], keep);
                } else if (mine == 0xffu) {
                    if (lane == 0) {
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            tma_load_3d(dst + x * (32 * D), &m_kv, 0, row[x], z[x], &sh.full[slot], stream);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        if (((mine >> x) & 1u) && lane == 0)
                            tma_load_3d(dst + x * (2 * bt * D), &m_kv, 0, row[x], z[x], &sh.full[slot], stream);
                    }
                }
                ++used;
                slot += 2;
                if (slot >= NS) {
                    slot -= NS;
                    phase ^= 1;
                }
            }
            cur = next;
            next = far;
            sc = sc1;
        }
        if (lane == 0) {
            if (!ok) raise_status(A.status, SPEC_DEV_TIMEOUT);
            // do not leave while copies into this CTA's shared memory are in
            // flight (the default limit: these copies were issued and complete)
            for (int i = used - 1; i >= 0 && i >= used - NS / 2; --i)
                if (!mbar_wait(&sh.full[w + 2 * (i % (NS / 2))], (uint32_t)((i / (NS / 2)) & 1))) {
                    raise_status(A.status, SPEC_DEV_TIMEOUT);
                    break;
                }
        }
    } else if (n_steps > 0 && (warp == kScoreWarp || warp == kValueWarp)) {
        // ---------------------------------------------------- MMA issuers
        // One thread issues S, another PV (one alone took ~2000 cycles a step,
        // more than the tile takes to stream).  Slot: 8-token groups of 8 key
        // rows, then 8 value rows, D bytes each.  K (K-major): groups 16 D
        // apart, a step of 32 head dimensions 32 bytes on.  V (MN-major): the
        // same groups, 8 D further; a step of 32 tokens is four groups.  At
        // D = 64 the 128 rows of M are the 64 dimensions twice (leading
        // offset 0).  The first also fetches the units' queries, the next
        // unit's while this one's first scores are computed or, with one
        // buffer, once its last ones are.
        const bool scores = warp == kScoreWarp;
        Cursor c = range_begin();
        constexpr uint32_t id_s = idesc_e4m3(kStep, C::SN, false, false, false);
        constexpr uint32_t id_pv = idesc_e4m3(kStep, C::PN, true, true, true);
        const uint64_t kd0 = smem_desc_sw<D>(smem_u32(ring), 16, 16 * D);
        const uint64_t vd0 = smem_desc_sw<D>(smem_u32(ring) + 8 * D, 0, 16 * D);
        const uint64_t qd0 = smem_desc_sw<D>(smem_u32(qbuf), 16, 8 * D);
        const uint64_t pd0 = smem_desc_sw<C::PW>(smem_u32(pbuf), C::kPTile, 8 * C::PW);
        int nq = 0, slot = 0, phase = 0, k = 0, sb = 0, sphase = 0;
        // every lane waits and counts, lane 0 issues
        auto wait = [&](uint64_t *bar, int parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)parity, T.wait)) != 0;
        };
        bool ok = true;
        // the queries of the unit at `at`, once the buffer's unit is done with it
        int asked = 0;
        auto queries = [&](const Cursor &at) {
            const int qb = asked % C::QB, turn = asked / C::QB;
            if (turn > 0 && !wait(&sh.q_empty[qb], (turn - 1) & 1)) return false;
            if (lane == 0) {
                mbar_arrive_expect_tx(&sh.q_full[qb], C::kQ);
                tma_load_2d(qbuf + qb * C::kQ, &m_q, 0, unit_of(at) * (2 * RB), &sh.q_full[qb],
                            policy_evict_last());
            }
            ++asked;
            return true;
        };
        if (scores) ok = queries(c);
        while (ok && k < n_steps) {
            // a unit's steps of this range
            const int k0 = k;
            const int n = __shfl_sync(0xffffffffu, min(n_steps - k, c.n_tiles - c.tile), 0);
            const int n_prefix =              // of them prefix steps
                __shfl_sync(0xffffffffu, (c.S + kStep - 1) / kStep - c.tile, 0);
            Cursor c1 = c;                   // the next unit
            c1.tile += n - 1;
            cursor_next(T, c1);
            const int qb = nq % C::QB;
            if (scores && !wait(&sh.q_full[qb], (nq / C::QB) & 1)) {
                ok = false;
                break;
            }
            ++nq;
            const uint64_t qd = qd0 + (uint64_t)((qb * C::kQ) >> 4);
            for (int i = 0; i < n && ok; ++i, ++k) {
                const int parts = i >= n_prefix ? 2 : 1, b = k & 1;
                if (scores) {
                    if (!wait(&sh.s_free[sb], sphase ^ 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t ts = tmem + C::kColS + (uint32_t)(sb * C::SN);
                    for (int part = 0; part < parts; ++part) {
                        if (!wait(&sh.full[slot], phase)) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        const uint64_t kd = kd0 + (uint64_t)((slot * C::kSlot) >> 4);
                        if (lane == 0) {
#pragma unroll
                            for (int e = 0; e < D / 32; ++e)
                                mma8_ss(ts, kd + (uint64_t)(e * 32 >> 4), qd + (uint64_t)(e * 32 >> 4),
                                        id_s, (e > 0 || part > 0) ? 1u : 0u);
                            if constexpr (C::kSumQ) {
#pragma unroll
                                for (int e = 0; e < D / 32; ++e)
                                    mma8_ss(ts, kd + (uint64_t)(e * 32 >> 4),
                                            qd + (uint64_t)((RB * D + e * 32) >> 4), id_s, 1u);
                            }
                        }
                        if (++slot == NS) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
                    if (!ok) break;
                    if (lane == 0) {
                        commit(&sh.s_full[sb]);
                        if (i == n - 1) commit(&sh.q_empty[qb]);
                    }
                    if (++sb == C::NB) {
                        sb = 0;
                        sphase ^= 1;
                    }
                    if (i == (C::QB > 1 ? 0 : n - 1) && k0 + n < n_steps && !queries(c1)) {
                        ok = false;
                        break;
                    }
                } else {
                    if (!wait(&sh.p_full[b], (k >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint64_t pd = pd0 + (uint64_t)((b * C::kP) >> 4);
                    const uint32_t to = tmem + (C::kAlt ? (uint32_t)(b * C::kOStep) : 0u);
                    const bool first = k - k0 < (C::kAlt ? 2 : 1);       // into its O
                    for (int part = 0; part < parts; ++part) {
                        // (met: S(k) has read the slot)
                        if (!wait(&sh.full[slot], phase)) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        const uint64_t vd = vd0 + (uint64_t)((slot * C::kSlot) >> 4);
                        if (lane == 0) {
#pragma unroll
                            for (int e = 0; e < kStep / 32; ++e)
                                mma8_ss(to, vd + (uint64_t)((e * 4 * 16 * D) >> 4),
                                        pd + (uint64_t)((e * 32 * C::PW) >> 4), id_pv,
                                        (e > 0 || part > 0 || !first) ? 1u : 0u);
                            commit(&sh.empty[slot]);
                        }
                        if (++slot == NS) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
                    if (!ok) break;
                    if (lane == 0) commit(&sh.o_upd[b]);
                }
            }
            c = c1;
        }
        if (lane == 0) {
            if (!ok) raise_status(A.status, SPEC_DEV_TIMEOUT);
            // the queries asked for have landed, and every MMA issued above has completed before TMEM is released
            // (the default limit)
            for (int q = asked - 1; q >= 0 && q >= asked - C::QB; --q)
                if (!mbar_wait(&sh.q_full[q % C::QB], (uint32_t)((q / C::QB) & 1)))
                    raise_status(A.status, SPEC_DEV_TIMEOUT);
            uint64_t *drain = &sh.drain[scores ? 0 : 1];
            commit(drain);
            if (!mbar_wait(drain, 0)) raise_status(A.status, SPEC_DEV_TIMEOUT);
        }
    } else if (n_steps > 0 && warp < kProducerWarp) {
        // -------------------------------------------------------- softmax
        // warpgroup g: the steps k = g (mod 2), or rows RW g .. of every step;
        // a thread: one token of the step (TMEM lane), later one dimension of O
        constexpr bool kAlt = C::kAlt;
        constexpr int CH = C::CH;
        const int g = warp >> 2, wq = warp & 3, bar = 1 + g;
        const int tok = wq * 32 + lane, gi = threadIdx.x & 127;
        const int ga = g / NR, row0 = g % NR * RW;
        const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
        const uint32_t to = tmem + lane_base;          // O of both warpgroups
        const uint32_t og = to + (uint32_t)(g * C::kOStep);    // and of this one
        Cursor c = range_begin();
        float l[RW];
        // ok: this warp's waits were met; dead: the warpgroup has stopped (it
        // still meets the others at the units' barriers)
        bool ok = true, dead = false;
        int k = 0;
        uint32_t taken = 0;                      // ring slots before the unit

        RowMeta meta{0.f, -1};             // the unit's row gi, loaded a unit ahead
        if (gi < RW) meta = P.q_meta[(size_t)unit_of(c) * RB + row0 + gi];
        while (k < n_steps) {
            // --- a unit's steps of this range
            const int k0 = k, tile0 = c.tile, n = min(n_steps - k, c.n_tiles - c.tile), S = c.S;
            const int np = (S + kStep - 1) / kStep, seg_b = c.b, seg_h = c.h, seg_id = unit_of(c);
            const bool seg_whole = tile0 == 0 && n == c.n_tiles;
            if (gi < RW) {
                sh.out[g][gi] = meta.out;
                sh.qs[g][gi] = meta.scale;
                sh.neg_m[g][gi] = 0.f;
            }
            bool unset = true;           // rows without a reference: M (0) is still to be set
            c.tile += n - 1;
            cursor_next(T, c);
            if (gi < RW && k + n < n_steps) meta = P.q_meta[(size_t)unit_of(c) * RB + row0 + gi];
#pragma unroll
            for (int i = 0; i < RW; ++i) l[i] = 0.f;
            group_sync<128>(bar);

            k = k0 + (kAlt ? (k0 ^ ga) & 1 : 0);
            for (; k < k0 + n; k += kAlt ? 2 : 1) {
                if (dead) continue;
                const int tile = tile0 + k - k0;
                const bool tail = tile >= np;
                // (a tail step takes two slots)
                const uint32_t at = taken + (uint32_t)(k - k0 + max(0, tile - max(np, tile0)));
                const int slot0 = (int)(at % NS), phase0 = (int)((at / NS) & 1u);
                const int sb = k % C::NB;
                const int left = tail ? P.tail_len - (tile - np) * kStep : S - tile * kStep;
                const bool here = tok < left;
                // rows' visibility of this warp's 32 tail tokens, lane i: row i
                uint32_t seen = 0u;
                float4 sc = make_float4(0.f, 0.f, 1.f, 0.f);
                if (tail) {
                    const int tt0 = (tile - np) * kStep + wq * 32;
                    if (here) {
                        const float2 x =
                            P.tail_scale[((size_t)seg_b * A.Hkv + seg_h) * P.tail_pad + tt0 + lane];
                        sc = token_scale(x.x, x.y);
                    }
                    const int out = lane < RW ? sh.out[g][lane] : -1;
                    if (out >= 0 && (out & 1)) {
                        const int rr = (out >> 1) / A.Hq;
                        const uint32_t *vr = A.vis + ((size_t)seg_b * A.R + rr) * A.W;
                        auto word = [&](int w) {
                            if (w < 0 || w >= A.W) return 0u;
                            const int cols = A.R - w * 32;      // from the word's first
                            return cols >= 32 ? vr[w] : vr[w] & ((1u << cols) - 1u);
                        };
                        // block columns c0 .. c0 + 31
                        const int c0 = tt0 - A.n_soft, sft = c0 & 31, w0 = c0 >> 5;     // (floor)
                        seen = word(w0) >> sft;
                        if (sft) seen |= word(w0 + 1) << (32 - sft);
                        const int ns = A.n_soft - tt0;          // soft tokens from here on
                        if (ns > 0 && (A.row_flags[(size_t)seg_b * A.R + rr] & SPEC_ROW_SEES_SOFT))
                            seen |= ns >= 32 ? 0xffffffffu : (1u << ns) - 1u;
                    }
                }
                if (ok) {
                    // S; the slots' own barriers for the scales and for the rows
                    // cleared below; PV(k - 2) has read the P buffer written
                    // below (and, where the warpgroups alternate, is in their O)
                    uint64_t *const bs = &sh.s_full[sb], *const bf = &sh.full[slot0], *const bo = &sh.o_upd[k & 1];
                    const uint32_t ps = (uint32_t)((k / C::NB) & 1), po = (uint32_t)(((k >> 1) - 1) & 1);
                    const bool s_in = mbar_test_wait(bs, ps), f_in = mbar_test_wait(bf, (uint32_t)phase0),
                               o_in = k < 2 || mbar_test_wait(bo, po);
                    ok = (s_in || mbar_wait(bs, ps, T.wait)) &&
                         (f_in || mbar_wait(bf, (uint32_t)phase0, T.wait)) &&
                         (o_in || mbar_wait(bo, po, T.wait));
                    if (tail) {
                        const int s1 = slot0 + 1 == NS ? 0 : slot0 + 1;
                        ok = ok && mbar_wait(&sh.full[s1], (uint32_t)(s1 ? phase0 : phase0 ^ 1), T.wait);
                    }
                    ok = __all_sync(0xffffffffu, ok);
                }
                const uint32_t ts = to + C::kColS + (uint32_t)(sb * C::SN + row0);
                float y[RW];
                // y = s x (key scale, softmax scale) + log2(value scale) - M: the
                // exponents of P, from S or the two parts of it
                auto exponents = [&] {
                    const uint64_t sk2 = pair(sc.x, sc.x), lv2 = pair(sc.y, sc.y), z = pair(0.f, 0.f);
#pragma unroll
                    for (int i0 = 0; i0 < RW; i0 += CH) {
                        uint32_t hi[CH], lo[CH];
                        ldn<CH>(ts + i0, hi);
                        if constexpr (C::kSumQ) {
                            wait_ldn<CH>(hi);
                        } else {
                            ldn<CH>(ts + RB + i0, lo);
                            wait_ldn<CH>(hi, lo);
                        }
                        auto score = [&](int i) {
                            const uint64_t x = pair(__uint_as_float(hi[i]), __uint_as_float(hi[i + 1]));
                            if constexpr (C::kSumQ) return x;
                            else return add2(x, pair(__uint_as_float(lo[i]), __uint_as_float(lo[i + 1])));
                        };
#pragma unroll
                        for (int i = 0; i < CH; i += 4) {
                            const float4 q = *reinterpret_cast<const float4 *>(&sh.qs[g][i0 + i]);
                            const float4 m = *reinterpret_cast<const float4 *>(&sh.neg_m[g][i0 + i]);
                            unpair(fma2(score(i), fma2(pair(q.x, q.y), sk2, z), add2(pair(m.x, m.y), lv2)),
                                   y[i0 + i], y[i0 + i + 1]);
                            unpair(fma2(score(i + 2), fma2(pair(q.z, q.w), sk2, z), add2(pair(m.z, m.w), lv2)),
                                   y[i0 + i + 2], y[i0 + i + 3]);
                        }
                    }
                };
                // -inf for what a row does not see
                auto mask = [&] {
                    if (tail) {
#pragma unroll
                        for (int i = 0; i < RW; ++i) {
                            const uint32_t row = __shfl_sync(0xffffffffu, seen, i);
                            y[i] = here && ((row >> lane) & 1u) ? y[i] : -INFINITY;
                        }
                    } else if (!here) {
#pragma unroll
                        for (int i = 0; i < RW; ++i) y[i] = -INFINITY;
                    }
                };
                float top = -INFINITY;
                if (ok) {
                    fence_after();
                    if (!tail && here) sc = sh.scale[slot0][tok >> P.box_log2];
                    exponents();
                    mask();
#pragma unroll
                    for (int i = 0; i < RW; i += 2) top = max3(top, y[i], y[i + 1]);
                }
                if (group_or<128>(bar, unset || top > kTop || !ok)) {
                    if (group_or<128>(bar, !ok)) {
                        dead = true;
                        continue;
                    }
                    // set M, or raise it where a row's maximum grew
                    float mine = -INFINITY;
#pragma unroll
                    for (int i = 0; i < RW; ++i) {
                        const float m = warp_redux_max(y[i]);
                        mine = lane == i ? m : mine;
                    }
                    if (lane < RW) sh.red[g][wq][lane] = mine;
                    group_sync<128>(bar);
                    bool none = false;
                    if (gi < RW) {
                        // (fmaxf leaves out a NaN: a row of NaN alone counts as unseen)
                        const float m = fmaxf(fmaxf(fmaxf(sh.red[g][0][gi], sh.red[g][1][gi]),
                                                    fmaxf(sh.red[g][2][gi], sh.red[g][3][gi])), -INFINITY);
                        // (a row without a reference has M = 0 and no sums yet)
                        const float was = sh.neg_m[g][gi];
                        none = m == -INFINITY && was == 0.f;
                        const float up = m == -INFINITY ? 0.f : was == 0.f ? m - kAim : fmaxf(0.f, m - kAim);
                        sh.red[g][0][gi] = up;
                        sh.fac[g][gi] = was == 0.f ? 0.f : exp2f(-up);
                        sh.neg_m[g][gi] = was - up == 0.f && !none ? -1e-30f : was - up;
                    }
                    unset = group_or<128>(bar, none);
#pragma unroll
                    for (int i = 0; i < RW; i += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&sh.fac[g][i]);
                        const float4 d = *reinterpret_cast<const float4 *>(&sh.red[g][0][i]);
                        l[i] *= f.x;
                        l[i + 1] *= f.y;
                        l[i + 2] *= f.z;
                        l[i + 3] *= f.w;
                        y[i] -= d.x;
                        y[i + 1] -= d.y;
                        y[i + 2] -= d.z;
                        y[i + 3] -= d.w;
                    }
                    if (k - k0 >= (kAlt ? 2 : 1)) {        // O holds earlier steps
                        if (!kAlt)
                            ok = mbar_wait_warp(&sh.o_upd[(k - 1) & 1], (uint32_t)(((k - 1) >> 1) & 1),
                                                T.wait);
                        if (ok) {
                            fence_after();
                            constexpr int CO = RW < 16 ? RW : 16;
#pragma unroll 1
                            for (int e = 0; e < kParts * RW; e += CO) {
                                uint32_t x[CO];
                                const uint32_t at = og + (uint32_t)(e / RW * C::QS + (e & (RW - 1)));
                                ldn<CO>(at, x);
                                wait_ldn<CO>(x);
#pragma unroll
                                for (int i = 0; i < CO; i += 4) {
                                    const float4 f =
                                        *reinterpret_cast<const float4 *>(&sh.fac[g][(e & (RW - 1)) + i]);
                                    x[i] = __float_as_uint(__uint_as_float(x[i]) * f.x);
                                    x[i + 1] = __float_as_uint(__uint_as_float(x[i + 1]) * f.y);
                                    x[i + 2] = __float_as_uint(__uint_as_float(x[i + 2]) * f.z);
                                    x[i + 3] = __float_as_uint(__uint_as_float(x[i + 3]) * f.w);
                                }
                                stn<CO>(at, x);
                            }
                            wait_st();
                        }
                    }
                }
                // (the scores are in registers for good)
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_free[sb]);
                {
                    const uint64_t is2 = pair(sc.z, sc.z);
#pragma unroll
                    for (int i = 0; i < RW; i += 2) {
                        y[i] = fast_exp2(y[i]);
                        y[i + 1] = fast_exp2(y[i + 1]);
                        unpair(fma2(pair(y[i], y[i + 1]), is2, pair(l[i], l[i + 1])), l[i], l[i + 1]);
                    }
                }
                if (__any_sync(0xffffffffu, sc.w != sc.w)) {
                    // a NaN value scale: NaN in the rows that see the token
#pragma unroll
                    for (int i = 0; i < RW; ++i) {
                        const uint32_t row = __shfl_sync(0xffffffffu, seen, i);
                        if (here && (!tail || ((row >> lane) & 1u))) y[i] += sc.w;
                    }
                }
                if (ok) {
                    // 16 bytes of part q, rows 16 j ..: PW / 16 of them a tile's row,
                    // in the order of the swizzle
                    uint8_t *const prow = pbuf + (k & 1) * C::kP + tok * C::PW;
                    const int swz = C::PW == 64 ? (tok >> 1) & 3 : (tok >> 2) & 1;
                    constexpr int RJ = RW < 16 ? RW : 16;   // rows at a time
#pragma unroll
                    for (int j = 0; j < RW; j += RJ) {
                        uint32_t w[kParts][RJ / 4];
#pragma unroll
                        for (int i = 0; i < RJ; i += 4) {
                            uint32_t a[kParts], b[kParts];
                            split_p(y[j + i], y[j + i + 1], a);
                            split_p(y[j + i + 2], y[j + i + 3], b);
#pragma unroll
                            for (int q = 0; q < kParts; ++q) w[q][i / 4] = a[q] | (b[q] << 16);
                        }
                        auto at = [&](int q, int byte) {    // (byte: a multiple of 16 within the part)
                            const int col = RB <= 16 ? q * RB + byte : byte;
                            return prow + (RB <= 16 ? 0 : q * C::kPTile) + (((col >> 4) ^ swz) << 4);
                        };
                        if constexpr (RW == 8) {
                            *reinterpret_cast<uint4 *>(at(0, 0)) = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
                            *reinterpret_cast<uint2 *>(at(2, 0)) = make_uint2(w[2][0], w[2][1]);
                        } else {
#pragma unroll
                            for (int q = 0; q < kParts; ++q)
                                *reinterpret_cast<uint4 *>(at(q, row0 + j)) =
                                    make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
                        }
                    }
                    // V rows past the last token hold whatever the copy left: P
                    // is 0 there, but 0 x NaN is NaN
                    if (!here && row0 == 0) {
                        const int s1 = slot0 + 1 == NS ? 0 : slot0 + 1;
                        clear_row<D>(ring + slot0 * C::kSlot, tok);
                        if (tail) clear_row<D>(ring + s1 * C::kSlot, tok);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_full[k & 1]);
                }
            }

            // --- the unit's end in this range: PV(k - 1) and all before it, the
            // row sums over the tokens' threads, then O / l and LSE, or the
            // partials (two running softmaxes merged where the groups alternate)
            k = k0 + n;
            taken += (uint32_t)(n + max(0, tile0 + n - max(np, tile0)));
            const int j = k - 1;
            constexpr int kPer = 32 / RW;
            const float sum = warp_sums<RW>(l);
            // (each group waits for its own last PV, behind the last use of sh.red
            // by any of its warps)
            const int jw = kAlt && (j & 1) != ga ? j - 1 : j;
            const bool got = !dead && ok &&
                             (jw < k0 || mbar_wait_warp(&sh.o_upd[jw & 1], (uint32_t)((jw >> 1) & 1), T.wait));
            if (lane % kPer == 0) sh.red[g][wq][lane / kPer] = sum;
            if (group_or<NG * 128>(kAllBar, !got)) {
                ok = false;
                break;
            }
            fence_after();
            const size_t prow = slot_row(T, seg_id, cta, 0, 1, 0);
            if (threadIdx.x < RB) {
                const int r = threadIdx.x, rg = r / RW, ri = r % RW;
                auto row_sum = [&](int q) {
                    return (sh.red[q][0][ri] + sh.red[q][1][ri]) + (sh.red[q][2][ri] + sh.red[q][3][ri]);
                };
                // (-M of 0: the row has seen nothing)
                auto ref = [&](int q) { return sh.neg_m[q][ri] == 0.f ? kNoRef : -sh.neg_m[q][ri]; };
                // What has seen nothing is left out: a warpgroup without a step in
                // the range has not written its O.
                auto none_in = [&](int q) { return sh.neg_m[q][ri] == 0.f && row_sum(q) == 0.f; };
                float M = ref(rg), L = row_sum(rg), f0 = 1.f, f1 = 0.f;
                if (kAlt) {
                    const float m0 = M, m1 = ref(NR + rg);
                    M = fmaxf(m0, m1);
                    f0 = exp2f(m0 - M);
                    f1 = exp2f(m1 - M);
                    L = f0 * L + f1 * row_sum(NR + rg);
                }
                const int out = sh.out[rg][ri];
                const bool none = !(out & 1) || L == 0.f;
                const float inv = !seg_whole ? 1.f : none ? 0.f : 1.f / L;
                // (a factor that underflows still passes on a NaN: 2^-149, not 0,
                // which leaves the O out)
                auto factor = [&](float f, int q) {
                    return (none && seg_whole) || none_in(q) ? 0.f : f * inv == 0.f ? 1.4e-45f : f * inv;
                };
                sh.fac[rg][ri] = factor(f0, rg);
                if (kAlt) sh.fac[(NG - 1) / NR * NR + rg][ri] = factor(f1, NR + rg);
                if (seg_whole && out >= 0) {
                    const int rr = (out >> 1) / A.Hq, hq = (out >> 1) - rr * A.Hq;
                    A.lse[((size_t)seg_b * A.Hq + hq) * A.R + rr] =
                        none ? -INFINITY : (M + log2f(L)) * kLn2;
                } else if (!seg_whole) {
                    *reinterpret_cast<float2 *>(A.part_ml + (prow + r) * 2) = make_float2(M, L);
                }
            }
            group_sync<NG * 128>(kAllBar);
            // warpgroup g writes rows (RB / NG) g ..
            constexpr int HB = RB / NG, CE = HB < 8 ? HB : 8;
#pragma unroll 1
            for (int i0 = g * HB; i0 < (g + 1) * HB; i0 += CE) {
                const int rg = i0 / RW, oi = i0 % RW;
                // O of rows i0 .., its parts summed
                auto o_sum = [&](uint32_t at, float (&x)[CE]) {
                    uint32_t a[CE], b[CE], c2[CE];
                    ldn<CE>(at, a);
                    ldn<CE>(at + C::QS, b);
                    ldn<CE>(at + 2 * C::QS, c2);
                    wait_ldn<CE>(a, b);
                    wait_ldn<CE>(c2);
#pragma unroll
                    for (int i = 0; i < CE; ++i)
                        x[i] = fmaf(fmaf(__uint_as_float(c2[i]), 1.f / kPartUp, __uint_as_float(b[i])),
                                    1.f / kPartUp, __uint_as_float(a[i]));
                };
                float x[CE], x1[CE];
                o_sum(to + (uint32_t)(kAlt ? oi : rg * C::kOStep + oi), x);
                if constexpr (kAlt) o_sum(to + (uint32_t)(C::kOStep + oi), x1);
                if (tok < D) {
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(A.o) + (size_t)seg_b * A.R * A.Hq * D + tok;
                    float *po = A.part_o + (prow + i0) * D + tok;
                    int out[CE];
                    // (read ahead of the stores, which the compiler keeps them behind)
#pragma unroll
                    for (int i = 0; i < CE; i += 4) {
                        float f0[4], f1[4];
                        *reinterpret_cast<float4 *>(f0) = *reinterpret_cast<const float4 *>(&sh.fac[rg][oi + i]);
                        if constexpr (kAlt)
                            *reinterpret_cast<float4 *>(f1) =
                                *reinterpret_cast<const float4 *>(&sh.fac[(NG - 1) / NR * NR + rg][oi + i]);
                        *reinterpret_cast<int4 *>(&out[i]) = *reinterpret_cast<const int4 *>(&sh.out[rg][oi + i]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // (a factor of 0: nothing seen, and O may hold anything)
                            x[i + e] = f0[e] == 0.f ? 0.f : f0[e] * x[i + e];
                            if constexpr (kAlt)
                                if (f1[e] != 0.f) x[i + e] = fmaf(f1[e], x1[i + e], x[i + e]);
                        }
                    }
                    if (seg_whole) {
#pragma unroll
                        for (int i = 0; i < CE; ++i)
                            if (out[i] >= 0) o[(size_t)(out[i] >> 1) * D] = __float2bfloat16_rn(x[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < CE; ++i) po[i * D] = x[i];
                    }
                }
            }
            fence_before();
            group_sync<NG * 128>(kAllBar);              // O, M and l may be written again
        }
        if (!ok) raise_status(A.status, SPEC_DEV_TIMEOUT);
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kScoreWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(C::kCols));
}

// Merge of the units split between CTAs: block (i, rows) takes four rows, a
// warp each, of the unit whose first boundary lies between CTAs i and i + 1.
template <int D>
__global__ void __launch_bounds__(128) attn_kv8_tc_combine_kernel(const __grid_constant__ TcParams T) {
    pdl_wait();
    const AttnParams &A = T.a;
    const BoundaryRec rec = T.recs[blockIdx.x + 1];
    if (rec.seg < 0) return;
    const int rb = rec.seg % T.seg_rb, h = (rec.seg / T.seg_rb) % T.seg_h;
    const int b = rec.seg / (T.seg_rb * T.seg_h);
    const int lane = threadIdx.x & 31, r = blockIdx.y * 4 + (threadIdx.x >> 5);
    const int p = rb * A.rb_rows + r;
    if (p >= A.M) return;
    auto has_part = [&](int i) {
        if (rec.last - rec.first < 32) return ((rec.parts >> (i - rec.first)) & 1u) != 0;
        return max(T.bounds[i], rec.s0) < min(T.bounds[i + 1], rec.s1);
    };
    // lane i: part first + i, first + i + 32, ...
    float m = kNoRef;
    for (int i = rec.first + lane; i <= rec.last; i += 32)
        if (has_part(i)) m = fmaxf(m, A.part_ml[slot_row(T, rec.seg, i, 0, 1, r) * 2]);
    m = warp_max(m);
    constexpr int E = D / 32;
    float out[E], L = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = 0.f;
    for (int i0 = rec.first; i0 <= rec.last; i0 += 32) {
        const int i = i0 + lane;
        float w = 0.f;
        const bool part = i <= rec.last && has_part(i);
        if (part) {
            const size_t row = slot_row(T, rec.seg, i, 0, 1, r);
            w = exp2f(A.part_ml[row * 2] - m);
            L = fmaf(w, A.part_ml[row * 2 + 1], L);
        }
        unsigned todo = __ballot_sync(0xffffffffu, part);
        while (todo) {
            // four parts' rows in flight
            float x[4][E], wj[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = todo ? __ffs(todo) - 1 : -1;
                if (todo) todo &= todo - 1;
                wj[u] = j >= 0 ? __shfl_sync(0xffffffffu, w, j) : 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[u][e] = j >= 0 ? A.part_o[slot_row(T, rec.seg, i0 + j, 0, 1, r) * D + lane + 32 * e]
                                     : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) out[e] = fmaf(wj[u], x[u][e], out[e]);
        }
    }
    L = warp_sum(L);
    const int rr = p / A.G, hq = h * A.G + p % A.G;
    const bool valid = (A.row_flags[(size_t)b * A.R + rr] & SPEC_ROW_VALID) != 0;
    const bool none = !valid || L == 0.f;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(A.o) + (((size_t)b * A.R + rr) * A.Hq + hq) * D;
#pragma unroll
    for (int e = 0; e < E; ++e) o[lane + 32 * e] = __float2bfloat16_rn(none ? 0.f : out[e] / L);
    if (lane == 0)
        A.lse[((size_t)b * A.Hq + hq) * A.R + rr] = none ? -INFINITY : (m + log2f(L)) * kLn2;
}

// ------------------------------------------------------------ preparation

struct Prep8Params {
    TcParams t;              // (t.a: the call)
    CtaPlan *plan;
    int plan_ctas;           // blocks that lay out the schedule
    uint8_t *q8;             // [units][2][RB][D]
    RowMeta *q_meta;         // [units][RB]
    uint8_t *tail8;          // [B][Hkv][2][tail_pad / 8][2][8][D]
    float2 *tail_scale;      // [B][Hkv][tail_pad]
    int rb, seg_rb, tail_pad;
    int q_rows, t_rows;
};

// A row of D bf16 values (src NULL: zeros) as two e4m3 rows under one
// power-of-two scale, which is returned (NaN for a row that is not finite,
// whose codes are 0): eight lanes a row, D / 8 values each.
template <int D>
__device__ float split_row(const __nv_bfloat16 *src, uint8_t *hi, uint8_t *lo, bool value) {
    constexpr int E = D / 8;
    const int sub = threadIdx.x & 7;
    float x[E];
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < E; e += 8) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (src) v = *reinterpret_cast<const uint4 *>(src + sub * E + e);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[e + 2 * i] = __uint_as_float(w[i] << 16);
            x[e + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            amax = max(amax, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
        }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const bool bad = amax >= 0x7f800000u;
    // 2^e: the largest value lies in (224, 448] of it (or below: 1 / 2^e times P
    // adds up to a row's sum, which has to stay finite)
    const int e = min(max((int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0),
                          value ? -100 : -110), 119);
    const float r = bad ? 0.f : exp2_int(-e);
    uint32_t h[E / 4], w[E / 4];
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        const float a = bad ? 0.f : x[i] * r, b = bad ? 0.f : x[i + 1] * r;
        const float c = bad ? 0.f : x[i + 2] * r, d = bad ? 0.f : x[i + 3] * r;
        const uint32_t p = e4m3x2(a, b), q = e4m3x2(c, d);
        const float2 f = from_e4m3x2(p), g = from_e4m3x2(q);
        h[i / 4] = p | (q << 16);
        w[i / 4] = e4m3x2(a - f.x, b - f.y) | (e4m3x2(c - g.x, d - g.y) << 16);
    }
    if constexpr (E == 16) {
        *reinterpret_cast<uint4 *>(hi + sub * E) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(lo + sub * E) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *reinterpret_cast<uint2 *>(hi + sub * E) = make_uint2(h[0], h[1]);
        *reinterpret_cast<uint2 *>(lo + sub * E) = make_uint2(w[0], w[1]);
    }
    if (bad) return __uint_as_float(0x7fffffffu);
    // (a value row of zeros must not raise its readers' references)
    return amax == 0 && value ? exp2_int(kKv8MinExp) : exp2_int(e);
}

// Eight lanes a row: the query rows of every unit, then the tail's tokens
// (soft prompt first), a key row and a value row each.  It lets the attention
// kernel start at once: that one waits for it only where it reads these rows.
template <int D>
__global__ void __launch_bounds__(256) attn_kv8_prep_kernel(const __grid_constant__ Prep8Params P) {
    pdl_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const AttnParams &A = P.t.a;
    if ((int)blockIdx.x < P.plan_ctas) {
        // a warp each: a CTA's range, and its record for the merge
        const TcParams &T = P.t;
        const int cta = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
        if (cta < T.n_ctas) {
            const WarpSched ws = warp_sched(T);
            // its last position first, then its first (as sched_range_lo, which
            // does not say in which unit that is)
            int b = 0, S = 0, nt = 0, seg = 0, tile = 0;
            long long lo = ws.T, hi = ws.T, t0, c0 = 0;
#pragma unroll 1
            for (int i = cta + 1 == T.n_ctas ? cta : cta + 1; i >= cta; --i) {
                hi = lo;
                const long long x = div_nn(ws.C * i, T.n_ctas);
                sched_locate(T, ws, x, true, b, t0, c0, S);
                nt = seg_tiles(T, S);
                seg = (int)div_nn(x - c0, nt + T.seg_cost);
                const long long off = x - c0 - (long long)seg * (nt + T.seg_cost);
                tile = off > T.seg_cost ? (int)off - T.seg_cost : 0;
                lo = t0 + (long long)seg * nt + tile;
            }
            const int h = seg / T.seg_rb, rb = seg - h * T.seg_rb;
            if (lane < 2)
                reinterpret_cast<int4 *>(P.plan + cta)[lane] =
                    lane == 0 ? make_int4((int)(hi - lo), b, h, rb) : make_int4(S, nt, tile, 0);
            if (lane == 0) {
                T.bounds[cta] = lo;
                if (cta == T.n_ctas - 1) T.bounds[cta + 1] = ws.T;
            }
            const BoundaryRec rec =
                boundary_record(T, ws, cta, lo, hi, (b * T.seg_h + h) * T.seg_rb + rb, tile, nt,
                                c0 + (long long)seg * (nt + T.seg_cost));
            if (lane == 0) T.recs[cta] = rec;
        }
        if (blockIdx.x == 0)
            for (int b = threadIdx.x; b < A.B; b += 256) check_seq_len(A, b);
        return;
    }
    const int w = ((int)blockIdx.x - P.plan_ctas) * 32 + (threadIdx.x >> 3);
    const int sub = threadIdx.x & 7;
    const int q_pad = (P.q_rows + 3) & ~3;                // (a warp's four rows are of one kind)
    if (w < q_pad) {
        const bool real = w < P.q_rows;
        const unsigned at = real ? w : P.q_rows - 1, u = at / P.rb, r = at % P.rb;
        const unsigned bh = u / P.seg_rb;
        const int rb = (int)(u % P.seg_rb), h = (int)(bh % A.Hkv), b = (int)(bh / A.Hkv);
        const int p = rb * P.rb + (int)r;
        const __nv_bfloat16 *src = nullptr;
        RowMeta m{0.f, -1};
        if (p < A.M) {
            const int rr = p / A.G, hq = h * A.G + p % A.G, row = rr * A.Hq + hq;
            src = static_cast<const __nv_bfloat16 *>(A.q) + ((size_t)b * A.R * A.Hq + row) * D;
            m.out = 2 * row + (A.row_flags[(size_t)b * A.R + rr] & SPEC_ROW_VALID ? 1 : 0);
        }
        uint8_t *dst = P.q8 + ((size_t)u * 2 * P.rb + r) * D;
        m.scale = split_row<D>(src, dst, dst + (size_t)P.rb * D, false) * A.scale_log2;
        if (sub == 0 && real) P.q_meta[at] = m;
        return;
    }
    const unsigned t = min(w - q_pad, P.t_rows - 1), bh = t / P.tail_pad;
    const int tt = (int)(t % P.tail_pad), h = (int)(bh % A.Hkv);
    const __nv_bfloat16 *k = nullptr, *v = nullptr;
    if (tt < A.n_soft) {
        const size_t at = ((size_t)h * A.n_soft + tt) * D;
        k = static_cast<const __nv_bfloat16 *>(A.soft_k) + at;
        v = static_cast<const __nv_bfloat16 *>(A.soft_v) + at;
    } else if (tt - A.n_soft < A.R) {
        const size_t at = ((size_t)bh * A.R + tt - A.n_soft) * D;
        k = static_cast<const __nv_bfloat16 *>(A.kb) + at;
        v = static_cast<const __nv_bfloat16 *>(A.vb) + at;
    }
    uint8_t *hi = P.tail8 + (size_t)bh * 2 * (2 * P.tail_pad * D);
    uint8_t *lo = hi + (size_t)2 * P.tail_pad * D;
    const int ko = kv8_row(tt, 0, D), vo = kv8_row(tt, 1, D);
    const float sk = split_row<D>(k, hi + ko, lo + ko, false);
    const float sv_ = split_row<D>(v, hi + vo, lo + vo, true);
    if (sub == 0) P.tail_scale[t] = make_float2(sk, sv_);
}

// ------------------------------------------------------------------ host

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Offsets of the workspace's parts.
struct Ws8 {
    size_t o, ml, bounds, recs, plan, q8, q_meta, tail8, tail_scale, bytes;
    int n_ctas, rb, seg_rb, tail_pad;
    long long units;
};

Ws8 plan_ws(const AttnParams &A) {
    Ws8 w{};
    w.n_ctas = num_sms();
    w.rb = kv8_tc_rows(A);
    w.seg_rb = ceil_div(A.M, w.rb);
    w.units = (long long)A.B * A.Hkv * w.seg_rb;
    w.tail_pad = ceil_div(A.n_soft + A.R, 16) * 16;
    const size_t rows = ((size_t)w.units + w.n_ctas) * w.rb;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    w.o = take(rows * A.d * sizeof(float));
    w.ml = take(rows * 2 * sizeof(float));
    w.bounds = take(((size_t)w.n_ctas + 1) * sizeof(long long));
    w.recs = take((size_t)w.n_ctas * sizeof(BoundaryRec));
    w.plan = take((size_t)w.n_ctas * sizeof(CtaPlan));
    w.q8 = take((size_t)w.units * 2 * w.rb * A.d);
    w.q_meta = take((size_t)w.units * w.rb * sizeof(RowMeta));
    w.tail8 = take((size_t)A.B * A.Hkv * 4 * w.tail_pad * A.d);
    w.tail_scale = take((size_t)A.B * A.Hkv * w.tail_pad * sizeof(float2));
    w.bytes = at;
    return w;
}

template <int D, int RB>
spec_status_t launch_units(const Tc8Params &P, const CUtensorMap *m, cudaStream_t s) {
    const spec_status_t st =
        set_smem_limit(reinterpret_cast<const void *>(attn_kv8_tc_kernel<D, RB>), smem8<D, RB>());
    if (st != SPEC_OK) return st;
    return launch(attn_kv8_tc_kernel<D, RB>, dim3(P.t.n_ctas), dim3(Cfg<D, RB>::kThreads), smem8<D, RB>(), s, P,
                  m[0], m[1], m[2]);
}

template <int D>
spec_status_t launch_rows(const Tc8Params &P, const Prep8Params &R, const CUtensorMap *m, int rb,
                          cudaStream_t s) {
    const long long prep = ((R.q_rows + 3ll) & ~3ll) + R.t_rows;
    spec_status_t st = launch(attn_kv8_prep_kernel<D>, dim3((unsigned)(R.plan_ctas + ceil_div_ll(prep, 32))),
                              dim3(256), 0, s, R);
    if (st != SPEC_OK) return st;
    st = rb == 8    ? launch_units<D, 8>(P, m, s)
         : rb == 16 ? launch_units<D, 16>(P, m, s)
         : rb == 32 ? launch_units<D, 32>(P, m, s)
                    : launch_units<D, 64>(P, m, s);
    if (st != SPEC_OK) return st;
    if (P.t.n_ctas > 1)
        st = launch(attn_kv8_tc_combine_kernel<D>, dim3(P.t.n_ctas - 1, ceil_div(rb, 4)), dim3(128), 0,
                    s, P.t);
    return st != SPEC_OK ? st : launch_status();
}

}  // namespace

// Packed rows per unit: the fewest of 8, 16, 32 and 64 that hold a KV head's
// rows (a step's MMAs and softmax grow with them), 64-row blocks beyond.
int kv8_tc_rows(const AttnParams &P) { return P.M <= 8 ? 8 : P.M <= 16 ? 16 : P.M <= 32 ? 32 : 64; }

// TMA coordinates and unit numbers are 32-bit.
bool kv8_tc_supported(const AttnParams &P) {
    const Ws8 w = plan_ws(P);
    return w.units * 2 * w.rb < (1ll << 31) &&
           (long long)P.B * P.Hkv * 4 * w.tail_pad < (1ll << 31) && (long long)P.R * P.Hq < (1ll << 30);
}

size_t kv8_tc_workspace_bytes(const AttnParams &P) { return plan_ws(P).bytes; }

spec_status_t launch_attn_kv8_tc(const Kv8Params &Q, cudaStream_t s) {
    const Ws8 w = plan_ws(Q.a);
    char *base = reinterpret_cast<char *>(Q.a.part_o);
    Tc8Params P{};
    TcParams &T = P.t;
    T.a = Q.a;
    T.a.rb_rows = w.rb;
    T.a.n_rb = w.seg_rb;
    T.a.part_ml = reinterpret_cast<float *>(base + w.ml);
    T.n_ctas = w.n_ctas;
    T.bounds = reinterpret_cast<long long *>(base + w.bounds);
    T.recs = reinterpret_cast<BoundaryRec *>(base + w.recs);
    T.wait = wait_limit();
    T.seg_h = Q.a.Hkv;
    T.seg_rb = w.seg_rb;
    T.seg_cost = 4;
    T.pair_steps = 1;                       // a step: two of the schedule's 64-token tiles
    P.scales = Q.scales;
    P.q_meta = reinterpret_cast<const RowMeta *>(base + w.q_meta);
    P.tail_scale = reinterpret_cast<const float2 *>(base + w.tail_scale);
    P.tail_len = Q.a.n_soft + Q.a.R;
    P.tail_pad = w.tail_pad;
    P.n_tail = ceil_div(P.tail_len, kStep);
    T.tail = 2 * P.n_tail;
    P.box_log2 = 4;
    while ((1 << P.box_log2) < kStep && Q.a.page_size % (2 << P.box_log2) == 0) ++P.box_log2;
    P.ps16 = Q.a.page_size / 16;
    P.ps16_inv = ((1ull << 32) + P.ps16 - 1) / P.ps16;
    Prep8Params R{};
    R.plan = reinterpret_cast<CtaPlan *>(base + w.plan);
    R.plan_ctas = ceil_div(w.n_ctas, 8);
    P.plan = R.plan;
    R.t = T;
    R.q8 = reinterpret_cast<uint8_t *>(base + w.q8);
    R.q_meta = reinterpret_cast<RowMeta *>(base + w.q_meta);
    R.tail8 = reinterpret_cast<uint8_t *>(base + w.tail8);
    R.tail_scale = reinterpret_cast<float2 *>(base + w.tail_scale);
    R.rb = w.rb;
    R.seg_rb = w.seg_rb;
    R.tail_pad = w.tail_pad;
    R.q_rows = (int)(w.units * w.rb);
    R.t_rows = Q.a.B * Q.a.Hkv * w.tail_pad;

    const int D = Q.a.d, ps = Q.a.page_size;
    CUtensorMap m[3];
    // the cache as [page x head][rows: 8 keys, 8 values, ...][D]
    const cuuint64_t d0[3] = {(cuuint64_t)D, (cuuint64_t)2 * ps, (cuuint64_t)Q.a.n_pages * Q.a.Hkv};
    const cuuint64_t s0[2] = {(cuuint64_t)D, (cuuint64_t)2 * ps * D};
    const cuuint32_t b0[3] = {(cuuint32_t)D, (cuuint32_t)(2 << P.box_log2), 1u};
    const cuuint64_t s1[1] = {(cuuint64_t)D};
    const cuuint64_t d1[2] = {(cuuint64_t)D, (cuuint64_t)Q.a.B * Q.a.Hkv * 4 * w.tail_pad};
    const cuuint32_t b1[2] = {(cuuint32_t)D, 32u};
    const cuuint64_t d2[2] = {(cuuint64_t)D, (cuuint64_t)w.units * 2 * w.rb};
    const cuuint32_t b2[2] = {(cuuint32_t)D, (cuuint32_t)(2 * w.rb)};
    if (!encode_u8_map(&m[0], Q.a.kc, 3, d0, s0, b0) || !encode_u8_map(&m[1], R.tail8, 2, d1, s1, b1) ||
        !encode_u8_map(&m[2], R.q8, 2, d2, s1, b2))
        return SPEC_ERR_CUDA;
    return D == 128 ? launch_rows<128>(P, R, m, w.rb, s) : launch_rows<64>(P, R, m, w.rb, s);
}

}  // namespace sv
