// Tensor-core chunk attention (bf16 rows), over a bf16 cache or one in 8 bits.
//
// For each row, running over the keys once: S = q K^T (tcgen05, fp32), P = exp2(S
// scale log2(e) - m), l += sum P in fp32, O += P V (tcgen05, fp32) with P rounded
// to bf16, as the MMA wants it beside bf16 values (half a step, 2^-8 of a weight);
// o = O / l, lse = (m + log2 l) ln 2.
//
// Design (GB300, tcgen05):
// * A unit is 2 TB consecutive new tokens of one (request, KV head), TB =
//   128 / G: two query tiles A and B of up to 128 packed rows (row t G + g:
//   token t, query head g of the group), which share every K/V tile.  The
//   persistent grid, one CTA per SM, takes equal shares of the call's cost, cut
//   at 128-key steps (chunk_attn.cuh), so single tokens behind long histories
//   and long prompts fill the GPU alike.
//   A request whose rows fit one tile (single tokens among them) has units of two
//   KV heads instead, a tile and a stream of K/V tiles each.
// * Warps 0-3 run the softmax of tile A and 4-7 that of tile B, one row a
//   thread; warp 8 copies the units' queries and the cache's tiles, warps 9 and
//   10 issue the MMAs of tiles A and B from one thread each -- PV(j), S(j+1), PV
//   (j+1), .. -- so that the tensor core works on one tile while the other's
//   softmax, or its change of unit, runs.
// * bf16 cache: K and V tiles come by tensor copies, one a page (contiguous, or D =
//   64: one a tile or page and 64 elements), into a ring of 128-byte-swizzled
//   slots.  Warp 11 looks through the value tiles that not every row sees whole
//   (the last ones of a unit): rows past the unit's last token become zeros, and
//   non-finite values too, whose first place they note, for a hidden value's
//   weight of zero would not keep it out of the sum.
// * 8-bit cache: 16 tokens' codes, keys and values, are one run of memory, which
//   a bulk copy brings into a stage; warps 12-19 turn them into the slots' bf16
//   tiles (code * scale, exact for a power of two) and do what warp 11 does
//   on the way.
// * Softmax and TMEM as in the prefill kernel: O (fp32) and S of a tile side by
//   side, P (bf16) over the first half of S, the running maximum raised only
//   when it grows by more than 2^8.
// * A tile's whole rows leave by tensor copies through the place of its queries;
//   the last tokens' and a part's fp32 rows as whole lines by their warps.
// * Every wait is bounded; on expiry the kernel sets SPEC_DEV_TIMEOUT, stops
//   issuing work, waits (bounded) for its own copies and MMAs, frees its TMEM
//   and returns.
//
// What it measures, and what bounds it (heads of 128, the merging launch included;
// a graph's passes over one input -- of calls one by one, on inputs that change, the
// first three take 4.0 ms, 372 and 203 us, 1230, 976 and 700 TFLOP/s):
// * Three chunks of 1.5 - 2 K tokens behind 45 - 66 K, 32 heads over 8: 3.8 - 3.9
//   ms, 1250 - 1290 TFLOP/s.  The MMAs of a 128-key step of both tiles take 2.08 K
//   cycles of 3.1 K: a tile's chain of softmax, PV and next S is longer than the
//   other's MMAs, and the clock gives way to the power limit.
// * Whole prompts, 12.9 K tokens of 32 heads: 346 us (1050 TFLOP/s): a unit's start,
//   its last (masked) steps with their value check and its results, against 2 to 32
//   steps, and the merging launch (11).  What runs once a unit or less is kept in
//   rolled loops: unrolled it has to be fetched each time, beside the steps' code.
// * 39 single tokens and 9 chunks up to 512, behind 0.6 - 4 K: 191 us, of 79 for
//   the bytes and 75 for the products: a CTA streams for single tokens, G rows of
//   128 in a tile, or computes for the others, not both.  48 single tokens behind
//   4 K: 133 us, 89 % of a copy's rate, in pages of any size.
// * 8 bits: 4.9 ms and 290 us on the first and third: the codes' widening (two
//   tiles of 16 K elements a step, 8 warps) shares issue slots and shared memory
//   with the softmax.  MMAs on the codes themselves would need none, but queries
//   as two e4m3 values and P as three of e5m2, 2.5 products at twice the rate in
//   the place of one, and the splitting of P in the softmax's chain.
#include "chunk_attn.cuh"
#include "chunk_ring.cuh"
#include "kv8_common.cuh"
#include "ptx_sm103.cuh"

namespace sv {
namespace {

namespace ctc {

constexpr int kM = 128;                  // rows of a query tile
constexpr int kN = 128;                  // keys of a step
constexpr int kHalf = 128 * 128;         // 128 rows x 64 bf16
constexpr int kGroupWarps = 4;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;              // and 10
constexpr int kFixWarp = 11;             // bf16 cache
constexpr int kConvWarp = 12;            // 8-bit cache: 12 .. 19
constexpr int kConvWarps = 8;
constexpr int kTmemCols = 512;
constexpr int kParts = 8;                // parts announced ahead
// K/V pairs of a part that are copied before its queries: their slots (two each)
// or stages are free of it, so they come free without its queries.
constexpr int kAhead = 2;
__host__ __device__ constexpr uint32_t col_o(int x) { return 256u * (uint32_t)x; }
__host__ __device__ constexpr uint32_t col_s(int x) { return 256u * (uint32_t)x + 128u; }
constexpr float kRescale = 8.f;          // log2 growth allowed before rescaling
constexpr int kMaxSlots = 12, kMaxStages = 4;

// Sizes by head_dim and cache.  Registers: the launch gives every thread
// kLaunchRegs, the softmax warpgroups raise theirs and the others lower; the
// sum must fit the launch's, or the raise would wait forever.
template <int D, bool K8>
struct Cfg {
    static constexpr int NH = D / 64;
    static constexpr int kTile = NH * kHalf;             // a Q, K or V tile
    static constexpr int kSlots = D == 128 ? (K8 ? 3 : 5) : 8;
    static constexpr int kStages = K8 ? (D == 128 ? 2 : 4) : 0;
    static constexpr int kStage = 2 * kN * D;            // codes of a step, K and V
    static_assert(K8 ? kAhead <= kStages && kSlots >= 3 : 2 * kAhead < kSlots, "steps ahead of their queries");
    static constexpr int kWarps = K8 ? 20 : 12;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kLaunchRegs = K8 ? 96 : 168;
    static constexpr int kSoftmaxRegs = K8 ? 136 : 184;
    static constexpr int kOtherRegs = K8 ? 64 : 128;
    static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs,
                  "register split exceeds the launch allocation");
};

struct Params {
    ChunkParams c;
    int tb;                  // tokens of a query tile
    uint32_t g_mul;          // r / G = (r g_mul) >> 16, r < 128
    int box;                 // tokens of a tensor copy (paged: of one page)
    uint32_t ps_mul;         // t / ps = (t ps_mul) >> ps_shift, t < 2^31
    int ps_shift;
};

// A CTA's part of a unit, as the producer announces it: n steps of 128 keys from
// s0 on, of which tile x takes the first n_t[x] (tile A's rows may see fewer
// tokens).  A step brings `sets` pairs of a K and a V tile: one for both query
// tiles, or, in a unit of two heads, one for each.
struct Part {
    int n;                   // 0: no more parts
    int s0;
    int b, sets;
    int h[2];                // KV head of each tile
    int row[2];              // its first token's packed row
    int pos[2];              // and position: it sees pos + 1 tokens
    int nt[2], n_t[2];       // its tokens and steps
    int lim;                 // tokens that the unit's last one sees
    int slot;                // where a part that is not a whole unit goes; -1: whole
};

struct Shared {
    uint64_t part_full[kParts], part_free[kParts];
    uint64_t q_full[2], q_empty[2];
    uint64_t full[kMaxSlots], empty[kMaxSlots], fixed[kMaxSlots];
    uint64_t st_full[kMaxStages], st_empty[kMaxStages];
    uint64_t s_full[2], p_full[2][2], o_done[2], o_free[2], o_ready[2];      // p_full: by halves of the keys
    uint64_t drain[2];
    uint32_t tmem_base;
    uint32_t issued;         // fills of the ring begun
    int mma_busy;            // whether a tile's MMAs are being issued
    int abort;
    int bad[kParts][2 * kConvWarps];     // by part, looking warp and set: first token with a non-finite value
    Part parts[kParts];
    ChunkShare share;
};

template <int D, bool K8>
constexpr size_t smem_bytes() {
    using C = Cfg<D, K8>;
    return (size_t)(2 + C::kSlots) * C::kTile + (size_t)C::kStages * C::kStage + sizeof(Shared) + 1024;
}

__device__ __forceinline__ Part part_of(const Params &P, const ChunkPart &u) {
    Part t;
    const int tok = u.paired ? 0 : u.j * 2 * P.tb;
    t.n = u.s1 - u.s0;
    t.s0 = u.s0;
    t.b = u.b;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int tx = u.paired ? 0 : tok + x * P.tb;
        t.h[x] = u.paired ? 2 * u.h + x : u.h;
        t.row[x] = u.first + tx;
        t.pos[x] = u.S + tx;
        t.nt[x] = u.paired && t.h[x] >= P.c.Hkv ? 0 : max(0, min(P.tb, u.n - tx));
        const int end = (t.pos[x] + t.nt[x] + kN - 1) / kN;            // its last row's steps
        t.n_t[x] = t.nt[x] > 0 ? max(0, min(u.s1, end) - u.s0) : 0;
    }
    t.sets = u.paired && t.nt[1] > 0 ? 2 : 1;
    t.lim = max(t.pos[0] + t.nt[0], t.nt[1] > 0 ? t.pos[1] + t.nt[1] : 0);
    t.slot = u.s0 == 0 && u.s1 == u.steps ? -1 : chunk_slot(u);
    return t;
}

// Whether step s holds tokens that some row of the unit does not see.
__device__ __forceinline__ bool ragged(const Part &t, int s) { return (s + 1) * kN > t.pos[0] + 1; }

template <bool V> struct Bool { static constexpr bool value = V; };

// A reader's view of the announced parts.
struct PartReader {
    int i = 0;
    uint32_t ph = 0;
    // Waits for the next part (the whole warp, or one thread alone), which is
    // sh.parts[i] until it is let go of; false when there is none, *ok = false when
    // the wait ran out.
    template <bool kWarp>
    __device__ __forceinline__ bool next(Shared &sh, long long limit, bool *ok) {
        if (!(kWarp ? mbar_wait_warp(&sh.part_full[i], ph, limit) : mbar_wait(&sh.part_full[i], ph, limit))) {
            *ok = false;
            return false;
        }
        return sh.parts[i].n > 0;
    }
    // Lets go of the part (the whole warp, or one thread alone), which the producer
    // may then overwrite: a warp's lanes have all read what they need of it first.
    template <bool kWarp>
    __device__ __forceinline__ void release(Shared &sh) {
        if (kWarp) __syncwarp();
        if (!kWarp || (threadIdx.x & 31) == 0) mbar_arrive(&sh.part_free[i]);
    }
    __device__ __forceinline__ void advance() {
        if (++i == kParts) {
            i = 0;
            ph ^= 1u;
        }
    }
};

__device__ __forceinline__ int page_of(const Params &P, int t) {
    return (int)(((uint64_t)(uint32_t)t * P.ps_mul) >> P.ps_shift);
}

// 16 bytes of eight bf16: whether one of them is not finite.
__device__ __forceinline__ bool odd8(const uint4 &v) {
    const uint32_t m = 0x7f807f80u, one = 0x00800080u;
    return ((((v.x & m) + one) | ((v.y & m) + one) | ((v.z & m) + one) | ((v.w & m) + one)) & 0x80008000u) != 0;
}

// a * 0 + c of two bf16
__device__ __forceinline__ uint32_t times0(uint32_t a, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(0u), "r"(c));
    return d;
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A word of shared memory that one thread counts up and others look at.
__device__ __forceinline__ void store_release(uint32_t *p, uint32_t x) {
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(p)), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t load_acquire(const uint32_t *p) {
    uint32_t x;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(x) : "r"(smem_u32(p)) : "memory");
    return x;
}

// global -> shared bulk copy; both 16-byte aligned, bytes a multiple of 16
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// shared -> global tensor copy, and the wait until this thread's have read their
// source
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit_and_wait_read() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Four e4m3 codes as bf16 times 2^-120: sign, and exponent and mantissa in the
// low bits of bf16's (subnormal codes become subnormal).  NaN codes are not
// told apart.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
    return make_uint2((a & 0x80008000u) | ((a >> 4) & 0x07f007f0u), (b & 0x80008000u) | ((b >> 4) & 0x07f007f0u));
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 16 codes times 2^e as bf16; m: the bf16 pair 2^(120 + e).  Exact.
__device__ __forceinline__ void widen16(const uint4 &codes, uint32_t m, uint4 &lo, uint4 &hi) {
    const uint2 a = widen4(codes.x), b = widen4(codes.y), c = widen4(codes.z), d = widen4(codes.w);
    lo = make_uint4(mul2(a.x, m), mul2(a.y, m), mul2(b.x, m), mul2(b.y, m));
    hi = make_uint4(mul2(c.x, m), mul2(c.y, m), mul2(d.x, m), mul2(d.y, m));
}

// The same with any scale, and NaN codes.
__device__ __forceinline__ void widen16_any(const uint4 &codes, float scale, uint4 &lo, uint4 &hi) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = from_e4m3x2(w[i] & 0xffffu), b = from_e4m3x2(w[i] >> 16);
        out[2 * i] = pack_bf16(a.x * scale, a.y * scale);
        out[2 * i + 1] = pack_bf16(b.x * scale, b.y * scale);
    }
    lo = make_uint4(out[0], out[1], out[2], out[3]);
    hi = make_uint4(out[4], out[5], out[6], out[7]);
}

// Whether a NaN code is among the four (0x7f of its low seven bits).
__device__ __forceinline__ uint32_t nan4(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }

}  // namespace ctc

// kJoint (pages of the bf16 cache, D = 128): the K and V tiles' 64-element halves
// lie side by side, eight tokens of the one, then of the other, so that a page
// comes in one copy; a copy costs the producer its issue, whatever its size (48
// single tokens behind 4 K in pages of 16: 152 -> 133 us).  half_at, group_at: bytes
// between the halves, and between groups of eight tokens.
template <int D, bool K8, bool kJoint>
__global__ void __launch_bounds__(ctc::Cfg<D, K8>::kThreads, 1)
chunk_tc_kernel(const __grid_constant__ ctc::Params P, const __grid_constant__ CUtensorMap mq,
                const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv) {
    using namespace ctc;
    using namespace tc5;
    using C = Cfg<D, K8>;
    constexpr int NH = C::NH, kTile = C::kTile, kSlots = C::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = smem;                                // query tiles A and B
    uint8_t *ring = smem + 2 * kTile;                    // kSlots K / V tiles
    uint8_t *stages = ring + kSlots * kTile;             // 8 bits: codes
    Shared &sh = *reinterpret_cast<Shared *>(stages + C::kStages * C::kStage);
    const ChunkParams &A = P.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    constexpr uint32_t half_at = kJoint ? 1024u : (uint32_t)kHalf, group_at = kJoint ? 2048u : 1024u;

    if (threadIdx.x == kProducerWarp * 32) {
        const CUtensorMap *maps[4] = {&mq, &mo, &mk, &mv};
        for (int i = 0; i < (K8 ? 2 : 4); ++i)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[i]))
                         : "memory");
    }
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sh.q_full[x], 1);
            mbar_init(&sh.q_empty[x], kGroupWarps);
            mbar_init(&sh.s_full[x], 1);
            mbar_init(&sh.p_full[x][0], kGroupWarps);
            mbar_init(&sh.p_full[x][1], kGroupWarps);
            mbar_init(&sh.o_done[x], 1);
            mbar_init(&sh.o_free[x], kGroupWarps);
            mbar_init(&sh.o_ready[x], kGroupWarps);
            mbar_init(&sh.drain[x], 1);
        }
        for (int i = 0; i < kParts; ++i) {
            mbar_init(&sh.part_full[i], 1);
            mbar_init(&sh.part_free[i], 8 + 2 + (K8 ? kConvWarps : 1));  // softmax, MMA, and warp 11 or 12 on
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&sh.full[s], K8 ? kConvWarps : 1);
            mbar_init(&sh.empty[s], K8 ? 2 : 3);                     // MMA threads, warp 11
            mbar_init(&sh.fixed[s], 1);
        }
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&sh.st_full[s], 1);
            mbar_init(&sh.st_empty[s], kConvWarps);
        }
        sh.abort = 0;
        sh.issued = 0;
        sh.mma_busy = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // the rows of the query tiles that hold no query (128 is not a multiple of G)
    const int rows = P.tb * A.G;
    for (int i = threadIdx.x; i < (kM - rows) * 2 * NH * 8; i += C::kThreads) {
        const int r = rows + i / (2 * NH * 8), c = i % (2 * NH * 8);
        *reinterpret_cast<uint4 *>(qbuf + (c / 8) * kHalf + r * 128 + (c % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem_base)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    fence_before();
    chunk_share<C::kThreads>(A, sh.share);
    fence_after();
    const uint32_t tmem = sh.tmem_base;
    volatile int *abort = &sh.abort;
    const long long wait = A.wait;

    if (warp >= kProducerWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        if (warp == kProducerWarp) {
            // ------------------------------------------------------ producer
            // The whole warp walks; lane i issues copy i of a tile.
            // (evict-first for all: single tokens' keys and values are read once, and
            // those that units share are read again soon; against evict-last a mixed
            // batch takes 226 instead of 233 us, prompts 377 / 380, long chunks 3.74 /
            // 3.71 ms)
            const uint64_t pol = policy_evict_first();
            const int per = kN / P.box;                  // copies a tile, by tokens
            // rows cache: this lane's copy
            const int hh = kJoint ? 0 : lane % NH, bx = kJoint ? lane : lane / NH;
            const uint32_t copy_bytes = (uint32_t)P.box * (kJoint ? 256u : 128u);
            int slot = 0;                                // next slot (8 bits: stage)
            int nq[2] = {0, 0};                          // queries copied, per tile
            uint32_t ph = 1;                             // parity of its release
            long long ld = 0;                            // fills issued
            bool ok = true;
            ChunkWalk walk(A, sh.share);
            ChunkPart u;
            int pi = 0;                                  // next place for a part, and the
            uint32_t pph = 1;                            // parity of its release
            auto announce = [&](const Part &t) -> bool {
                if (!mbar_wait_warp(&sh.part_free[pi], pph, wait)) return false;
                if (lane == 0) {
                    sh.parts[pi] = t;
                    mbar_arrive(&sh.part_full[pi]);
                }
                if (++pi == kParts) {
                    pi = 0;
                    pph ^= 1u;
                }
                return true;
            };
            while (ok && walk.next(A, u)) {
                const Part t = part_of(P, u);
                if (__any_sync(0xffffffffu, *abort != 0) || !announce(t)) {
                    ok = false;
                    break;
                }
                // A tile's queries replace those of its part before, whose results
                // leave through their place, so their copy waits; the first steps'
                // K and V do not.
                uint32_t q_due = (t.n_t[0] > 0 ? 1u : 0u) | (t.n_t[1] > 0 ? 2u : 0u);
                auto load_q = [&](bool block) -> bool {
                    for (int x = 0; x < 2; ++x) {
                        if (!((q_due >> x) & 1u)) continue;
                        const uint32_t parity = (uint32_t)((nq[x] & 1) ^ 1);
                        if (block) {
                            if (!mbar_wait_warp(&sh.q_empty[x], parity, wait)) return false;
                        } else if (!__all_sync(0xffffffffu, mbar_test_wait(&sh.q_empty[x], parity))) {
                            continue;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&sh.q_full[x], (uint32_t)(NH * rows * 128));
                        __syncwarp();
                        if (lane < NH)
                            tma_load_3d(qbuf + x * kTile + lane * kHalf, &mq, lane * 64, t.h[x] * A.G, t.row[x],
                                        &sh.q_full[x], pol);
                        ++nq[x];
                        q_due &= ~(1u << x);
                    }
                    return true;
                };
                const int32_t *table = A.paged ? A.page_table + (size_t)u.b * A.max_pages : nullptr;
                // the page of this lane's copy, loaded a step ahead of its use
                const int at = K8 ? lane * 16 : bx * P.box;
                const bool mine = K8 ? lane < kN / 16 : bx < per;
                auto page_id = [&](int s) -> int {
                    const int tok = s * kN + at;
                    return A.paged && mine && s < u.s1 && tok < t.lim ? __ldg(table + page_of(P, tok)) : -1;
                };
                int next_id = page_id(u.s0), pairs = 0;
                for (int s = u.s0; s < u.s1 && ok; ++s) {
                    const int id = next_id, tok = s * kN + at;
                    next_id = page_id(s + 1);
                    bool in = mine && tok < t.lim;
                    if (in && A.paged && (id < 0 || id >= A.n_pages)) {
                        in = false;
                        raise_status(A.status, SPEC_DEV_BAD_PAGE);
                    }
                    const int off = A.paged ? tok - page_of(P, tok) * A.ps : tok;
                    const uint32_t n_in = (uint32_t)__popc(__ballot_sync(0xffffffffu, in));
                    for (int set = 0; set < t.sets && ok; ++set) {
                        const int h = t.h[set];
                        if (q_due && !load_q(pairs == kAhead)) {
                            ok = false;
                            break;
                        }
                        ++pairs;
                        if constexpr (K8) {
                            if (__any_sync(0xffffffffu, *abort != 0) || !mbar_wait_warp(&sh.st_empty[slot], ph, wait)) {
                                ok = false;
                                break;
                            }
                            if (lane == 0) mbar_arrive_expect_tx(&sh.st_full[slot], n_in * (32 * D));
                            __syncwarp();
                            if (in)
                                bulk_load(stages + slot * C::kStage + lane * (32 * D),
                                          static_cast<const uint8_t *>(A.kc) + kv8_block(id, h, A.Hkv, A.ps, D) +
                                              (size_t)off * (2 * D),
                                          32 * D, &sh.st_full[slot]);
                            ++ld;
                            if (++slot == C::kStages) {
                                slot = 0;
                                ph ^= 1u;
                            }
                        } else {
                            for (int kv = 0; kv < 2; ++kv) {
                                if (__any_sync(0xffffffffu, *abort != 0) ||
                                    !mbar_wait_warp(&sh.empty[slot], ph, wait)) {
                                    ok = false;
                                    break;
                                }
                                if (lane == 0) {
                                    mbar_arrive_expect_tx(&sh.full[slot], n_in * copy_bytes);
                                    store_release(&sh.issued, (uint32_t)ld + 1u);
                                }
                                __syncwarp();
                                uint8_t *dst = ring + slot * kTile + hh * kHalf + bx * copy_bytes;
                                if (in && kJoint)
                                    tma_load_5d(dst, kv ? &mv : &mk, 0, 0, 0, off >> 3, id * A.Hkv + h,
                                                &sh.full[slot], pol);
                                else if (in && A.paged)
                                    tma_load_3d(dst, kv ? &mv : &mk, 0, off, (id * A.Hkv + h) * NH + hh,
                                                &sh.full[slot], pol);
                                else if (in)
                                    tma_load_3d(dst, kv ? &mv : &mk, hh * 64, tok, t.b * A.Hkv + h, &sh.full[slot],
                                                pol);
                                ++ld;
                                if (++slot == kSlots) {
                                    slot = 0;
                                    ph ^= 1u;
                                }
                            }
                        }
                    }
                }
                ok = ok && load_q(true);
            }
            if (ok) {
                Part none{};
                ok = announce(none);
            }
            if (lane == 0) {
                if (!ok) {
                    raise_status(A.status, SPEC_DEV_TIMEOUT);
                    *abort = 1;
                }
                // do not leave while copies into this CTA's shared memory are in
                // flight (earlier ones were consumed, hence complete)
                constexpr int kFills = K8 ? C::kStages : kSlots;
                uint64_t *bars = K8 ? sh.st_full : sh.full;
                for (long long i = ld - 1; i >= 0 && i >= ld - kFills; --i)
                    if (!mbar_wait(&bars[i % kFills], (uint32_t)((i / kFills) & 1))) {
                        raise_status(A.status, SPEC_DEV_TIMEOUT);
                        break;
                    }
                for (int x = 0; x < 2; ++x)
                    if (nq[x] > 0 && !mbar_wait(&sh.q_full[x], (uint32_t)((nq[x] - 1) & 1)))
                        raise_status(A.status, SPEC_DEV_TIMEOUT);
            }
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // -------------------------------------------- MMA issuer of tile x
            if (lane == 0) {
                const int x = warp - kMmaWarp;
                const uint32_t id_s = idesc(kM, kN, false, false);
                const uint32_t id_pv = idesc(kM, D, false, true);
                const uint32_t tO = tmem + col_o(x), tS = tmem + col_s(x);
                const uint64_t qd = smem_desc(smem_u32(qbuf + x * kTile), 16, 1024);
                // descriptors of slot 0 (K: K-major, V: MN-major); a slot is kTile
                // further, i.e. kTile >> 4 in the address field
                const uint64_t kd0 = smem_desc(smem_u32(ring), 16, group_at);
                const uint64_t vd0 = smem_desc(smem_u32(ring), half_at, group_at);
                uint32_t base = 0;                       // fills of the ring before this part
                uint32_t known = 0;                      // and how many are known to have begun
                uint32_t np = 0, nact = 0;               // P hand-offs taken; parts with this tile
                bool ok = true;
                PartReader reader;
                while (ok && reader.next<false>(sh, wait, &ok)) {
                    const Part &t = sh.parts[reader.i];
                    const int n = t.n_t[x], sets = t.sets, other = sets == 2 ? 0 : t.n_t[1 - x];
                    const uint32_t fills = 2u * (uint32_t)(t.n * sets);
                    const int sure = t.pos[0] + 1 - t.s0 * kN;       // tokens that every row sees, from s0 on
                    reader.release<false>(sh);
                    reader.advance();
                    // fill of step j's K tile; its V tile is the next one
                    auto fill = [&](int j) -> uint32_t {
                        return base + 2u * (uint32_t)(j * sets + (sets == 2 ? x : 0));
                    };
                    // A slot's phase tells fill f by its parity alone, once the fill before it
                    // in the slot has landed: until then the phase two back has the same
                    // parity, and the old tile would pass for the new one.  The producer
                    // begins f when that fill has been let go of by all, so what is known to
                    // have begun may be waited for, on `full` or `fixed` (chunk_ring.cuh).
                    auto begun_now = [&](uint32_t f) -> bool {
                        if (known <= f) known = load_acquire(&sh.issued);
                        return known > f;
                    };
                    auto begun = [&](uint32_t f) -> bool {
                        const long long since = clock64();
                        while (!begun_now(f)) {
                            if (clock64() - since >= wait) return false;
                            __nanosleep(20);
                        }
                        return true;
                    };
                    // a slot is free once both threads have let go of it: each for
                    // itself, and for the other where that one has no use for it
                    auto release = [&](uint32_t slot, int j) {
                        commit(&sh.empty[slot]);
                        if (j >= other) mbar_arrive(&sh.empty[slot]);
                    };
                    // PV(j) and S(j + 1) of one tile are issued together, not in turns
                    // with the other's: interleaved, both come late, and the softmaxes
                    // that follow both run at once, with the tensor core idle (long
                    // chunks 4.14 -> 3.72 ms).
                    // (Over the 8-bit cache the codes' widening is what takes the time, and
                    // turns cost more than they give: 5.54 against 5.44 ms on long chunks.)
                    auto lock = [&]() -> bool {
                        if (K8) return true;
                        const long long since = clock64();
                        while (atomicExch(&sh.mma_busy, 1) != 0) {
                            if (clock64() - since >= wait) return false;
                            __nanosleep(20);
                        }
                        return true;
                    };
                    auto unlock = [&]() {
                        if (!K8) *(volatile int *)&sh.mma_busy = 0;
                    };
                    auto issue_s = [&](int j, bool locked) -> bool {
                        const uint32_t f = fill(j), slot = f % kSlots;
                        const bool ask = chunk_ring_asks(K8, j == 0);
                        if ((ask && !begun_now(f)) || !mbar_test_wait(&sh.full[slot], (f / kSlots) & 1u)) {
                            if (locked) unlock();
                            locked = false;
                            if ((ask && !begun(f)) || !mbar_wait(&sh.full[slot], (f / kSlots) & 1u, wait))
                                return false;
                        }
                        if (!locked && !lock()) return false;
                        fence_after();
                        const uint64_t kd = kd0 + (uint64_t)(slot * (kTile >> 4));
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint64_t q_off = (uint64_t)((((ks >> 2) * kHalf) + (ks & 3) * 32) >> 4);
                            const uint64_t k_off = (uint64_t)(((ks >> 2) * half_at + (ks & 3) * 32) >> 4);
                            mma_ss(tS, qd + q_off, kd + k_off, id_s, ks > 0 ? 1u : 0u);
                            // (a little ahead, as the queue holds some: after 2 / 4 / 6 / 8 of
                            // 8, whole prompts 358 / 347 / 342 / 347 us)
                            if (ks == (D == 128 ? 5 : 3)) unlock();
                        }
                        commit(&sh.s_full[x]);
                        release(slot, j);
                        return true;
                    };
                    if (n > 0) {
                        if (*abort || !begun(fill(0)) || !mbar_wait(&sh.q_full[x], nact & 1u, wait) ||
                            !issue_s(0, false)) {
                            ok = false;
                            break;
                        }
                    }
                    for (int j = 0; j < n; ++j) {
                        // O += P V, by halves of the keys as P comes; the part's first
                        // overwrites O, after the epilogue of the part before read it
                        const uint32_t f = fill(j) + 1u, slot = f % kSlots;
                        uint64_t *bar = !K8 && (j + 1) * kN > sure ? &sh.fixed[slot] : &sh.full[slot];
                        if ((chunk_ring_asks(K8, false) && !begun(f)) || !mbar_wait(bar, (f / kSlots) & 1u, wait) ||
                            (j == 0 && nact > 0 && !mbar_wait(&sh.o_free[x], (nact - 1) & 1u, wait))) {
                            ok = false;
                            break;
                        }
                        const uint64_t vd = vd0 + (uint64_t)(slot * (kTile >> 4));
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (!mbar_wait(&sh.p_full[x][half], np & 1u, wait) || (half == 0 && !lock())) {
                                ok = false;
                                break;
                            }
                            fence_after();
#pragma unroll
                            for (int ks = half * (kN / 32); ks < (half + 1) * (kN / 32); ++ks)
                                mma(tO, tS + ks * 8, vd + (uint64_t)((ks * 2 * group_at) >> 4), id_pv,
                                    (ks > 0 || j > 0) ? 1u : 0u);
                        }
                        if (!ok) break;
                        ++np;
                        if (j + 1 == n) commit(&sh.o_done[x]);
                        release(slot, j);
                        if (j + 1 == n) {
                            unlock();
                        } else if (!issue_s(j + 1, true)) {
                            ok = false;
                            break;
                        }
                    }
                    if (n > 0) ++nact;
                    base += fills;
                }
                if (!ok) {
                    raise_status(A.status, SPEC_DEV_TIMEOUT);
                    *abort = 1;
                }
                // every MMA issued above has completed before TMEM is released
                commit(&sh.drain[x]);
                if (!mbar_wait(&sh.drain[x], 0)) raise_status(A.status, SPEC_DEV_TIMEOUT);
            }
        } else if (!K8 && warp == kFixWarp) {
            // ------------------------- values that not every row sees, looked over
            // (The warp sees every fill of the ring, and releases it with the MMAs: one
            // that skipped fills could take an earlier phase for its own.)
            // this lane's vector of rows 0 .. 3 and of rows 4 .. 7 of an eight
            const uint32_t lo = (uint32_t)((lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4));
            const uint32_t hi = (uint32_t)((4 + (lane >> 3)) * 128 + (((lane & 7) ^ (4 + (lane >> 3))) << 4));
            int slot = 0;
            uint32_t ph = 0;
            bool ok = true;
            PartReader reader;
            while (ok && reader.next<true>(sh, wait, &ok)) {
                const Part &t = sh.parts[reader.i];
                int *bad = &sh.bad[reader.i][0];
                bool fresh = true;
                const int per = 2 * t.sets, n = per * t.n, s0 = t.s0;    // fills a step, of the part
                for (int i = 0; i < n; ++i) {
                    const int s = s0 + i / per;
                    if (__any_sync(0xffffffffu, *abort != 0) || !mbar_wait_warp(&sh.full[slot], ph, wait)) {
                        ok = false;
                        break;
                    }
                    if ((i & 1) && ragged(t, s)) {
                        if (fresh) {
                            if (lane < 2) bad[lane] = 0x7fffffff;
                            __syncwarp();
                            fresh = false;
                        }
                        uint8_t *v = ring + slot * kTile;
                        const int r0 = max(0, t.pos[0] + 1 - s * kN), r1 = max(0, min(kN, t.lim - s * kN));
                        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                        // past the last token: zeros
                        for (int g = r1 >> 3; g < kN / 8; ++g) {
                            for (int hh = 0; hh < NH; ++hh) {
                                uint8_t *p = v + hh * half_at + g * group_at;
                                if (8 * g + (lane >> 3) >= r1) *reinterpret_cast<uint4 *>(p + lo) = zero;
                                if (8 * g + 4 + (lane >> 3) >= r1) *reinterpret_cast<uint4 *>(p + hi) = zero;
                            }
                        }
                        // x * 0 + sum is NaN from the first x on that is not finite
                        uint32_t sum[8] = {};
#pragma unroll 4
                        for (int g = r0 >> 3; 8 * g < r1; ++g)
#pragma unroll
                            for (int hh = 0; hh < NH; ++hh) {
                                const uint8_t *p = v + hh * half_at + g * group_at;
                                const uint4 a = *reinterpret_cast<const uint4 *>(p + lo);
                                const uint4 b = *reinterpret_cast<const uint4 *>(p + hi);
                                sum[0] = times0(a.x, sum[0]);
                                sum[1] = times0(a.y, sum[1]);
                                sum[2] = times0(a.z, sum[2]);
                                sum[3] = times0(a.w, sum[3]);
                                sum[4] = times0(b.x, sum[4]);
                                sum[5] = times0(b.y, sum[5]);
                                sum[6] = times0(b.z, sum[6]);
                                sum[7] = times0(b.w, sum[7]);
                            }
                        uint32_t any = 0u;
#pragma unroll
                        for (int e = 0; e < 8; ++e) any |= sum[e] & 0x7fff7fffu;
                        if (__any_sync(0xffffffffu, any != 0u)) {
                            // (the tiles of a unit of two heads are noted apart)
                            int *mine = bad + (t.sets == 2 ? (i >> 1) & 1 : 0);
                            for (int r = r0; r < r1; ++r) {
                                if (lane >= NH * 8) continue;
                                uint4 *p = reinterpret_cast<uint4 *>(v + (lane >> 3) * half_at + (r >> 3) * group_at + (r & 7) * 128 +
                                                                     (((lane & 7) ^ (r & 7)) << 4));
                                if (!odd8(*p)) continue;
                                atomicMin(mine, s * kN + r);
                                *p = zero;
                            }
                        }
                        fence_async();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh.fixed[slot]);
                        mbar_arrive(&sh.empty[slot]);
                    }
                    if (++slot == kSlots) {
                        slot = 0;
                        ph ^= 1u;
                    }
                }
                reader.release<true>(sh);
                reader.advance();
            }
            if (!ok && lane == 0) {
                raise_status(A.status, SPEC_DEV_TIMEOUT);
                *abort = 1;
            }
        } else if (K8 && warp >= kConvWarp) {
            // ----------------------------------------- codes into bf16 tiles
            constexpr int kStages = C::kStages > 0 ? C::kStages : 1;
            constexpr int CPT = D / 16;              // 16-code vectors of a token
            constexpr int TPI = kConvWarps * 32 / CPT;   // tokens a round (32 or 64)
            constexpr int NI = kN / TPI;             // rounds
            const int tid = threadIdx.x - kConvWarp * 32;
            const int c = tid % CPT, tr = tid / CPT; // this thread's vector of tokens tr + i TPI
            // its codes in a stage (of the keys), and where they go in a tile: two
            // 16-byte chunks, which the lanes of a row's second half write in the
            // other order, so that eight lanes meet all banks
            const uint32_t from = (uint32_t)((tr >> 4) * (32 * D) + kv8_row(tr & 15, 0, D) + c * 16);
            const uint32_t to = (uint32_t)((c / 4) * kHalf + tr * 128);
            const uint32_t swap = c >= 4 ? 1u : 0u;
            const uint32_t at0 = to + (((2 * (c % 4) + swap) ^ (tr & 7)) << 4);
            const uint32_t at1 = to + (((2 * (c % 4) + 1 - swap) ^ (tr & 7)) << 4);
            int slot = 0, stage = 0;
            uint32_t fills = 0;
            uint32_t ph = 1, sph = 0;                // parity of the slot's release; of the stage's fill
            bool ok = true;
            PartReader reader;
            while (ok && reader.next<true>(sh, wait, &ok)) {
                const Part &t = sh.parts[reader.i];
                int *bad = &sh.bad[reader.i][2 * (warp - kConvWarp)];
                bool fresh = true;
                const int32_t *table = A.page_table + (size_t)t.b * A.max_pages;
                const int two = t.sets - 1, n_pairs = t.n << two;    // K/V pairs
                // scales of a pair's eight groups of 16 tokens: lane 2 g + x has group
                // g's of K (x = 0) or V.  Loaded a pair ahead, their pages' ids two: a
                // warp waits where it first needs a value
                auto load_id = [&](int i) -> int {
                    const int tok = (t.s0 + (i >> two)) * kN + (lane >> 1) * 16;
                    return lane < 16 && i < n_pairs && tok < t.lim ? __ldg(table + page_of(P, tok)) : -1;
                };
                auto load_scale = [&](int i, int id) -> float {
                    if (id < 0 || id >= A.n_pages) return 1.f;
                    return __ldg(A.scales + ((size_t)id * A.Hkv + t.h[i & two]) * 2 + (lane & 1));
                };
                float next_scale = load_scale(0, load_id(0));
                int next_id = load_id(1);
                for (int i = 0; i < n_pairs && ok; ++i) {
                    const int s = t.s0 + (i >> two);
                    int *mine = bad + (i & two);
                    const float my_scale = kv8_read_scale(next_scale);
                    next_scale = load_scale(i + 1, next_id);
                    next_id = load_id(i + 2);
                    // 2^e, e <= 7: its codes' factor 2^(120 + e) is a bf16
                    const uint32_t sb = __float_as_uint(my_scale);
                    const bool plain = (sb & 0x007fffffu) == 0u && sb <= 0x43000000u;
                    const uint32_t m = ((sb >> 23) + 120u) << 7, my_factor = m | (m << 16);
                    const bool all_plain = __all_sync(0xffffffffu, plain);
                    if (__any_sync(0xffffffffu, *abort != 0) || !mbar_wait_warp(&sh.st_full[stage], sph, wait)) {
                        ok = false;
                        break;
                    }
                    const bool rag = ragged(t, s);
                    if (rag && fresh) {
                        if (lane < 2) bad[lane] = 0x7fffffff;
                        __syncwarp();
                        fresh = false;
                    }
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        const uint8_t *codes = stages + stage * C::kStage + from + x * (8 * D);
                        uint4 v[NI];
                        uint32_t nan = 0;
#pragma unroll
                        for (int k = 0; k < NI; ++k) {
                            v[k] = *reinterpret_cast<const uint4 *>(codes + k * (TPI * 2 * D));
                            nan |= nan4(v[k].x) | nan4(v[k].y) | nan4(v[k].z) | nan4(v[k].w);
                        }
                        const bool fast = __all_sync(0xffffffffu, !(nan & 0x80808080u)) && all_plain;
                        if (x == 1 && lane == 0) mbar_arrive(&sh.st_empty[stage]);
                        if (!mbar_wait_warp(&sh.empty[slot], ph, wait)) {
                            ok = false;
                            break;
                        }
                        if (tid == 0) store_release(&sh.issued, ++fills);
                        uint8_t *dst = ring + slot * kTile;
                        if (fast && !rag) {
#pragma unroll
                            for (int k = 0; k < NI; ++k) {
                                uint4 lo, hi;
                                widen16(v[k], __shfl_sync(0xffffffffu, my_factor, ((k * TPI + tr) >> 4) * 2 + x), lo, hi);
                                *reinterpret_cast<uint4 *>(dst + at0 + k * (TPI * 128)) = swap ? hi : lo;
                                *reinterpret_cast<uint4 *>(dst + at1 + k * (TPI * 128)) = swap ? lo : hi;
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < NI; ++k) {
                                const int group = ((k * TPI + tr) >> 4) * 2 + x;
                                uint4 lo, hi;
                                if (fast) widen16(v[k], __shfl_sync(0xffffffffu, my_factor, group), lo, hi);
                                else widen16_any(v[k], __shfl_sync(0xffffffffu, my_scale, group), lo, hi);
                                const int tok = s * kN + k * TPI + tr;
                                if (tok >= t.lim) {
                                    lo = hi = make_uint4(0u, 0u, 0u, 0u);
                                } else if (x == 1 && tok > t.pos[0] && !fast && (odd8(lo) || odd8(hi))) {
                                    atomicMin(mine, tok);
                                    lo = hi = make_uint4(0u, 0u, 0u, 0u);
                                }
                                *reinterpret_cast<uint4 *>(dst + at0 + k * (TPI * 128)) = swap ? hi : lo;
                                *reinterpret_cast<uint4 *>(dst + at1 + k * (TPI * 128)) = swap ? lo : hi;
                            }
                        }
                        fence_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.full[slot]);
                        if (++slot == kSlots) {
                            slot = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    if (++stage == kStages) {
                        stage = 0;
                        sph ^= 1u;
                    }
                }
                reader.release<true>(sh);
                reader.advance();
            }
            if (!ok && lane == 0) {
                raise_status(A.status, SPEC_DEV_TIMEOUT);
                *abort = 1;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        // ------------------------------------------------------ softmax
        const int x = warp / kGroupWarps;               // query tile A (0) or B (1)
        const int r = (warp % kGroupWarps) * 32 + lane; // row of the tile
        const uint32_t lane_base = (uint32_t)((warp % kGroupWarps) * 32) << 16;
        const uint32_t tS = tmem + lane_base + col_s(x), tO = tmem + lane_base + col_o(x);
        const float sc = A.scale_log2;
        const int rt = r / A.G;                          // the row's token
        int ns = 0, nact = 0;      // S hand-offs taken; parts this tile took part in
        uint32_t n_full = 0;       // and those whose results were copied as a tile
        bool ok = true;
        PartReader reader;
        while (ok && reader.next<true>(sh, wait, &ok)) {
            const Part &t = sh.parts[reader.i];
            const bool row_ok = rt < t.nt[x];
            const int n = t.n_t[x], s0 = t.s0;
            if (n == 0) {                                // (no such tile, or tile A is through: an empty part)
                if (row_ok) A.part_ml[(size_t)t.slot * A.ru + x * rows + r] = make_float2(-INFINITY, kUnwritten);
                reader.release<true>(sh);
                reader.advance();
                continue;
            }
            const bool warp_ok = __any_sync(0xffffffffu, row_ok);
            const int sure = t.pos[x] + 1;               // tokens the tile's first row sees
            const int seen = sure + rt;                  // and this row
            float m_used = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                if (__any_sync(0xffffffffu, *abort != 0) ||
                    !mbar_wait_warp(&sh.s_full[x], (uint32_t)(ns & 1), wait)) {
                    ok = false;
                    break;
                }
                ++ns;
                fence_after();
                if (!warp_ok) {                          // (rows without a query: P is whatever is there)
                    fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh.p_full[x][0]);
                        mbar_arrive(&sh.p_full[x][1]);
                    }
                    continue;
                }
                const int c0 = (s0 + j) * kN;
                const bool masked = c0 + kN > sure;
                // The S row: four TMEM loads in flight, one wait (each wait_ld ties its
                // registers; the later ones return at once).  Beside eight widening
                // warps there are registers for half of it: the other half is read
                // again once the maximum is known.
                constexpr int kHeld = K8 ? 2 : 4;        // 32-key parts of the row held
                uint32_t v[kHeld][32];
                float tmv[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                // Hidden scores become -inf where they lie: a few rolled instructions, so
                // that all steps run the same unrolled ones below (masked there, whole
                // prompts take 370 us instead of 359, and the 8-bit mixed batch 347
                // instead of 310; a copy of them for such steps alone 427 and 332).
                // hidden: parts of which no row of the warp sees any, whose weights are
                // left out beside the widening warps (elsewhere the branch costs more:
                // prompts 383 us).
                uint32_t hidden = 0u;
                if (masked) {
#pragma unroll 1
                    for (int c = 0; c < kN / 32; ++c) {
                        const int n = seen - c0 - c * 32;            // seen ones of these 32
                        if (__all_sync(0xffffffffu, n >= 32)) continue;
                        if (K8 && __all_sync(0xffffffffu, n <= 0)) hidden |= 1u << c;
                        uint32_t w[32];
                        ld32(tS + c * 32, w);
                        wait_ld(w);
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e] = e < n ? w[e] : 0xff800000u;
                        st32(tS + c * 32, w);
                    }
                    wait_st();
                }
                // the row maximum (three-input max, four chains)
                auto top = [&](const uint32_t (&w)[32]) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tmv[q] = max3(tmv[q], __uint_as_float(w[e + 2 * q]), __uint_as_float(w[e + 2 * q + 1]));
                };
#pragma unroll
                for (int c = 0; c < kHeld; ++c) ld32(tS + c * 32, v[c]);
#pragma unroll
                for (int c = 0; c < kHeld; ++c) wait_ld(v[c]);
#pragma unroll
                for (int c = 0; c < kHeld; ++c) top(v[c]);
#pragma unroll
                for (int c = kHeld; c < kN / 32; ++c) {
                    uint32_t w[32];
                    ld32(tS + c * 32, w);
                    wait_ld(w);
                    top(w);
                }
                const float traw = fmaxf(fmaxf(tmv[0], tmv[1]), fmaxf(tmv[2], tmv[3]));
                const float tm = traw == -INFINITY ? -INFINITY : traw * sc;
                const bool raise = tm > m_used + kRescale || (m_used == -INFINITY && tm != -INFINITY);
                // (a sum that is NaN before any maximum stays so)
                const float alpha =
                    !raise ? 1.f : (m_used == -INFINITY) ? 1.f : fast_exp2(m_used - tm);
                // O holds every earlier PV of this tile (issued before the S
                // just waited for): rescale the rows that raised their max
                // (TMEM loads and stores are warp-collective: the whole warp
                // takes part, the other rows scaled by exactly 1)
                const bool scale_o = raise && j > 0 && m_used != -INFINITY;
                if (__any_sync(0xffffffffu, scale_o)) {
                    const float a = scale_o ? alpha : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        ld32(tO + c * 32, o);
                        wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                        st32(tO + c * 32, o);
                    }
                }
                if (raise) {
                    l *= alpha;
                    m_used = tm;
                }
                const float mu = m_used == -INFINITY ? 0.f : m_used;
                // P = exp2(s * scale - mu) (pairs: one f32x2 FMA, two ex2,
                // one f32x2 add, one pack) over the first 64 columns of S
                const uint64_t sc2 = pair(sc, sc), nmu2 = pair(-mu, -mu);
                uint64_t rs2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < kN / 32; ++c) {
                    uint32_t pw[16];
                    uint32_t (&w)[32] = v[c % kHeld];
                    if (K8 && ((hidden >> c) & 1u)) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) pw[e] = 0u;
                    } else {
                        if (c >= kHeld) {
                            ld32(tS + c * 32, w);
                            wait_ld(w);
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float t0, t1;
                            unpair(fma2(pair(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1])), sc2, nmu2),
                                   t0, t1);
                            const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
                            rs2[e & 1] = add2(rs2[e & 1], pair(p0, p1));
                            pw[e] = pack_bf16(p0, p1);
                        }
                    }
                    st16(tS + c * 16, pw);
                    if (c == kN / 64 - 1) {              // the first half's MMAs may start
                        wait_st();
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.p_full[x][0]);
                    }
                }
                float rs[4];
                unpair(rs2[0], rs[0], rs[1]);
                unpair(rs2[1], rs[2], rs[3]);
                l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[x][1]);
            }
            if (!ok) break;
            // epilogue: O / l (bf16) and the LSE of this row, or its part of them
            if (!mbar_wait_warp(&sh.o_done[x], (uint32_t)(nact & 1), wait)) {
                ok = false;
                break;
            }
            fence_after();
            // a non-finite value among those looked over, which this row sees
            bool odd = false;
            if (ragged(t, t.s0 + n - 1)) {
                const volatile int *bad = sh.bad[reader.i] + (t.sets == 2 ? x : 0);
                for (int w = 0; w < (K8 ? kConvWarps : 1); ++w) odd = odd || seen > bad[2 * w];
            }
            const bool whole = t.slot < 0;
            const float inv = odd ? __uint_as_float(0x7fffffffu) : whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            // A row's 2 D bytes -- all of it as bf16, or half of it as fp32 -- pass through
            // the place of its query, 16-byte chunks swizzled, and leave as whole lines,
            // two (D = 64: four) rows an instruction; what waits for the tile's O or
            // the place goes on before the stores.
            constexpr int RB = 2 * D, CH = RB / 16;      // bytes, chunks of a row
            constexpr int RI = 32 / CH;                  // rows an instruction
            uint8_t *stage = qbuf + x * kTile + (warp % kGroupWarps) * (32 * RB);
            const int r0 = (warp % kGroupWarps) * 32, nr = min(32, t.nt[x] * A.G - r0);
            // row r of the tile is row first + r + (its token) * skip of o (or of the parts)
            const size_t first = whole ? (size_t)t.row[x] * A.Hq + (size_t)t.h[x] * A.G : (size_t)t.slot * A.ru + x * rows;
            const uint32_t skip = whole ? (uint32_t)(A.Hq - A.G) : 0u;
            auto let_go_of_o = [&]() {
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.o_free[x]);
            };
            auto let_go_of_q = [&]() {
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_empty[x]);
                reader.release<true>(sh);
            };
            // N columns of O from column c0 on, as 16-byte chunks of bf16 or fp32
            // (kFull: a whole query tile, laid out as its queries were)
            auto pass = [&](auto as_bf16, auto as_tile, int c0, bool last) {
                constexpr bool kBf16 = decltype(as_bf16)::value, kFull = decltype(as_tile)::value;
                constexpr int N = kBf16 ? D : D / 2;
                constexpr int kPer = kBf16 ? 4 : 8;                  // chunks of 32 columns
#pragma unroll 1
                for (int n0 = 0; n0 < N; n0 += 32) {
                    uint32_t y[32];
                    ld32(tO + c0 + n0, y);
                    wait_ld(y);
                    if (last && n0 + 32 == N) let_go_of_o();
#pragma unroll
                    for (int k = 0; k < kPer; ++k) {
                        uint4 w;
                        if constexpr (kBf16) {
                            const int e = 8 * k;
                            w = make_uint4(pack_bf16(__uint_as_float(y[e]) * inv, __uint_as_float(y[e + 1]) * inv),
                                           pack_bf16(__uint_as_float(y[e + 2]) * inv, __uint_as_float(y[e + 3]) * inv),
                                           pack_bf16(__uint_as_float(y[e + 4]) * inv, __uint_as_float(y[e + 5]) * inv),
                                           pack_bf16(__uint_as_float(y[e + 6]) * inv, __uint_as_float(y[e + 7]) * inv));
                        } else {
                            const int e = 4 * k;
                            w = make_uint4(__float_as_uint(__uint_as_float(y[e]) * inv),
                                           __float_as_uint(__uint_as_float(y[e + 1]) * inv),
                                           __float_as_uint(__uint_as_float(y[e + 2]) * inv),
                                           __float_as_uint(__uint_as_float(y[e + 3]) * inv));
                        }
                        const int at = n0 / 32 * kPer + k;
                        if constexpr (kFull)
                            *reinterpret_cast<uint4 *>(qbuf + x * kTile + (at / 8) * kHalf + r * 128 +
                                                       (((at % 8) ^ (r & 7)) << 4)) = w;
                        else
                            *reinterpret_cast<uint4 *>(stage + lane * RB + ((at ^ (lane & 7)) << 4)) = w;
                    }
                }
                if constexpr (kFull) return;
                __syncwarp();
                uint8_t *dst = kBf16 ? static_cast<uint8_t *>(A.o) : reinterpret_cast<uint8_t *>(A.part_o) + c0 * 4;
                constexpr int kAtOnce = 8;
#pragma unroll 1
                for (int k0 = 0; k0 < CH; k0 += kAtOnce) {
                    uint4 w[kAtOnce];
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        const int rr = (k0 + k) * RI + lane / CH;
                        w[k] = *reinterpret_cast<const uint4 *>(stage + rr * RB + (((lane % CH) ^ (rr & 7)) << 4));
                    }
                    __syncwarp();
                    if (last && k0 + kAtOnce == CH) let_go_of_q();
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        const int rr = (k0 + k) * RI + lane / CH;
                        if (rr >= nr) continue;
                        const uint32_t tok = ((uint32_t)(r0 + rr) * P.g_mul) >> 16;
                        const size_t at = first + (uint32_t)(r0 + rr) + (size_t)tok * skip;
                        *reinterpret_cast<uint4 *>(dst + at * (kBf16 ? 2 * D : 4 * D) + (lane % CH) * 16) = w[k];
                    }
                }
            };
            if (whole && t.nt[x] == P.tb) {
                // all of the tile's tokens: one warp has them copied once the four have
                // written them (a warp's own stores wait behind the MMAs' reads of
                // shared memory: 5 K cycles a tile)
                if (warp_ok) pass(Bool<true>{}, Bool<true>{}, 0, true);
                else let_go_of_o();
                fence_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.o_ready[x]);
                    if (warp % kGroupWarps == 0) {
                        if (mbar_wait(&sh.o_ready[x], n_full & 1u, wait)) {
                            for (int hh = 0; hh < NH; ++hh)
                                tma_store_3d(&mo, qbuf + x * kTile + hh * kHalf, hh * 64, t.h[x] * A.G, t.row[x]);
                            bulk_commit_and_wait_read();
                        } else {
                            ok = false;
                        }
                    }
                    mbar_arrive(&sh.q_empty[x]);
                }
                reader.release<true>(sh);
                ok = __all_sync(0xffffffffu, ok);
                ++n_full;
            } else if (!warp_ok) {
                let_go_of_o();
                let_go_of_q();
            } else if (whole) {
                pass(Bool<true>{}, Bool<false>{}, 0, true);
            } else {
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += D / 2) pass(Bool<false>{}, Bool<false>{}, c0, c0 > 0);
            }
            if (row_ok) {
                const size_t at = first + r + (size_t)rt * skip;
                if (whole) A.lse[at] = l == 0.f ? -INFINITY : l != l ? l : (m_used + log2f(l)) * kLn2;
                else A.part_ml[at] = make_float2(m_used, l);
            }
            reader.advance();
            ++nact;
        }
        if (!ok) {
            if (lane == 0) raise_status(A.status, SPEC_DEV_TIMEOUT);
            *abort = 1;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols));
}

template <int D, bool K8, bool kJoint>
spec_status_t launch_tc(const ctc::Params &P, const CUtensorMap (&m)[4], int n_cta, cudaStream_t s) {
    constexpr size_t smem = ctc::smem_bytes<D, K8>();
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    if (set_smem_limit(reinterpret_cast<const void *>(chunk_tc_kernel<D, K8, kJoint>), smem) != SPEC_OK)
        return SPEC_ERR_CUDA;
    return launch(chunk_tc_kernel<D, K8, kJoint>, dim3(n_cta), dim3(ctc::Cfg<D, K8>::kThreads), smem, s, P, m[0], m[1], m[2],
                  m[3]);
}

}  // namespace

ChunkPlan chunk_tc_plan(const ChunkParams &P, bool kv8) {
    const int tb = ctc::kM / P.G;
    // What a key costs a unit of two heads, against one of a single head's two tiles:
    // 39 single tokens and 9 chunks, by eighths 8 / 9 / 10 / 11 / 12 / 16: 213 / 202 /
    // 191 / 195 / 198 / 213 us; 8 bits, 10 / 12 / 13 / 14 / 16: 322 / 297 / 285 / 290 /
    // 303.  A unit's start counts as three steps (2 / 3 / 4 / 6: whole prompts 345 /
    // 347 / 350 / 365, mixed 219 / 213 / 212 / 224 at 16 eighths).
    const int pair_cost = kv8 ? 13 : 10;
    return ChunkPlan{2 * tb * P.G, 2 * tb, ctc::kN, 3 * ctc::kN, pair_cost, ctc::kN, num_sms()};
}

spec_status_t launch_chunk_tc(const ChunkParams &C, bool kv8, int n_cta, cudaStream_t s) {
    ctc::Params P{};
    P.c = C;
    P.tb = ctc::kM / C.G;
    P.g_mul = (uint32_t)((65536 + C.G - 1) / C.G);
    P.box = ctc::kN;
    if (C.paged) {
        int a = C.ps, b = ctc::kN;                       // the greatest common divisor
        while (b) {
            const int r = a % b;
            a = b;
            b = r;
        }
        P.box = a;
        // floor(t / ps) = (t m) >> (31 + L), L = ceil(log2 ps), m = ceil(2^(31 + L) / ps),
        // exact for t < 2^31
        int L = 0;
        while ((1ll << L) < C.ps) ++L;
        P.ps_shift = 31 + L;
        P.ps_mul = (uint32_t)(((1ull << (31 + L)) + C.ps - 1) / C.ps);
    }
    const bool joint = !kv8 && C.paged && C.d == 128;
    CUtensorMap m[4] = {};
    const cuuint64_t d0[3] = {(cuuint64_t)C.d, (cuuint64_t)C.Hq, (cuuint64_t)C.n_tokens};
    const cuuint64_t s0[2] = {(cuuint64_t)C.d * 2, (cuuint64_t)C.stride_q * 2};
    const cuuint32_t b0[3] = {64u, (cuuint32_t)C.G, (cuuint32_t)P.tb};
    const cuuint64_t so[2] = {(cuuint64_t)C.d * 2, (cuuint64_t)C.Hq * C.d * 2};
    if (!encode_bf16_map(&m[0], C.q, 3, d0, s0, b0) || !encode_bf16_map(&m[1], C.o, 3, d0, so, b0))
        return SPEC_ERR_CUDA;
    if (!kv8) {
        const cuuint64_t nh = C.d / 64;
        cuuint64_t d1[3] = {(cuuint64_t)C.d, (cuuint64_t)C.capacity, (cuuint64_t)C.cache_heads};
        cuuint64_t s1[2] = {(cuuint64_t)C.d * 2, (cuuint64_t)C.capacity * C.d * 2};
        if (C.paged) {
            d1[0] = 64;
            d1[1] = C.ps;
            d1[2] = (cuuint64_t)C.n_pages * C.Hkv * nh;
            s1[0] = 128;
            s1[1] = (cuuint64_t)C.ps * 128;
        }
        const cuuint32_t b1[3] = {64u, (cuuint32_t)P.box, 1u};
        // pages of two halves: eight tokens of the one, of the other, and so on
        const cuuint64_t d2[5] = {64u, 8u, nh, (cuuint64_t)C.ps / 8, (cuuint64_t)C.n_pages * C.Hkv};
        const cuuint64_t s2[4] = {128u, (cuuint64_t)C.ps * 128, 1024u, (cuuint64_t)C.ps * 128 * nh};
        const cuuint32_t b2[5] = {64u, 8u, (cuuint32_t)nh, (cuuint32_t)P.box / 8, 1u};
        for (int kv = 0; kv < 2; ++kv) {
            const void *base = kv ? C.vc : C.kc;
            if (!(joint ? encode_bf16_map(&m[2 + kv], base, 5, d2, s2, b2)
                        : encode_bf16_map(&m[2 + kv], base, 3, d1, s1, b1)))
                return SPEC_ERR_CUDA;
        }
    }
    if (C.d == 64) return kv8 ? launch_tc<64, true, false>(P, m, n_cta, s) : launch_tc<64, false, false>(P, m, n_cta, s);
    if (kv8) return launch_tc<128, true, false>(P, m, n_cta, s);
    return joint ? launch_tc<128, false, true>(P, m, n_cta, s) : launch_tc<128, false, false>(P, m, n_cta, s);
}

}  // namespace sv
