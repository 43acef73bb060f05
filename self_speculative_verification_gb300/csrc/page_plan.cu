// spec_page_plan: block tables and slot maps from request lengths.
//
// Every CTA scans the requests by itself -- pages and tokens before each, kept
// in shared memory a chunk of requests at a time -- and then takes its share
// of the packed tokens, 256 to a warp; a token that opens a new page also
// records it in the page table.  A small batch is one CTA and one launch; a
// larger one is spread over the SMs, and a second launch moves free_head,
// which every CTA of the first has to have read.  Bound by launch and scan
// latency: 64 requests 9.7 us, 400 K tokens of 200 requests 8.9 us of GPU time
// (on one CTA 40); the slots are 8 bytes each.
#include "common.cuh"

namespace sv {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanChunk = 2048;                     // requests scanned at a time
constexpr int kPlanItems = kPlanChunk / kPlanThreads;
constexpr int kPlanTokens = 256;                     // packed tokens a warp takes at a time
constexpr int kPlanAlone = 4096;                     // slots that one CTA takes alone

struct PlanParams {
    const int32_t *seq_len, *n_new, *free_pages;
    int32_t *page_table, *free_head, *cu_new, *new_len;
    int64_t *slot_map;
    long long n_slots;
    int B, ps, n_pages, max_pages, n_free, capacity;
    // pos / ps as (pos ps_mul) >> ps_shift: with L = ceil(log2 ps), ps_mul =
    // ceil(2^(31 + L) / ps) and ps_shift = 31 + L, exact for pos < 2^31
    uint64_t ps_mul;
    int ps_shift;
    int *status;
};

struct PlanReq {
    int S, n;          // tokens held; tokens asked for (n < 0: 0)
    int had, take;     // pages held, pages it takes
    bool ok;           // its tokens get slots
};

__device__ __forceinline__ PlanReq plan_request(const PlanParams &P, int b, int *bits) {
    PlanReq r{0, 0, 0, 0, false};
    r.S = P.seq_len[b];
    r.n = P.n_new[b];
    if (r.n < 0) {
        *bits |= SPEC_DEV_BAD_INDEX;
        r.n = 0;
    }
    if (r.S < 0 || r.S > P.capacity) {
        *bits |= SPEC_DEV_SEQ_OVERFLOW;
        return r;
    }
    if ((long long)r.S + r.n > P.capacity) {
        *bits |= SPEC_DEV_CAPACITY;
        return r;
    }
    r.ok = true;
    r.had = (r.S + P.ps - 1) / P.ps;
    r.take = (r.S + r.n + P.ps - 1) / P.ps - r.had;
    return r;
}

// Exclusive sums over the block of two values a thread.
__device__ void block_scan2(long long a, long long p, long long *ex_a, long long *ex_p,
                            long long *tot_a, long long *tot_p) {
    constexpr int kWarps = kPlanThreads / 32;
    __shared__ long long sa[kWarps], sp[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto scan = [&](long long x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += v;
        }
        return x;
    };
    const long long ia = scan(a), ip = scan(p);
    if (lane == 31) {
        sa[warp] = ia;
        sp[warp] = ip;
    }
    __syncthreads();
    const long long wa = scan(lane < kWarps ? sa[lane] : 0), wp = scan(lane < kWarps ? sp[lane] : 0);
    *tot_a = __shfl_sync(0xffffffffu, wa, 31);
    *tot_p = __shfl_sync(0xffffffffu, wp, 31);
    const long long ba = __shfl_sync(0xffffffffu, wa, warp > 0 ? warp - 1 : 0);
    const long long bp = __shfl_sync(0xffffffffu, wp, warp > 0 ? warp - 1 : 0);
    *ex_a = ia - a + (warp > 0 ? ba : 0);
    *ex_p = ip - p + (warp > 0 ? bp : 0);
    __syncthreads();          // sa / sp may be written again
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PlanParams P, bool move_head) {
    pdl_wait();
    const int nc = (int)gridDim.x, rank = (int)blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31;
    __shared__ int s_cu[kPlanChunk + 1];      // first packed token, within the chunk
    __shared__ int s_S[kPlanChunk];
    __shared__ int s_pg[kPlanChunk];          // its first free-list entry - pages it holds
    __shared__ uint8_t s_ok[kPlanChunk];      // its tokens get slots

    // totals, and with them whether the batch can be served at all
    int bits = 0;
    long long tok = 0, pages = 0, tot_tok, tot_pages, d0, d1;
    for (int b = tid; b < P.B; b += kPlanThreads) {
        const PlanReq r = plan_request(P, b, &bits);
        tok += r.n;
        pages += r.take;
    }
    block_scan2(tok, pages, &d0, &d1, &tot_tok, &tot_pages);
    const int head = *P.free_head;
    bool serve = head >= 0 && (long long)head + tot_pages <= P.n_free;
    if (!serve) bits |= SPEC_DEV_CAPACITY;       // (every CTA finds the same)
    const bool fits = tot_tok <= (1ll << 31) - 1024;
    if (!fits || tot_tok > P.n_slots) bits |= SPEC_DEV_BAD_INDEX;
    serve = serve && fits;

    long long tok0 = 0, page0 = 0;            // packed tokens and pages before the chunk
    const int chunks = (P.B + kPlanChunk - 1) / kPlanChunk;
    for (int c = 0; c < chunks && fits; ++c) {
        const int b0 = c * kPlanChunk, nb = min(kPlanChunk, P.B - b0);
        PlanReq r[kPlanItems];
        long long a = 0, p = 0;
        int dummy = 0;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            const int k = tid * kPlanItems + i;
            r[i] = k < nb ? plan_request(P, b0 + k, &dummy) : PlanReq{0, 0, 0, 0, false};
            a += r[i].n;
            p += r[i].take;
        }
        long long ea, ep, ta, tp;
        block_scan2(a, p, &ea, &ep, &ta, &tp);
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            const int k = tid * kPlanItems + i;
            if (k < nb) {
                s_cu[k] = (int)ea;
                s_S[k] = r[i].S;
                s_pg[k] = (int)(head + page0 + ep - r[i].had);
                s_ok[k] = (uint8_t)(r[i].ok && serve);
                if (rank == 0) {
                    P.cu_new[b0 + k] = (int32_t)(tok0 + ea);
                    if (P.new_len) P.new_len[b0 + k] = r[i].S + (r[i].ok && serve ? r[i].n : 0);
                }
            }
            ea += r[i].n;
            ep += r[i].take;
        }
        if (tid == 0) s_cu[nb] = (int)ta;
        __syncthreads();
        // this CTA's pieces of the chunk
        const int n_tok = (int)ta;
        const int warps = kPlanThreads / 32 * nc, w = rank * (kPlanThreads / 32) + (tid >> 5);
        for (long long t0 = (long long)w * kPlanTokens; t0 < n_tok; t0 += (long long)warps * kPlanTokens) {
            int lo = 0, hi = nb - 1;          // last request starting at or before t0
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_cu[mid] <= t0) lo = mid;
                else hi = mid - 1;
            }
            int k = lo;
            // every token's page first, so that their loads are in flight at once
            constexpr int kPer = kPlanTokens / 32;
            int page[kPer], off[kPer];
            int32_t *entry[kPer];            // where a page it opens is recorded
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int t = (int)t0 + i * 32 + lane;
                page[i] = -2;                // no slot
                off[i] = 0;
                entry[i] = nullptr;
                if (t >= n_tok) continue;
                while (t >= s_cu[k + 1]) ++k;
                if (!s_ok[k]) continue;
                const int S = s_S[k], pos = S + t - s_cu[k];
                const int j = (int)(((uint64_t)pos * P.ps_mul) >> P.ps_shift);
                off[i] = pos - j * P.ps;
                int32_t *at = P.page_table + (size_t)(b0 + k) * P.max_pages + j;
                const bool fresh = j * P.ps >= S;            // a page it takes now
                page[i] = fresh ? P.free_pages[s_pg[k] + j] : *at;
                if (fresh && off[i] == 0) entry[i] = at;
                if (page[i] < 0) page[i] = -1;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int t = (int)t0 + i * 32 + lane;
                if (t >= n_tok) continue;
                long long slot = -1;
                if (page[i] >= 0 && page[i] < P.n_pages) {
                    slot = (long long)page[i] * P.ps + off[i];
                    if (entry[i]) *entry[i] = page[i];
                } else if (page[i] != -2) {
                    bits |= SPEC_DEV_BAD_PAGE;
                }
                if (tok0 + t < P.n_slots) P.slot_map[tok0 + t] = slot;
            }
        }
        tok0 += ta;
        page0 += tp;
        __syncthreads();          // the chunk's arrays may be written again
    }
    // behind the last token
    for (long long t = (fits ? tot_tok : 0) + rank * kPlanThreads + tid; t < P.n_slots;
         t += (long long)nc * kPlanThreads)
        P.slot_map[t] = -1;
    if (!fits && rank == 0)
        for (int b = tid; b < P.B; b += kPlanThreads) {
            P.cu_new[b] = 0;
            if (P.new_len) P.new_len[b] = P.seq_len[b];
        }
    if (rank == 0 && tid == 0) P.cu_new[P.B] = fits ? (int32_t)tot_tok : 0;
    if (bits) raise_status(P.status, bits);
    if (move_head) {                          // (one CTA, whose threads have all read it)
        __syncthreads();
        if (tid == 0 && serve) *P.free_head = head + (int)tot_pages;
    }
}

// free_head, behind a plan of several CTAs (which has reported what is wrong).
__global__ void __launch_bounds__(kPlanThreads) page_plan_head_kernel(PlanParams P) {
    pdl_wait();
    int bits = 0;
    long long tok = 0, pages = 0, tot_tok, tot_pages, d0, d1;
    for (int b = threadIdx.x; b < P.B; b += kPlanThreads) {
        const PlanReq r = plan_request(P, b, &bits);
        tok += r.n;
        pages += r.take;
    }
    block_scan2(tok, pages, &d0, &d1, &tot_tok, &tot_pages);
    const int head = *P.free_head;
    __syncthreads();
    if (threadIdx.x == 0 && head >= 0 && (long long)head + tot_pages <= P.n_free &&
        tot_tok <= (1ll << 31) - 1024)
        *P.free_head = head + (int)tot_pages;
}

struct PlanArray {
    const void *at;
    size_t bytes;
};

bool overlap(const PlanArray &a, const PlanArray &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return a.bytes && b.bytes && a.at && b.at && x < y + b.bytes && y < x + a.bytes;
}

}  // namespace
}  // namespace sv

extern "C" spec_status_t spec_page_plan(int batch, int page_size, int n_pages,
                                        int max_pages_per_seq, const int32_t *seq_len,
                                        const int32_t *n_new, int32_t *page_table,
                                        const int32_t *free_pages, int n_free, int32_t *free_head,
                                        int32_t *cu_new, long long n_slots, int64_t *slot_map,
                                        int32_t *new_len, void *stream) {
    using namespace sv;
    if (batch < 0 || page_size <= 0 || n_pages <= 0 || max_pages_per_seq <= 0 || n_free < 0 ||
        n_slots < 0 || !cu_new)
        return SPEC_ERR_INVALID_ARG;
    if ((long long)max_pages_per_seq * page_size > (1ll << 30)) return SPEC_ERR_UNSUPPORTED;
    if (n_slots > 0 && !slot_map) return SPEC_ERR_INVALID_ARG;
    if (!free_head || (batch > 0 && (!seq_len || !n_new || !page_table)) ||
        (n_free > 0 && !free_pages))
        return SPEC_ERR_INVALID_ARG;
    // outputs are written while other threads still read the inputs
    const size_t b4 = (size_t)batch * 4;
    const PlanArray arrays[] = {{cu_new, b4 + 4}, {slot_map, (size_t)n_slots * 8}, {new_len, b4},
                                {seq_len, b4}, {n_new, b4}, {page_table, b4 * max_pages_per_seq},
                                {free_pages, (size_t)n_free * 4}, {free_head, 4}};
    for (int o = 0; o < 3; ++o)
        for (int i = o + 1; i < (int)(sizeof(arrays) / sizeof(arrays[0])); ++i)
            if (overlap(arrays[o], arrays[i])) return SPEC_ERR_INVALID_ARG;
    PlanParams P{};
    P.seq_len = seq_len;
    P.n_new = n_new;
    P.free_pages = free_pages;
    P.page_table = page_table;
    P.free_head = free_head;
    P.cu_new = cu_new;
    P.new_len = new_len;
    P.slot_map = slot_map;
    P.n_slots = n_slots;
    P.B = batch;
    P.ps = page_size;
    P.n_pages = n_pages;
    P.max_pages = max_pages_per_seq;
    P.n_free = n_free;
    P.capacity = max_pages_per_seq * page_size;
    P.status = status_ptr();
    if (!P.status) return SPEC_ERR_CUDA;
    int log = 0;
    while ((1ll << log) < page_size) ++log;
    P.ps_shift = 31 + log;
    P.ps_mul = ((1ull << P.ps_shift) + page_size - 1) / page_size;
    cudaStream_t s = as_stream(stream);
    // a plan of few slots is one CTA's; others: 8 warps' pieces a CTA
    int nc = 1;
    if (n_slots > kPlanAlone) {
        const long long want = (n_slots + 8 * kPlanTokens - 1) / (8 * kPlanTokens);
        nc = (int)(want < num_sms() ? want : num_sms());
    }
    spec_status_t st = launch(page_plan_kernel, dim3(nc), dim3(kPlanThreads), 0, s, P, nc == 1);
    if (st == SPEC_OK && nc > 1) st = launch(page_plan_head_kernel, dim3(1), dim3(kPlanThreads), 0, s, P);
    return st != SPEC_OK ? st : launch_status();
}
