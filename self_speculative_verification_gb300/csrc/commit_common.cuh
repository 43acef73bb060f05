// Bookkeeping shared by kv_commit and kv8_commit: which rows of a request
// are written, the deterministic page allocation (requests in ascending
// order, each first fills its partly used last page, then takes pages from
// the free list in order), and the kernel that records it afterwards.
#pragma once

#include "common.cuh"

namespace sv {
namespace {

struct CommitParams {
    char *kc, *vc;                 // cache K/V (bytes)
    const char *kb, *vb;           // block K/V (bytes)
    int32_t *page_table;
    const int32_t *path, *acc_len;
    int32_t *seq_len;
    const int32_t *free_pages;
    int32_t *free_head;
    int n_free;
    int B, Hkv, R, path_cap, row_bytes;
    int blk_bytes, vec_per_blk;    // paged: bytes / 16-byte vectors of a 64-element block
    int paged, max_seq, page_size, max_pages, n_pages, capacity;
    int *status;
};

// Accepted rows of request b that will be written (0 when the request is
// skipped), with the reason bits for a skip.
__device__ __forceinline__ int effective_acc(const CommitParams &P, int b, int *bits) {
    const int a = P.acc_len[b];
    const int S = P.seq_len[b];
    if (a < 0 || a > P.path_cap) {
        *bits |= SPEC_DEV_BAD_INDEX;
        return 0;
    }
    if (S < 0 || S > P.capacity) {
        *bits |= SPEC_DEV_SEQ_OVERFLOW;
        return 0;
    }
    if ((long long)S + a > P.capacity) {
        *bits |= SPEC_DEV_CAPACITY;
        return 0;
    }
    return a;
}

__device__ __forceinline__ int pages_for(int tokens, int ps) { return (tokens + ps - 1) / ps; }

__device__ __forceinline__ int new_pages(const CommitParams &P, int b) {
    int bits = 0;
    const int a = effective_acc(P, b, &bits);
    const int S = P.seq_len[b];
    return a ? pages_for(S + a, P.page_size) - pages_for(S, P.page_size) : 0;
}

// Block-wide sums over requests: pages taken by requests before b and by all.
__device__ void page_prefix(const CommitParams &P, int b, int *before, int *total) {
    __shared__ int s_before[32], s_total[32];
    int mb = 0, mt = 0;
    for (int i = threadIdx.x; i < P.B; i += blockDim.x) {
        const int n = new_pages(P, i);
        mt += n;
        if (i < b) mb += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        mb += __shfl_xor_sync(0xffffffffu, mb, o);
        mt += __shfl_xor_sync(0xffffffffu, mt, o);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        s_before[warp] = mb;
        s_total[warp] = mt;
    }
    __syncthreads();
    int tb = 0, tt = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
        tb += s_before[w];
        tt += s_total[w];
    }
    __syncthreads();
    *before = tb;
    *total = tt;
}

// One CTA: new page-table entries, seq_len += accepted, free_head += taken.
__global__ void __launch_bounds__(256) kv_commit_finalize_kernel(CommitParams P) {
    pdl_wait();
    int head = 0, total = 0;
    if (P.paged) {
        int dummy = 0;
        page_prefix(P, 0, &dummy, &total);
        head = *P.free_head;
        if (head < 0 || (long long)head + total > P.n_free) return;
    }
    __syncthreads();   // every thread has read free_head
    // exclusive prefix of new pages over requests, in chunks of blockDim
    __shared__ int s_scan[256];
    int carry = 0;
    for (int base = 0; base < P.B; base += blockDim.x) {
        const int b = base + threadIdx.x;
        int bits = 0;
        const int a = b < P.B ? effective_acc(P, b, &bits) : 0;
        const int S = b < P.B ? P.seq_len[b] : 0;
        const int n = (P.paged && a) ? pages_for(S + a, P.page_size) - pages_for(S, P.page_size) : 0;
        s_scan[threadIdx.x] = n;
        __syncthreads();
        for (int o = 1; o < (int)blockDim.x; o <<= 1) {
            const int x = threadIdx.x >= o ? s_scan[threadIdx.x - o] : 0;
            __syncthreads();
            s_scan[threadIdx.x] += x;
            __syncthreads();
        }
        const int excl = carry + s_scan[threadIdx.x] - n;
        const int chunk_total = s_scan[blockDim.x - 1];
        __syncthreads();
        if (b < P.B && a > 0) {
            if (P.paged) {
                const int used = pages_for(S, P.page_size);
                for (int k = 0; k < n; ++k)
                    P.page_table[(size_t)b * P.max_pages + used + k] = P.free_pages[head + excl + k];
            }
            P.seq_len[b] = S + a;
        }
        carry += chunk_total;
    }
    if (P.paged && threadIdx.x == 0) *P.free_head = head + total;
}

}  // namespace
}  // namespace sv
