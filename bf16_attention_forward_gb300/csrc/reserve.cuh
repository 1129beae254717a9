// reserve.cuh -- the pages and slots of a step's tokens, from the requests' lengths.
//
// Arithmetic (whole numbers).  Sequence b of len[b] tokens wants want[b] = max(ceil(len[b] / page_size), shared[b]) pages
// and holds held[b].  Pages past want[b] go on top of the stack of free pages, in the order (sequence, page); then pages
// that are missing come off its top, in the same order.  Token t of sequence b, cu[b] <= t < cu[b + 1], is key
// j = len[b] - (cu[b + 1] - t) of it and goes to slot table[b][j / page_size] * page_size + j % page_size.
//
// Bound: latency.  The reads and writes of a step are some 10 KB to 1 MB, a microsecond's; what takes the time is the
// launch and a chain of reads: lengths -> (sums over the sequences) -> table -> stack -> table -> slots.  One launch of
// one cluster: its CTAs all form the sums for themselves (a sequence a thread, more in longer batches), then deal out
// the pages and after a cluster barrier the tokens; so the table is read where it was just written, without a kernel
// boundary between (1.5 to 2 us).  Nothing is written before every check has passed in every CTA.
#pragma once
#include "cache_common.cuh"

namespace cache {

struct ReserveParams {
    const int32_t* seqlens;
    const int32_t* cu_new;
    int32_t* table;
    const int32_t* held;
    int32_t* held_out;
    const int32_t* shared;         // or null
    int32_t* free_pages;
    const int32_t* count;
    int32_t* count_out;
    int64_t* slots;                // [total]
    int32_t* positions;            // [total] or null
    Pages pages;                   // (num_pages is not looked at)
    int B, capacity;
    long long total;
};

constexpr int kReserveThreads = 1024;
constexpr int kReserveWarps = kReserveThreads / 32;
constexpr int kReserveCu = 4096;   // offsets that a CTA searches in shared memory

// inclusive sums of two numbers over the threads of a block
__device__ __forceinline__ int2 block_scan(int2 v, int2* warp_s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v.x, off), y = __shfl_up_sync(0xFFFFFFFFu, v.y, off);
        if (lane >= off) { v.x += x; v.y += y; }
    }
    if (lane == 31) warp_s[warp] = v;
    __syncthreads();
    int2 before = lane < warp ? warp_s[lane] : make_int2(0, 0);
    before.x = __reduce_add_sync(0xFFFFFFFFu, before.x);
    before.y = __reduce_add_sync(0xFFFFFFFFu, before.y);
    return make_int2(v.x + before.x, v.y + before.y);
}

__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kReserveThreads, 1) attn_reserve_kernel(const __grid_constant__ ReserveParams p) {
    __shared__ int2 warp_s[kReserveWarps];
    __shared__ int back_s[kReserveThreads + 1], take_s[kReserveThreads + 1];   // pages returned / taken by the threads before
    __shared__ int cu_s[kReserveCu];
    pdl_wait();
    pdl_launch();
    const int t = threadIdx.x, per = (p.B - 1) / kReserveThreads + 1;          // sequences a thread
    const bool staged = p.B < kReserveCu;
    const int count = p.count[0];
    int bad = count < 0 || count > p.capacity;
    // sequence b: pages it holds and wants
    auto pages_of = [&](int b) {
        const int len = p.seqlens[b], shared = p.shared ? p.shared[b] : 0;
        const int n = len > 0 ? page_of(p.pages, len - 1) + 1 : 0;
        return make_int2(p.held[b], max(n, shared));
    };
    int back = 0, take = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const int b = t * per + i;
        if (b >= p.B) break;
        const int len = p.seqlens[b], c0 = p.cu_new[b], c1 = p.cu_new[b + 1];
        const int shared = p.shared ? p.shared[b] : 0;
        const int held = p.held[b];
        bad |= len < 0 || (long long)len > (long long)p.pages.max_pages * p.pages.page_size;
        bad |= c0 < 0 || c1 < c0 || c1 > p.total || (long long)c1 - c0 > len;
        bad |= shared < 0 || held < shared || held > p.pages.max_pages;
        if (!bad) {
            const int want = pages_of(b).y;
            back += max(held - want, 0);
            take += max(want - held, 0);
        }
        if (staged) cu_s[b] = c0;
    }
    if (staged && t == 0) cu_s[p.B] = p.cu_new[p.B];
    // (B * max_pages is below 2^31, and so are the sums)
    const int2 incl = block_scan(make_int2(back, take), warp_s);
    back_s[t + 1] = incl.x;
    take_s[t + 1] = incl.y;
    if (t == 0) back_s[0] = take_s[0] = 0;
    bad = __syncthreads_or(bad);
    const int all_back = back_s[kReserveThreads], all_take = take_s[kReserveThreads];
    // a stack with room for what comes back, and enough pages for what is taken
    bad = bad || (long long)count + all_back > p.capacity || (long long)count + all_back < all_take;
    const int rank = blockIdx.x, ctas = gridDim.x, first = rank * kReserveThreads + t, step = ctas * kReserveThreads;
    if (bad) {
        if (first == 0) report_invalid(ATTN_CACHE_SITE_RESERVE);
        if (first == 0) p.count_out[0] = count;
        for (int b = first; b < p.B; b += step) p.held_out[b] = p.held[b];
        for (long long i = first; i < p.total; i += step) {
            p.slots[i] = -1;
            if (p.positions) p.positions[i] = 0;
        }
        return;
    }
    // the sequence that has the k-th page of `sums`, and the page's number among its own
    auto find = [&](const int* sums, int k, bool taken) {
        int lo = 0, hi = kReserveThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sums[mid + 1] > k) hi = mid; else lo = mid + 1;
        }
        int b = lo * per, left = k - sums[lo];
        int2 hw = pages_of(b);
#pragma unroll 1
        while (true) {
            const int n = max(taken ? hw.y - hw.x : hw.x - hw.y, 0);
            if (left < n) break;
            left -= n;
            hw = pages_of(++b);
        }
        return make_int2(b, (taken ? hw.x : hw.y) + left);
    };
    for (int k = first; k < all_back; k += step) {
        const int2 at = find(back_s, k, false);
        p.free_pages[count + k] = p.table[(long long)at.x * p.pages.max_pages + at.y];
    }
    if (all_back > 0) cluster_barrier();               // pages that came back may be taken again
    const int top = count + all_back;
    for (int k = first; k < all_take; k += step) {
        const int2 at = find(take_s, k, true);
        p.table[(long long)at.x * p.pages.max_pages + at.y] = p.free_pages[top - 1 - k];
    }
    cluster_barrier();                                 // the table is complete; nobody reads `held` or `count` any more
    for (int b = first; b < p.B; b += step) p.held_out[b] = pages_of(b).y;
    if (first == 0) p.count_out[0] = top - all_take;
    const int* cu = staged ? cu_s : p.cu_new;
    const int cu_end = cu[p.B];
    for (long long i = first; i < p.total; i += step) {
        long long slot = -1;
        int j = 0;
        if (i >= cu[0] && i < cu_end) {
            int lo = 0, hi = p.B - 1;                  // the last sequence that starts at or before the token
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= i) lo = mid; else hi = mid - 1;
            }
            j = p.seqlens[lo] - (cu[lo + 1] - (int)i);
            const int pg = page_of(p.pages, j);
            const int phys = p.table[(long long)lo * p.pages.max_pages + pg];
            // (of a negative page never -1, which would pass for padding)
            slot = phys < 0 ? -2 : (long long)phys * p.pages.page_size + (j - pg * p.pages.page_size);
        }
        p.slots[i] = slot;
        if (p.positions) p.positions[i] = j;
    }
}

}  // namespace cache
