// evict.cuh -- cuts the caches of sequences to a budget of keys by accumulated attention weight.
//
// Rule.  A sequence of n keys with n <= budget stays as it is.  Otherwise every K/V head keeps `budget`
// keys: slots 0 .. sinks - 1, the last `recent` slots, and of the slots between them the budget - sinks -
// recent keys of largest weight (of equal weights the lower slots; a NaN ranks below every number).
// With end = budget - recent, the survivors below `end` stay where they are; the i-th survivor at or
// past `end` moves into the i-th freed slot below it; the recent keys follow in order at end ..
// budget - 1.  Attention does not depend on the order of the keys, and the recent window stays at the end for
// the next call.  No more rows move than have to: min(evicted, kept) at most, and the recent ones.
//
// Select kernel (a CTA per (sequence, K/V head)): the threshold weight by a radix select over the
// order-preserving 32-bit keys, then one ordered pass that lists freed slots and late survivors.
// Move kernel: the rows.  A source slot of one move can be the target of another only from the late
// survivors to the recent block, and inside the recent block from a later to an earlier slot, so one CTA
// moves a (tensor, sequence, head) in that order; columns are independent, and a few long
// caches split their rows into column pieces for more CTAs.
//
// Bound: the moved rows' bytes (K and V, read and written) and 4 bytes per key; below a few
// MB the two launches' latency.
#pragma once
#include "cache_common.cuh"

namespace cache {

struct EvictParams {
    char* k;
    char* v;
    const float* weights;
    float* weights_out;
    const int32_t* seqlens_k;
    int32_t* seqlens_out;
    Pages pages;
    int B, Hkv, row_bytes;
    int budget, sinks, recent;
    int pieces;                // column pieces of a row
    // workspace
    int32_t* owner;            // [num_pages]: -1, the sequence that uses the page, or -2 for several uses
    int32_t* lens;             // [B]
    int32_t* moves;            // [B][Hkv]: rows that move into freed slots
    int32_t* list;             // [B][Hkv][2 * most_moves]: freed slots, then the survivors that fill them
    long long most_moves;
};

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;

// order-preserving: a < b as numbers iff key(a) < key(b); -0 equals +0; NaN is 0, below -inf
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ bool valid_len(const EvictParams& p, int n) {
    return n >= 0 && (long long)n <= (long long)p.pages.max_pages * p.pages.page_size;
}

__global__ void __launch_bounds__(kSelThreads, 1) attn_evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int hist[256];
    __shared__ uint32_t prefix_s;
    __shared__ int want_s;
    __shared__ int warp_n[2][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_launch();
    const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
    const int n = __ldg(p.seqlens_k + b);
    const long long room = (long long)p.pages.max_pages * p.pages.page_size;
    const bool ok = valid_len(p, n);
    if (h == 0) {
        if (tid == 0) p.lens[b] = n;
        if (ok) {
            const int used = n > 0 ? (n - 1) / p.pages.page_size + 1 : 0;
            for (int i = tid; i < used; i += kSelThreads) {
                const int pg = __ldg(p.pages.table + (long long)b * p.pages.max_pages + i);
                if ((unsigned)pg < (unsigned)p.pages.num_pages && atomicCAS(p.owner + pg, -1, b) != -1)
                    atomicExch(p.owner + pg, -2);
            }
        }
    }
    if (!ok || n <= p.budget) return;
    const float* w = p.weights + blockIdx.x * room;
    const int lo = p.sinks, hi = n - p.recent, keep = p.budget - p.sinks - p.recent, end = p.budget - p.recent;
    // the keep-th largest key of [lo, hi), and how many equal to it are kept
    uint32_t prefix = 0;
    int want = keep;
    if (keep > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int j = lo + tid; j < hi; j += kSelThreads) {
                const uint32_t key = weight_key(w[j]);
                if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
            }
            __syncthreads();
            if (warp == 0) {
                // lane i holds bins 8i .. 8i + 7; counts of larger bins from the top
                int mine = 0;
                for (int e = 0; e < 8; ++e) mine += hist[lane * 8 + e];
                int above = mine;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int x = __shfl_down_sync(0xFFFFFFFFu, above, off);
                    if (lane + off < 32) above += x;
                }
                above -= mine;
                if (above < want && above + mine >= want) {
                    int e = 7;
                    while (above + hist[lane * 8 + e] < want) above += hist[lane * 8 + e--];
                    prefix_s = (prefix << 8) | (uint32_t)(lane * 8 + e);
                    want_s = want - above;
                }
            }
            __syncthreads();
            prefix = prefix_s;
            want = want_s;
        }
    }
    // freed slots below `end`, then survivors past it, in order
    int32_t* list = p.list + blockIdx.x * 2 * p.most_moves;
    int listed = 0, ties = 0;
    for (int base = lo; base < hi; base += kSelThreads) {
        const int j = base + tid;
        const uint32_t key = j < hi ? weight_key(w[j]) : 0u;
        const bool in = j < hi && keep > 0, tie = in && key == prefix;
        const unsigned tb = __ballot_sync(0xFFFFFFFFu, tie);
        if (lane == 0) warp_n[0][warp] = __popc(tb);
        __syncthreads();
        int before = 0, all = 0;
        for (int i = 0; i < 32; ++i) {
            const int x = warp_n[0][i];
            before += i < warp ? x : 0;
            all += x;
        }
        const bool kept = in && (key > prefix || (tie && ties + before + __popc(tb & ((1u << lane) - 1)) < want));
        ties += all;
        const bool out = j < hi && (j < end ? !kept : kept);
        const unsigned ob = __ballot_sync(0xFFFFFFFFu, out);
        if (lane == 0) warp_n[1][warp] = __popc(ob);
        __syncthreads();
        before = all = 0;
        for (int i = 0; i < 32; ++i) {
            const int x = warp_n[1][i];
            before += i < warp ? x : 0;
            all += x;
        }
        if (out) list[listed + before + __popc(ob & ((1u << lane) - 1))] = j;
        listed += all;
    }
    if (tid == 0) p.moves[blockIdx.x] = listed >> 1;
}

// One CTA per (sequence, K/V head) and task: a column piece of K or V, or the weights.
__global__ void __launch_bounds__(kMoveThreads) attn_evict_move_kernel(const __grid_constant__ EvictParams p) {
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch();
    const int tasks = 2 * p.pieces + 1;
    const long long bh = blockIdx.x / tasks;
    const int task = (int)(blockIdx.x - bh * tasks);
    const int b = (int)(bh / p.Hkv), h = (int)(bh - (long long)b * p.Hkv);
    const int n = p.lens[b];
    const long long room = (long long)p.pages.max_pages * p.pages.page_size;
    const bool weights = task == tasks - 1;
    bool bad = !valid_len(p, n);
    const bool over = !bad && n > p.budget;
    const int32_t* table = p.pages.table + (long long)b * p.pages.max_pages;
    if (over) {
        // every used page has to be the sequence's alone
        const int used = (n - 1) / p.pages.page_size + 1;
        int wrong = 0;
        for (int i = tid; i < used; i += kMoveThreads) {
            const int pg = __ldg(table + i);
            wrong |= (unsigned)pg >= (unsigned)p.pages.num_pages || p.owner[pg] != b;
        }
        bad = __syncthreads_or(wrong);
    }
    if (weights && h == 0 && tid == 0) {
        if (bad) report_invalid(ATTN_CACHE_SITE_EVICT);
        p.seqlens_out[b] = over && !bad ? p.budget : n;
    }
    if (bad) return;
    const int end = p.budget - p.recent, shift = n - p.budget;
    const int moves = over ? p.moves[bh] : 0;
    const int32_t* freed = p.list + bh * 2 * p.most_moves;
    const int32_t* late = freed + moves;

    if (weights) {
        const float* w = p.weights + bh * room;
        float* out = p.weights_out + bh * room;
        if (out != w)
            for (int j = tid; j < (over ? end : n); j += kMoveThreads) out[j] = w[j];
        if (!over) return;
        __syncthreads();
        for (int i = tid; i < moves; i += kMoveThreads) out[freed[i]] = w[late[i]];
        __syncthreads();
        for (int i0 = 0; i0 < p.recent; i0 += kMoveThreads) {
            const int i = i0 + tid;
            const float x = i < p.recent ? w[n - p.recent + i] : 0.0f;
            __syncthreads();           // (a slot is read before it is written: targets lie below the sources left)
            if (i < p.recent) out[end + i] = x;
        }
        __syncthreads();
        for (int j = p.budget + tid; j < n; j += kMoveThreads) out[j] = 0.0f;
        return;
    }
    if (!over) return;

    const int piece = task % p.pieces, bytes = p.row_bytes / p.pieces;   // 32 .. 256 bytes
    const int lanes = bytes / 16, rows = kMoveThreads / lanes;
    char* base = (task < p.pieces ? p.k : p.v) + (long long)h * p.row_bytes + piece * bytes + (tid % lanes) * 16;
    const long long stride = (long long)p.Hkv * p.row_bytes;
    const int r = tid / lanes;
    constexpr int kU = 4;
    for (int i0 = 0; i0 < moves; i0 += rows * kU) {
        uint4 x[kU];
        int to[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * rows + r;
            to[u] = -1;
            if (i < moves) {
                to[u] = page_row(p.pages, table, freed[i]);
                x[u] = *reinterpret_cast<const uint4*>(base + page_row(p.pages, table, late[i]) * stride);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (to[u] >= 0) *reinterpret_cast<uint4*>(base + to[u] * stride) = x[u];
    }
    __syncthreads();                   // the late survivors are out before the recent block covers their slots
    for (int i0 = 0; i0 < p.recent; i0 += rows * kU) {
        uint4 x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * rows + r;
            if (i < p.recent)
                x[u] = *reinterpret_cast<const uint4*>(base + page_row(p.pages, table, n - p.recent + i) * stride);
        }
        // this step's reads before its writes; its targets lie below every later step's sources
        if (shift < p.recent) __syncthreads();
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * rows + r;
            if (i < p.recent) *reinterpret_cast<uint4*>(base + page_row(p.pages, table, end + i) * stride) = x[u];
        }
    }
}

}  // namespace cache
