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
// Prepare kernel (one cluster of 8 CTAs): counts each page's uses in the table and decides which sequences are
// cut: over the budget, a valid length, every page in the cache and used once.
// Select kernel (a cluster of 1 to 8 CTAs per (sequence, K/V head)): the weights are read once, as
// order-preserving 32-bit keys that stay in shared memory; a radix select of 11 + 11 + 10 bits over the
// cluster's summed histograms gives the threshold, and an ordered pass lists freed slots and late survivors.
// Fill kernel: the rows that move into freed slots.  Their sources and targets are disjoint, so all
// sequences' moves lie on one list (in no fixed order) that the warps share evenly.
// Shift kernel: the recent block, and the weights.  Its rows may overlap their targets, so one CTA
// moves a (tensor, sequence, head) in ascending order, each step's reads before its writes; columns are
// independent, and a few long caches split their rows into column pieces for more CTAs.
//
// Bound: the moved rows' bytes (K and V, read and written) and 4 bytes per key; below a few
// MB the launches' latency.
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
    int cluster;               // CTAs of a (sequence, K/V head) in the select kernel
    int pieces;                // column pieces of a row in the shift kernel
    int staged;                // keys that a select CTA has room for in shared memory
    // workspace
    int32_t* uses;             // [num_pages]: table entries of used pages that name the page
    int32_t* cut;              // [B]: the length n of a sequence that is cut, -1 - n of one that fits, 0: refused
    int32_t* total;            // moves on the fill list
    int32_t* moves;            // [B][Hkv]: rows that move into freed slots
    int32_t* list;             // [B][Hkv][2 * most_moves]: freed slots, then the survivors that fill them
    int2* fill;                // [B * Hkv * most_moves]: (to, from) as rows of [cache rows * Hkv]
    long long most_moves;
};

constexpr int kPrepThreads = 1024;
constexpr int kPrepCtas = 8;
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMostStaged = 16384;     // 64 KB: three CTAs an SM
constexpr int kFillThreads = 256;
constexpr int kShiftThreads = 256;

// order-preserving: a < b as numbers iff key(a) < key(b); -0 equals +0; NaN is 0, below -inf
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ bool valid_len(const EvictParams& p, int n) {
    return n >= 0 && (long long)n <= (long long)p.pages.max_pages * p.pages.page_size;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// (a CTA that is not launched in a cluster is one of size 1)
__device__ __forceinline__ int4 cluster_ld4(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int cluster_ld(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__global__ void __launch_bounds__(kPrepThreads, 1) attn_evict_prep_kernel(const __grid_constant__ EvictParams p) {
    const int tid = blockIdx.x * kPrepThreads + threadIdx.x, lane = threadIdx.x & 31, warp = tid >> 5;
    constexpr int kThreads = kPrepThreads * kPrepCtas;
    pdl_wait();
    pdl_launch();
    for (int i = tid; i < p.pages.num_pages; i += kThreads) p.uses[i] = 0;
    if (tid == 0) *p.total = 0;
    cluster_sync();
    // a warp per sequence
    for (int b = warp; b < p.B; b += kThreads / 32) {
        const int n = __ldg(p.seqlens_k + b);
        if (n < 1 || !valid_len(p, n)) continue;
        const int used = (n - 1) / p.pages.page_size + 1;
#pragma unroll 4
        for (int i = lane; i < used; i += 32) {
            const int pg = __ldg(p.pages.table + (long long)b * p.pages.max_pages + i);
            if ((unsigned)pg < (unsigned)p.pages.num_pages) atomicAdd(p.uses + pg, 1);
        }
    }
    cluster_sync();
    for (int b = warp; b < p.B; b += kThreads / 32) {
        const int n = __ldg(p.seqlens_k + b);
        const bool valid = valid_len(p, n), over = valid && n > p.budget;
        bool bad = !valid;
        if (over) {
            const int used = (n - 1) / p.pages.page_size + 1;
#pragma unroll 4
            for (int i = lane; i < used; i += 32) {
                const int pg = __ldg(p.pages.table + (long long)b * p.pages.max_pages + i);
                bad |= (unsigned)pg >= (unsigned)p.pages.num_pages || __ldcg(p.uses + pg) != 1;
            }
            bad = __any_sync(0xFFFFFFFFu, bad);
        }
        __syncwarp();                      // seqlens_out may be seqlens_k: every lane has read it
        if (lane == 0) {
            if (bad) report_invalid(ATTN_CACHE_SITE_EVICT);
            p.cut[b] = bad ? 0 : over ? n : -1 - n;
            p.seqlens_out[b] = over && !bad ? p.budget : n;
        }
    }
}

__global__ void __launch_bounds__(kSelThreads) attn_evict_select_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ uint32_t key_s[];
    __shared__ __align__(16) int hist[3][kBins];
    __shared__ int warp_n[3][kSelWarps];
    __shared__ int total_s[2];             // ties and listed slots of this CTA, read by the cluster
    __shared__ int start_s;                // rank 0: the row's place on the fill list
    __shared__ uint32_t prefix_s;
    __shared__ int want_s, tied_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned below = (1u << lane) - 1;
    pdl_wait();
    pdl_launch();
    const int C = p.cluster, rank = blockIdx.x % C, bh = blockIdx.x / C;
    const int b = bh / p.Hkv, h = bh - b * p.Hkv;
    const int n = p.cut[b];
    if (n <= 0) return;                    // (the whole cluster)
    const long long room = (long long)p.pages.max_pages * p.pages.page_size;
    const int32_t* table = p.pages.table + (long long)b * p.pages.max_pages;
    const float* w = p.weights + bh * room;
    const int keep = p.budget - p.sinks - p.recent, end = p.budget - p.recent;
    // this CTA's slots, and each warp's
    const int per = (n - p.recent - p.sinks - 1) / C + 1;
    const int lo = p.sinks + min(rank * per, n - p.recent - p.sinks), hi = min(lo + per, n - p.recent);
    const bool staged = hi - lo <= p.staged;
    const int per_warp = ((hi - lo - 1) / kSelThreads + 1) * 32;
    const int wlo = min(lo + warp * per_warp, hi), whi = min(wlo + per_warp, hi);
    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
    __syncthreads();

    // the keep-th largest key of the row, and how many equal to it are kept
    uint32_t prefix = 0;
    int want = keep, tied = 0;
    for (int pass = 0; pass < 3 && keep > 0; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        if (pass > 0 && staged) {
            for (int j = tid; j < hi - lo; j += kSelThreads) {
                const uint32_t key = key_s[j];
                if ((key >> (shift + bits)) == prefix) atomicAdd(&hist[pass][(key >> shift) & ((1u << bits) - 1)], 1);
            }
        } else {
            constexpr int kU = 8;          // loads in flight
            for (int j0 = lo + tid; j0 < hi; j0 += kU * kSelThreads) {
                float x[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (j0 + u * kSelThreads < hi) x[u] = w[j0 + u * kSelThreads];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int j = j0 + u * kSelThreads;
                    if (j >= hi) break;
                    const uint32_t key = weight_key(x[u]);
                    if (staged) key_s[j - lo] = key;
                    if (pass == 0 || (key >> (shift + bits)) == prefix) atomicAdd(&hist[pass][(key >> shift) & ((1u << bits) - 1)], 1);
                }
            }
        }
        if (C > 1) cluster_sync(); else __syncthreads();
        // thread t: bins 4t .. 4t + 3, summed over the cluster, and the count of larger bins
        int4 sum = make_int4(0, 0, 0, 0);
        for (int r = 0; r < C; ++r) {
            const int4 x = C > 1 ? cluster_ld4(cluster_map(ptx::smem_u32(&hist[pass][4 * tid]), r))
                                 : *reinterpret_cast<const int4*>(&hist[pass][4 * tid]);
            sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
        }
        const int mine = sum.x + sum.y + sum.z + sum.w;
        int above = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_down_sync(0xFFFFFFFFu, above, off);
            if (lane + off < 32) above += x;
        }
        if (lane == 0) warp_n[pass][warp] = above;
        __syncthreads();
        above -= mine;
        for (int i = warp + 1; i < kSelWarps; ++i) above += warp_n[pass][i];
        if (above < want && above + mine >= want) {
            const int bin[4] = {sum.x, sum.y, sum.z, sum.w};
            int e = 3;
            while (above + bin[e] < want) above += bin[e--];
            prefix_s = (prefix << bits) | (uint32_t)(4 * tid + e);
            want_s = want - above;
            tied_s = bin[e];
        }
        __syncthreads();
        prefix = prefix_s;
        want = want_s;
        tied = tied_s;
    }

    auto key_at = [&](int j) { return staged ? key_s[j - lo] : weight_key(w[j]); };
    // of the keys equal to the threshold the first `want` are kept: where not all are, their ranks count
    int ties = 0;                          // ties before this warp's slots
    const bool some = tied > want;
    if (some) {
        int count = 0;
        for (int j0 = wlo; j0 < whi; j0 += 32)
            count += __popc(__ballot_sync(0xFFFFFFFFu, j0 + lane < whi && key_at(min(j0 + lane, hi - 1)) == prefix));
        if (lane == 0) warp_n[0][warp] = count;
        __syncthreads();
        int all = 0;
        for (int i = 0; i < kSelWarps; ++i) {
            const int x = warp_n[0][i];
            ties += i < warp ? x : 0;
            all += x;
        }
        if (C > 1) {
            if (tid == 0) total_s[0] = all;
            cluster_sync();
            for (int r = 0; r < rank; ++r) ties += cluster_ld(cluster_map(ptx::smem_u32(&total_s[0]), r));
        }
    }
    // freed slots below `end`, and survivors at or past it, counted and then listed in order
    auto out_at = [&](int j0, int& seen) {
        const int j = j0 + lane;
        const bool in = j < whi;
        const uint32_t key = in ? key_at(j) : 0u;
        const bool tie = in && keep > 0 && key == prefix;
        bool kept = in && keep > 0 && (key > prefix || tie);
        if (some) {
            const unsigned tb = __ballot_sync(0xFFFFFFFFu, tie);
            if (tie) kept = seen + __popc(tb & below) < want;
            seen += __popc(tb);
        }
        return in && (j < end ? !kept : kept);
    };
    int count = 0, seen = ties;
    for (int j0 = wlo; j0 < whi; j0 += 32) count += __popc(__ballot_sync(0xFFFFFFFFu, out_at(j0, seen)));
    if (lane == 0) warp_n[1][warp] = count;
    __syncthreads();
    int at = 0, all = 0;
    for (int i = 0; i < kSelWarps; ++i) {
        const int x = warp_n[1][i];
        at += i < warp ? x : 0;
        all += x;
    }
    if (C > 1) {
        if (tid == 0) total_s[1] = all;
        cluster_sync();
        all = 0;
        for (int r = 0; r < C; ++r) {
            const int x = cluster_ld(cluster_map(ptx::smem_u32(&total_s[1]), r));
            at += r < rank ? x : 0;
            all += x;
        }
    }
    const int moves = all >> 1;
    if (rank == 0 && tid == 0) {
        p.moves[bh] = moves;
        start_s = atomicAdd(p.total, moves);
    }
    if (C > 1) cluster_sync(); else __syncthreads();
    int2* fill = p.fill + cluster_ld(cluster_map(ptx::smem_u32(&start_s), 0));
    int32_t* list = p.list + bh * 2 * p.most_moves;
    seen = ties;
    for (int j0 = wlo; j0 < whi; j0 += 32) {
        const bool out = out_at(j0, seen);
        const unsigned ob = __ballot_sync(0xFFFFFFFFu, out);
        if (out) {
            const int i = at + __popc(ob & below), row = page_row(p.pages, table, j0 + lane) * p.Hkv + h;
            list[i] = j0 + lane;
            if (i < moves) fill[i].x = row; else fill[i - moves].y = row;
        }
        at += __popc(ob);
    }
    if (C > 1) cluster_sync();             // no CTA leaves while its shared memory may be read
}

// K and V rows into freed slots: 16 bytes a lane, a warp takes 512 bytes of rows at a time, 8 of them in flight.
template <int D>
__global__ void __launch_bounds__(kFillThreads, 4) attn_evict_fill_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kLanes = 2 * D / 16;                 // lanes of a K (or V) row
    constexpr int kPer = 16 / kLanes;                  // moves of a warp's instruction: 1 or 2
    constexpr int kU = 8;
    pdl_wait();
    pdl_launch();
    const int lane = threadIdx.x & 31, warps = gridDim.x * (kFillThreads / 32);
    const int total = *p.total;
    char* base = (lane < 16 ? p.k : p.v) + (lane % kLanes) * 16;       // lanes 0-15: K, 16-31: V
    const int sub = (lane % 16) / kLanes;
    for (long long m = (long long)(blockIdx.x * (kFillThreads / 32) + (threadIdx.x >> 5)) * kU * kPer; m < total;
         m += (long long)warps * kU * kPer) {
        int2 mv = make_int2(0, 0);
        if (lane < kU * kPer && m + lane < total) mv = p.fill[m + lane];
        uint4 x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int src = __shfl_sync(0xFFFFFFFFu, mv.y, u * kPer + sub);
            if (m + u * kPer + sub < total) x[u] = *reinterpret_cast<const uint4*>(base + (long long)src * (2 * D));
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int dst = __shfl_sync(0xFFFFFFFFu, mv.x, u * kPer + sub);
            if (m + u * kPer + sub < total) *reinterpret_cast<uint4*>(base + (long long)dst * (2 * D)) = x[u];
        }
    }
}

// The recent block and the weights.  One CTA per (sequence, K/V head) and task: a column piece of K or V, or the
// weights.
__global__ void __launch_bounds__(kShiftThreads) attn_evict_shift_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kU = 8;                              // loads in flight
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch();
    const int tasks = 2 * p.pieces + 1;
    const long long bh = blockIdx.x / tasks;
    const int task = (int)(blockIdx.x - bh * tasks);
    const int b = (int)(bh / p.Hkv), h = (int)(bh - (long long)b * p.Hkv);
    const long long room = (long long)p.pages.max_pages * p.pages.page_size;
    const int cut = p.cut[b];
    if (cut == 0) return;
    const bool over = cut > 0;
    const int n = over ? cut : -1 - cut, end = p.budget - p.recent, shift = n - p.budget;

    if (task == tasks - 1) {
        const float* w = p.weights + bh * room;
        float* out = p.weights_out + bh * room;
        if (out != w) {
            const int upto = over ? end : n;
            for (int j0 = tid; j0 < upto; j0 += kU * kShiftThreads) {
                float x[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (j0 + u * kShiftThreads < upto) x[u] = w[j0 + u * kShiftThreads];
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (j0 + u * kShiftThreads < upto) out[j0 + u * kShiftThreads] = x[u];
            }
        }
        if (!over) return;
        const int moves = p.moves[bh];
        const int32_t* freed = p.list + bh * 2 * p.most_moves;
        __syncthreads();
        for (int i0 = tid; i0 < moves; i0 += kU * kShiftThreads) {
            float x[kU];
            int to[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int i = i0 + u * kShiftThreads;
                if (i < moves) {
                    to[u] = freed[i];
                    x[u] = w[freed[moves + i]];
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (i0 + u * kShiftThreads < moves) out[to[u]] = x[u];
        }
        __syncthreads();
        for (int i0 = 0; i0 < p.recent; i0 += kU * kShiftThreads) {
            float x[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (i0 + u * kShiftThreads + tid < p.recent) x[u] = w[n - p.recent + i0 + u * kShiftThreads + tid];
            __syncthreads();           // (a slot is read before it is written: targets lie below the sources left)
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (i0 + u * kShiftThreads + tid < p.recent) out[end + i0 + u * kShiftThreads + tid] = x[u];
        }
        __syncthreads();
        for (int j = p.budget + tid; j < n; j += kShiftThreads) out[j] = 0.0f;
        return;
    }
    if (!over) return;

    const int piece = task % p.pieces, bytes = p.row_bytes / p.pieces;   // 32 .. 256 bytes
    const int lanes = bytes / 16, rows = kShiftThreads / lanes;
    const int32_t* table = p.pages.table + (long long)b * p.pages.max_pages;
    char* base = (task < p.pieces ? p.k : p.v) + (long long)h * p.row_bytes + piece * bytes + (tid % lanes) * 16;
    const long long stride = (long long)p.Hkv * p.row_bytes;
    const int r = tid / lanes;
    for (int i0 = 0; i0 < p.recent; i0 += rows * kU) {
        uint4 x[kU];
        int to[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * rows + r;
            to[u] = -1;
            if (i < p.recent) {
                x[u] = *reinterpret_cast<const uint4*>(base + page_row(p.pages, table, n - p.recent + i) * stride);
                to[u] = page_row(p.pages, table, end + i);
            }
        }
        // this step's reads before its writes; its targets lie below every later step's sources
        if (shift < p.recent) __syncthreads();
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (to[u] >= 0) *reinterpret_cast<uint4*>(base + to[u] * stride) = x[u];
    }
}

}  // namespace cache
