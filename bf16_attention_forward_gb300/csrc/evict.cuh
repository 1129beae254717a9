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
// order-preserving 32-bit keys that stay in registers (up to 16 a thread; longer rows are read again for
// each pass).  A histogram of the upper 11 bits, summed over the cluster, gives the bin of the threshold, and
// two more histograms (of 11 and 10 bits) of that bin's keys the threshold itself; a bin of up to 4096 keys
// is gathered into every CTA's registers for that, which spares those two the cluster's exchange and the
// walk over all keys.  An ordered pass then lists freed slots and late survivors.
// Fill kernel: the rows that move into freed slots.  Their sources and targets are disjoint, so all
// sequences' moves lie on one list (in no fixed order) that the warps share evenly.
// Shift kernel: the recent block, and the weights.  Its rows may overlap their targets, so one CTA
// moves a (tensor, sequence, head) in ascending order, each step's reads before its writes; columns are
// independent, and a few long caches split their rows into column pieces for more CTAs.
// Where few rows can move (kMostWhole), each select CTA moves its own, and fill and shift are not launched
// (32 caches a few keys over 1024, 8 heads: 19.5 -> 14.2 us).  The host decides that, and the clusters, by the slots
// that the table has room for, since lengths are on the device: the same caches in tables of 1280 slots take 14.3 us, of
// 1536 (four kernels) 17.3, of 4096 24.7 and of 32,768 (clusters; the weights' rows lie far apart) 38.5.
//
// Bound: the moved rows' bytes (K and V, read and written) and 4 bytes per key; below a few MB the
// launches' latency.  16 caches of 2048 to 16,384 keys, 8 heads, to 4096: 69 us, of them 18 for select (one
// SM per head, its phases' barriers and instructions), 38 for fill (0.28 GB, 7 TB/s) and 9 for shift.
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
    // workspace
    int32_t* uses;             // [num_pages]: table entries of used pages that name the page
    int32_t* cut;              // [B]: the length n of a sequence that is cut, -1 - n of one that fits, 0: refused
    int32_t* lens;             // [B]: lengths after the call (seqlens_out may be seqlens_k, which the select kernel reads)
    int32_t* total;            // moves on the fill list
    int32_t *to, *from;        // [B * Hkv * most_moves]: rows of [cache rows * Hkv]
    uint32_t *w_to, *w_from;   // the same as elements of weights
};

constexpr int kPrepThreads = 1024;
constexpr int kPrepCtas = 8;
constexpr int kMostCluster = 8;        // (16 took 25 us longer to start, for 1 us less in the select kernel)
constexpr int kBins = 2048;
constexpr int kMostGathered = 2 * kBins;   // keys of the threshold's bin that are searched in registers
constexpr int kMostWhole = 256;        // most moves, and most recent keys, that the select kernel does itself
constexpr int kMostRanked = 128;       // ... and up to which each key's rank says it (0.6 us less than the two passes)
constexpr int kListRows = 8;           // rows of 32 slots that a warp lists at a time
constexpr int kHeldMost = 16;          // rows of 32 slots whose keys a warp of 1024 threads' CTA holds in registers
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
// (a CTA that is not launched in a cluster is one of size 1)
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_add(uint32_t addr, int v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
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
    pdl_launch();                                      // (not sooner: select reads lengths and weights at once)
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
        if (lane == 0) {
            if (bad) report_invalid(ATTN_CACHE_SITE_EVICT);
            p.cut[b] = bad ? 0 : over ? n : -1 - n;
            p.lens[b] = over && !bad ? p.budget : n;
        }
    }
}

// The recent block of a head's rows, 16 bytes a thread: `base` is the thread's place in a row, r its row of `rows` that
// a step moves. Each step's reads come before its writes, and its targets lie below every later step's sources.
__device__ __forceinline__ void shift_rows(const EvictParams& p, const int32_t* table, char* base, int n, int r, int rows) {
    constexpr int kU = 8;                              // rows in flight
    const long long stride = (long long)p.Hkv * p.row_bytes;
    const int end = p.budget - p.recent;
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
        if (n - p.budget < p.recent) __syncthreads();  // (else sources and targets do not overlap)
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (to[u] >= 0) *reinterpret_cast<uint4*>(base + to[u] * stride) = x[u];
    }
}

// The recent block of a head's weights, and zeros behind the budget (if the new weights take the place of the old).
__device__ __forceinline__ void shift_weights(const EvictParams& p, const float* w, float* out, int n, int tid, int threads) {
    constexpr int kU = 8;
    const int end = p.budget - p.recent;
    for (int i0 = 0; i0 < p.recent; i0 += kU * threads) {
        float x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (i0 + u * threads + tid < p.recent) x[u] = w[n - p.recent + i0 + u * threads + tid];
        __syncthreads();                               // (as above)
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (i0 + u * threads + tid < p.recent) out[end + i0 + u * threads + tid] = x[u];
    }
    __syncthreads();
    if (out == w)
        for (int j = p.budget + tid; j < n; j += threads) out[j] = 0.0f;
}

// It starts while the prepare kernel runs, and waits for that before it touches what that one writes, and before it
// writes anything.  What it reads sooner, lengths and weights, the prepare kernel does not write, and all that ran before
// the prepare kernel is complete once that lets this one start.
// kWhole: the CTA (a cluster of one) moves its own rows too, in place of the fill and shift kernels.
template <int T, bool kWhole>
__global__ void __launch_bounds__(T, 1024 / T) attn_evict_select_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kWarps = T / 32, kU = 16;            // kU: loads in flight
    constexpr int kEach = kMostGathered / T;
    constexpr int kHeldRows = T == 1024 ? kHeldMost : 4, kList = kHeldRows < kListRows ? kHeldRows : kListRows;
    __shared__ __align__(16) int pool[4][kBins];
    int* const hist = pool[0];                         // this CTA's counts,
    int(* const sum_s)[kBins] = &pool[1];              // and the cluster's of each pass;
    uint32_t* const near_s = reinterpret_cast<uint32_t*>(pool[2]);   // instead of the last two, its keys of the
                                                                     // threshold's bin;
    static_assert(kWarps * kListRows * 32 * 2 <= 2 * sizeof pool[0], "the warps' lists take the place of the first two");
    uint16_t* const slot_s = reinterpret_cast<uint16_t*>(pool[0]) + (threadIdx.x >> 5) * (kListRows * 32);
    __shared__ int near_n, warp_n[2][kWarps];
    __shared__ int count_s[2][kWarps];     // ties and listed slots of each warp, read by the cluster
    __shared__ int start_s;                // rank 0: the row's place on the fill list
    __shared__ uint32_t prefix_s;
    __shared__ int want_s, tied_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned below = (1u << lane) - 1;
    const int C = p.cluster, rank = blockIdx.x % C, bh = blockIdx.x / C;
    const int b = bh / p.Hkv, h = bh - b * p.Hkv;
    pdl_launch();
    const int n = __ldg(p.seqlens_k + b);
    const long long room = (long long)p.pages.max_pages * p.pages.page_size;
    const float* w = p.weights + bh * room;
    float* out = p.weights_out + bh * room;
    // slots j0 .. j1 - 1 of the weights as they are, where the new ones have a buffer of their own
    auto copy_weights = [&](int j0, int j1, int thread, int threads) {
        for (int j = j0 + thread; j < j1; j += kU * threads) {
            float x[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (j + u * threads < j1) x[u] = w[j + u * threads];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (j + u * threads < j1) out[j + u * threads] = x[u];
        }
    };
    if (!valid_len(p, n) || n <= p.budget) {           // (the whole cluster)
        pdl_wait();                                    // the kernels behind this one rely on the one before it too
        if (out != w && rank == 0 && valid_len(p, n)) copy_weights(0, n, tid, T);
        if (kWhole && h == 0 && tid == 0 && p.seqlens_out != p.seqlens_k) p.seqlens_out[b] = p.lens[b];
        return;
    }
    const int32_t* table = p.pages.table + (long long)b * p.pages.max_pages;
    const int keep = p.budget - p.sinks - p.recent, end = p.budget - p.recent;
    // The slots between the sinks and the recent ones go to the warps of the cluster in runs of `run`, CTA by CTA within
    // a warp number: freed slots lie at the front and would otherwise all be one CTA's.
    const int all_slots = n - p.recent - p.sinks, run = ((all_slots - 1) / (C * T) + 1) * 32;
    const int place = warp * C + rank;                 // of this warp among the cluster's
    const int wlo = p.sinks + min(place * run, all_slots), whi = min(wlo + run, n - p.recent);
    // Their keys, kHeldRows rows of 32 slots at a time: row r of chunk c holds slots wlo + 32 (kHeldRows c + r) + lane.
    const int chunks = (run / 32 - 1) / kHeldRows + 1; // (the same for the whole cluster)
    const bool held = chunks == 1;                     // loaded once, for the histogram's first pass
    uint32_t key[kHeldRows];
    int rows = 0, mine_n = 0;                          // of the chunk: the warp's rows, and this lane's keys
    auto load = [&](int c) {
        const int left = whi - wlo - c * (32 * kHeldRows);
        const float* from = w + wlo + c * (32 * kHeldRows) + lane;
        rows = min(max((left + 31) / 32, 0), kHeldRows);
        mine_n = min(max((left - lane + 31) / 32, 0), kHeldRows);
        float x[kHeldRows];
#pragma unroll
        for (int r = 0; r < kHeldRows; ++r)
            if (r < mine_n) x[r] = from[32 * r];
#pragma unroll
        for (int r = 0; r < kHeldRows; ++r) key[r] = r < mine_n ? weight_key(x[r]) : 0u;
    };
    for (int i = tid; i < 4 * kBins; i += T) pool[0][i] = 0;
    if (tid == 0) near_n = 0;
    if (C > 1) cluster_sync(); else __syncthreads();   // no CTA adds to another's counts before they are zero

    // the keep-th largest key of the row, and how many equal to it are kept
    uint32_t prefix = 0;
    int want = keep, tied = 0;
    bool gathered = false;
    int first_tied = 0;
    uint32_t near[kEach];
    for (int pass = 0; pass < 3 && keep > 0; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        if (gathered) {
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                if (tid + e * T < first_tied && (near[e] >> (shift + bits)) == prefix)
                    atomicAdd(&hist[(near[e] >> shift) & ((1u << bits) - 1)], 1);
        } else {
            for (int c = 0; c < chunks; ++c) {
                if (pass == 0 || !held) load(c);
#pragma unroll
                for (int r = 0; r < kHeldRows; ++r) {
                    if (r >= rows) break;
                    if (r < mine_n && (pass == 0 || (key[r] >> (shift + bits)) == prefix))
                        atomicAdd(&hist[(key[r] >> shift) & ((1u << bits) - 1)], 1);
                }
            }
        }
        __syncthreads();
        // of the first 512 threads thread t takes bins 4t .. 4t + 3: few are not empty, and those go to every CTA
        int4 mine = make_int4(0, 0, 0, 0);
        int* to = &sum_s[pass][4 * tid];
        if (tid < kBins / 4) {
            int4* from = reinterpret_cast<int4*>(&hist[4 * tid]);
            mine = *from;
            *from = make_int4(0, 0, 0, 0);
            if (C > 1 && !gathered)
                for (int r = 0; r < C; ++r) {
                    const uint32_t at = cluster_map(ptx::smem_u32(to), r);
                    if (mine.x) cluster_add(at, mine.x);
                    if (mine.y) cluster_add(at + 4, mine.y);
                    if (mine.z) cluster_add(at + 8, mine.z);
                    if (mine.w) cluster_add(at + 12, mine.w);
                }
        }
        if (C > 1 && !gathered) {
            cluster_sync();
            if (tid < kBins / 4) mine = *reinterpret_cast<const int4*>(to);
        }
        // larger bins: of the warps behind this one, then (in the one warp that holds the threshold) of the lanes
        const int count = mine.x + mine.y + mine.z + mine.w, in_warp = __reduce_add_sync(0xFFFFFFFFu, count);
        if (lane == 0) warp_n[pass & 1][warp] = in_warp;
        __syncthreads();
        const int behind = __reduce_add_sync(0xFFFFFFFFu, lane < kBins / 4 / 32 && lane > warp ? warp_n[pass & 1][lane] : 0);
        if (behind < want && behind + in_warp >= want) {
            int above = count;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_down_sync(0xFFFFFFFFu, above, off);
                if (lane + off < 32) above += x;
            }
            above += behind - count;
            if (above < want && above + count >= want) {
                int e = 3, c = mine.w;
                if (above + c < want) { above += c; e = 2; c = mine.z; }
                if (e == 2 && above + c < want) { above += c; e = 1; c = mine.y; }
                if (e == 1 && above + c < want) { above += c; e = 0; c = mine.x; }
                prefix_s = (prefix << bits) | (uint32_t)(4 * tid + e);
                want_s = want - above;
                tied_s = c;
            }
        }
        __syncthreads();
        prefix = prefix_s;
        want = want_s;
        tied = tied_s;
        if (pass > 0 || !held || tied > kMostGathered) continue;

        // gather the bin's keys, of every CTA
#pragma unroll
        for (int r = 0; r < kHeldRows; ++r) {
            if (r >= rows) break;
            if (r < mine_n && (key[r] >> 21) == prefix) near_s[atomicAdd(&near_n, 1)] = key[r];
        }
        if (C > 1) cluster_sync(); else __syncthreads();
        if (C == 1 && tied <= kMostRanked) {           // each key's rank among them
            if (tid < tied) {
                const uint32_t key = near_s[tid];
                int larger = 0, equal = 0;
#pragma unroll 4
                for (int i = 0; i < tied; ++i) {
                    larger += near_s[i] > key;
                    equal += near_s[i] == key;
                }
                if (larger < want && larger + equal >= want) {       // (keys equal to the threshold write the same)
                    prefix_s = key;
                    want_s = want - larger;
                    tied_s = equal;
                }
            }
            __syncthreads();
            prefix = prefix_s;
            want = want_s;
            tied = tied_s;
            break;
        }
        gathered = true;
        first_tied = tied;
        const int near_r = lane < C ? cluster_ld(cluster_map(ptx::smem_u32(&near_n), lane)) : 0;
        int before[kEach], from[kEach];                // keys of the CTAs before the one that holds key tid + e * T
#pragma unroll
        for (int e = 0; e < kEach; ++e) before[e] = from[e] = 0;
        int sum = 0;
        for (int r = 0; r + 1 < C; ++r) {
            sum += __shfl_sync(0xFFFFFFFFu, near_r, r);
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                if (tid + e * T >= sum) { before[e] = sum; from[e] = r + 1; }
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (tid + e * T < tied)
                near[e] = (uint32_t)cluster_ld(cluster_map(ptx::smem_u32(near_s) + 4 * (tid + e * T - before[e]), from[e]));
    }

    if (keep == 0 && held) load(0);                    // (no pass has; only the slots matter then)
    // Of a count of this warp's: the sum over the warps before it in the cluster, and over all.  Every warp of the
    // cluster leaves its count in its CTA, and each reads them all.
    auto sums_before = [&](int count, int which, int& all) {
        if (lane == 0) count_s[which][warp] = count;
        if (C > 1) cluster_sync(); else __syncthreads();
        int before = 0, total = 0;
        for (int r = 0; r < C; ++r) {
            const uint32_t from = ptx::smem_u32(&count_s[which][lane]);
            const int x = lane < kWarps ? (C > 1 ? cluster_ld(cluster_map(from, r)) : count_s[which][lane]) : 0;
            total += x;
            before += lane * C + r < place ? x : 0;
        }
        all = __reduce_add_sync(0xFFFFFFFFu, total);
        return __reduce_add_sync(0xFFFFFFFFu, before);
    };
    // of the keys equal to the threshold the first `want` are kept: where not all are, their ranks count
    int ties = 0, all = 0;                 // ties before this warp's slots
    const bool some = tied > want;
    if (some) {
        int count = 0;
        for (int c = 0; c < chunks; ++c) {
            if (!held) load(c);
#pragma unroll
            for (int r = 0; r < kHeldRows; ++r) {
                if (r >= rows) break;
                count += __popc(__ballot_sync(0xFFFFFFFFu, r < mine_n && key[r] == prefix));
            }
        }
        ties = sums_before(count, 0, all);
    }
    // listed are freed slots below `end` and survivors at or past it: counted here, and listed below
    const uint32_t least = keep > 0 ? prefix : 0xFFFFFFFFu;      // (above every key)
    auto listed = [&](int c, int r, int& seen) {
        bool kept = key[r] >= least;
        if (some) {
            const bool tie = r < mine_n && key[r] == prefix;
            const unsigned tb = __ballot_sync(0xFFFFFFFFu, tie);
            if (tie) kept = seen + __popc(tb & below) < want;
            seen += __popc(tb);
        }
        const bool late = wlo + 32 * (kHeldRows * c + r) + lane >= end;
        return __ballot_sync(0xFFFFFFFFu, r < mine_n && kept == late);
    };
    int count = 0, seen = ties;
    for (int c = 0; c < chunks; ++c) {
        if (!held) load(c);
#pragma unroll
        for (int r = 0; r < kHeldRows; ++r) {
            if (r >= rows) break;
            count += __popc(listed(c, r, seen));
        }
    }
    int at = sums_before(count, 1, all);
    pdl_wait();                            // the prepare kernel's verdict, and its zero in p.total
    const bool stays = p.cut[b] == 0;
    const int moves = stays ? 0 : all >> 1;
    if (!kWhole && rank == 0 && tid == 0) start_s = atomicAdd(p.total, moves);
    if (out != w && !stays) {
        if (rank == 0) copy_weights(0, p.sinks, tid, T);
        copy_weights(wlo, min(whi, end), lane, 32);
        for (int j = p.budget + rank * T + tid; j < n; j += C * T) out[j] = 0.0f;
    }
    if (C > 1) cluster_sync(); else __syncthreads();
    const int start = kWhole ? 0 : C > 1 ? cluster_ld(cluster_map(ptx::smem_u32(&start_s), 0)) : start_s;
    int* const list = pool[2];                         // kWhole: freed slots, then the survivors that fill them
    const uint32_t w0 = (uint32_t)(bh * room);
    seen = ties;
    for (int c = 0; moves > 0 && c < chunks; ++c) {
        if (!held) load(c);
#pragma unroll
        for (int r0 = 0; r0 < kHeldRows; r0 += kList) {
            if (r0 >= rows) break;
            // slots (from j0 on) that are listed, close together: about one in four is, and each costs a page lookup
            const int j0 = wlo + 32 * (kHeldRows * c + r0);
            int m = 0;
#pragma unroll
            for (int r = 0; r < kList; ++r) {
                if (r0 + r >= rows) break;
                const unsigned bits = listed(c, r0 + r, seen);
                if ((bits >> lane) & 1) slot_s[m + __popc(bits & below)] = (uint16_t)(32 * r + lane);
                m += __popc(bits);
            }
            __syncwarp();
            if constexpr (kWhole) {
                for (int e = lane; e < m; e += 32) list[at + e] = j0 + slot_s[e];
                at += m;
                __syncwarp();
                continue;
            }
            constexpr int kE = 4;              // page lookups in flight
            for (int e0 = lane; e0 < m; e0 += 32 * kE) {
                int j[kE], row[kE];
#pragma unroll
                for (int u = 0; u < kE; ++u)
                    if (e0 + 32 * u < m) {
                        j[u] = j0 + slot_s[e0 + 32 * u];
                        row[u] = page_row(p.pages, table, j[u]) * p.Hkv + h;
                    }
#pragma unroll
                for (int u = 0; u < kE; ++u) {
                    const int i = at + e0 + 32 * u;
                    if (e0 + 32 * u >= m) continue;
                    const uint32_t we = w0 + (uint32_t)j[u];
                    (i < moves ? p.to + start : p.from + start - moves)[i] = row[u];
                    (i < moves ? p.w_to + start : p.w_from + start - moves)[i] = we;
                }
            }
            at += m;
            __syncwarp();
        }
    }
    if (C > 1) cluster_sync();             // no CTA leaves while its shared memory may be read
    if constexpr (kWhole) {
        // (lengths in place are the next kernel's: another head's CTA may not have read them yet)
        if (h == 0 && tid == 0 && p.seqlens_out != p.seqlens_k) p.seqlens_out[b] = p.lens[b];
        if (stays) return;
        __syncthreads();                   // the list is complete
        const int lanes = p.row_bytes / 16, rows = T / (2 * lanes), r = tid / (2 * lanes), c = tid % (2 * lanes);
        char* base = (c < lanes ? p.k : p.v) + (long long)h * p.row_bytes + (c % lanes) * 16;
        const long long stride = (long long)p.Hkv * p.row_bytes;
        for (int i = tid; i < moves; i += T) out[list[i]] = w[list[moves + i]];
        for (int i0 = r; i0 < moves; i0 += 4 * rows) {
            uint4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + u * rows < moves)
                    x[u] = *reinterpret_cast<const uint4*>(base + page_row(p.pages, table, list[moves + i0 + u * rows]) * stride);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + u * rows < moves)
                    *reinterpret_cast<uint4*>(base + page_row(p.pages, table, list[i0 + u * rows]) * stride) = x[u];
        }
        __syncthreads();                   // the late survivors are out before the recent block covers their slots
        shift_rows(p, table, base, n, r, rows);
        shift_weights(p, w, out, n, tid, T);
    }
}

// K and V rows and weights into freed slots: 16 bytes a lane, a warp takes 512 bytes of rows at a time, 8 of them in flight.
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
        int to = 0, from = 0;
        if (lane < kU * kPer && m + lane < total) {
            to = p.to[m + lane];
            from = p.from[m + lane];
            p.weights_out[p.w_to[m + lane]] = p.weights[p.w_from[m + lane]];
        }
        uint4 x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int src = __shfl_sync(0xFFFFFFFFu, from, u * kPer + sub);
            if (m + u * kPer + sub < total) x[u] = *reinterpret_cast<const uint4*>(base + (long long)src * (2 * D));
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int dst = __shfl_sync(0xFFFFFFFFu, to, u * kPer + sub);
            if (m + u * kPer + sub < total) *reinterpret_cast<uint4*>(base + (long long)dst * (2 * D)) = x[u];
        }
    }
}

__global__ void __launch_bounds__(256) attn_evict_lens_kernel(const __grid_constant__ EvictParams p) {
    pdl_wait();
    pdl_launch();
    for (int b = threadIdx.x; b < p.B; b += 256) p.seqlens_out[b] = p.lens[b];
}

// The recent block and the weights.  One CTA per (sequence, K/V head) and task: a column piece of K or V, or the
// weights.
__global__ void __launch_bounds__(kShiftThreads) attn_evict_shift_kernel(const __grid_constant__ EvictParams p) {
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch();
    const int tasks = 2 * p.pieces + 1;
    const long long bh = blockIdx.x / tasks;
    const int task = (int)(blockIdx.x - bh * tasks);
    const int b = (int)(bh / p.Hkv), h = (int)(bh - (long long)b * p.Hkv);
    const long long room = (long long)p.pages.max_pages * p.pages.page_size;
    const int cut = p.cut[b];
    if (task == tasks - 1 && h == 0 && tid == 0) p.seqlens_out[b] = p.lens[b];
    if (cut == 0) return;
    const bool over = cut > 0;
    const int n = cut;

    if (task == tasks - 1) {
        if (!over) return;
        shift_weights(p, p.weights + bh * room, p.weights_out + bh * room, n, tid, kShiftThreads);
        return;
    }
    if (!over) return;

    const int piece = task % p.pieces, bytes = p.row_bytes / p.pieces;   // 32 .. 256 bytes
    const int lanes = bytes / 16, rows = kShiftThreads / lanes;
    const int32_t* table = p.pages.table + (long long)b * p.pages.max_pages;
    char* base = (task < p.pieces ? p.k : p.v) + (long long)h * p.row_bytes + piece * bytes + (tid % lanes) * 16;
    shift_rows(p, table, base, n, tid / lanes, rows);
}

}  // namespace cache
