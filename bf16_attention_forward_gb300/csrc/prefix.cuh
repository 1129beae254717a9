// prefix.cuh -- attention of one new token per sequence over keys that the whole batch shares: the shared part, and
// the join with each sequence's own keys (decode.cuh).
//
// Mathematics.  The prefix's keys are the same for all sequences, so the queries of a K/V head's group in all sequences,
// B * G rows (G = H / Hkv), form one matrix against them:
//   S = Q K^T,  m_i = max_j S_ij,  P_ij = exp((S_ij - m_i) / sqrt(d)),  l_i = sum_j P_ij,  O_i = sum_j P_ij v_j,
// with a running m and l over tiles of 128 keys; a row's parts (m, l, O in fp32) and those of its own keys are joined as
// in decode.cuh.
//
// Work.  A unit is a block of rows of a K/V head, with all tiles of keys as its steps.  The steps of all units form one line,
// which one CTA per SM divide evenly (the host knows every length, so the places are arithmetic): a CTA takes a
// contiguous range, and leaves one part for each unit that it meets.  Behind each unit's steps the line has kPfEnd more places,
// for the change of units, which takes as long (without them the CTAs that met one ended 6 to 10 us after the others).
//
// Bound.  Every key of the prefix is read once for a block of 256 rows, and from HBM once for the batch while the prefix fits in
// the L2 (2 * d * 2 bytes); it costs 6 * d * B * G flops (P V twice, below): with some 190 rows and more the tensor pipe bounds it, with fewer
// HBM.  512 sequences of 40 heads, 8 K/V heads, us of this kernel: 4,000 keys 57, 8,000 98, 16,000 178, 32,000 (131 MB) 351: 2.5 a step of
// 25 MFLOP a CTA, 80 % of the measured peak, and 15 for first loads, changes of units and last parts.  So the products run on tcgen05, with queries as the 128
// rows of a tile, S and O in TMEM, P written over S.  Two tiles of P are in work at a time, one softmax warpgroup each,
// so that the products of one run beside the exponentials of the other:
//   more than 128 rows: two tiles of rows against one tile of keys;
//   128 rows and fewer (kSingle): one tile of rows against two tiles of keys, even and odd ones, which keep
//   an m, l and O each.
// P goes to the second product as two bf16 parts, as in decode.cuh (an error of 2^-16, so that a sequence's outputs are as exact
// whichever kernels its batch's size chooses): both fit where S was, and the products are half as many again.  l sums
// the unrounded weights.
//
// Loads.  Three or six warps copy keys and values with cp.async, row by row, into the 128-byte-swizzled tiles that the tensor pipe
// reads: any page size, any number of heads, no tensor maps to make on the host (TMA boxes of a page's rows reach the
// same rate from 64 rows on, and half of HBM's with 8).  A slot's barrier counts the copies as they land, and the
// products' thread sets a proxy fence between that and its first product.  A unit's queries come first, as soon as the unit before
// it has had its last product with its own.
#pragma once
#include "cache_common.cuh"
#include "decode.cuh"

namespace cache {

constexpr int kPfEnd = 2;          // places behind a unit's steps

// x / n = x * mul >> shift for 0 <= x < 2^30 (as in Pages)
struct Divisor {
    uint32_t mul, shift;
    __device__ __forceinline__ int of(int x) const { return (int)(((unsigned long long)(uint32_t)x * mul) >> shift); }
};

struct PrefixParams {
    const __nv_bfloat16* q;        // [B][H][d]
    const char* k;                 // [rows][Hkv][d]
    const char* v;
    Pages pages;                   // table: the first sequence's row
    int H, Hkv, group, rows;       // rows = B * group
    Divisor by_group;
    int prefix_len;
    int row_blocks;                // blocks of 256 rows (kSingle: 128)
    int steps;                     // of a unit: tiles of 128 keys (kSingle: pairs of them); it has steps + kPfEnd places
    int per, more, ctas;           // places of a CTA on the line: `per`, the first `more` CTAs one more
    Divisor by_places, by_per, by_more;    // by a unit's places, per, per + 1
    int slots;                     // parts that a CTA may leave
    float scale_log2;              // log2(e) / sqrt(d)
    float* part_o;                 // [ctas][slots][2][128][d]
    float2* part_ml;               // [ctas][slots][2][128]: (m in logits, l); l = -1: a bad page, or an expired wait
    unsigned long long wait_limit_ns;
    int test_hooks;                // ATTN_TEST_WITHHOLD_O_READY: CTA 0 skips its first share's output-ready signal of tile 0
    // the line has fewer than 2^30 places (the host checks)
    __device__ __forceinline__ int start(int c) const { return per * c + min(c, more); }
    __device__ __forceinline__ int cta_of(int u) const {
        const int v = u - more * (per + 1);
        return v < 0 ? by_more.of(u) : more + by_per.of(v);
    }
};

constexpr int kPfTile = 128;
constexpr int kPfBox = kPfTile * 64 * 2;       // 64 columns of a tile: rows of 128 bytes
constexpr uint32_t kPfTmemCols = 512;          // S0 | S1 | O0 | O1

template <int D, bool kSingle>
struct PfGeo {
    // Warpgroups 0, 1: softmax; warp 9 issues the products, and of the other warps those of other schedulers than its own load: three,
    // or with one tile of rows, where HBM bounds, six in a block of 512 threads (24 sequences of 32 heads, 65,500 keys: 64.1 us,
    // with three 70.2; with two tiles of rows no gain: 512 sequences of 40 heads, 8,000 keys: 152.6, with three 151.0).
    static constexpr int kLoaders = kSingle ? 6 : 3, kThreads = kSingle ? 512 : 384;
    static constexpr uint32_t kRegsSoftmax = kSingle ? 160 : 176, kRegsOther = kSingle ? 96 : 128;
    static_assert(256 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= 65536 / kThreads / 8 * 8 * kThreads, "more registers than at launch");
    static constexpr int kTileBytes = kPfTile * D * 2;
    static constexpr int kQTiles = kSingle ? 1 : 2;
    static constexpr int kStages = 6 * 128 / D - kQTiles;          // all the shared memory that Q and the parts' room leave
    static constexpr int kRing = kQTiles * kTileBytes;
    static constexpr int kRoom = kRing + kStages * kTileBytes;     // 4 KB a softmax warp, on a part's way out
    static constexpr int kBars = kRoom + 8 * 4096;
    // barriers
    static constexpr int kFull = 0, kEmpty = kStages, kQFull = 2 * kStages, kQEmpty = kQFull + 1, kSFull = kQEmpty + 1,
                         kPFull = kSFull + 2, kOFull = kPFull + 2, kDrain = kOFull + 2, kNumBars = kDrain + 1;
    static constexpr int kMisc = kBars + kNumBars * 8;             // TMEM address, abort flag, bad page
    static constexpr int kSmem = kMisc + 16 + 1024;                // from a 1024-byte boundary
    static_assert(kSmem <= 232448, "shared memory over the 227 KB limit");
};

// first timeout (or bad page) wins, as in report_invalid
__device__ __forceinline__ bool pf_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                        unsigned long long limit_ns) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (true) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (ptx::globaltimer_ns() - t0 > limit_ns) {
            if (atomicCAS(&g_status[0], 0u, (uint32_t)ATTN_ERR_DEVICE_TIMEOUT) == 0u)
                atomicExch(&g_status[1], (uint32_t)ATTN_CACHE_SITE_PREFIX);
            *abort_flag = 1u;
            return false;
        }
    }
}

// shared-memory descriptor of a 128-byte-swizzled operand
__device__ __forceinline__ uint64_t pf_desc(uint32_t addr, uint32_t leading, uint32_t stride) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((leading >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((stride >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// instruction descriptor: bf16 x bf16 -> fp32, M = 128, N columns, B along its rows or (V) along its columns
__host__ __device__ constexpr uint32_t pf_idesc(int N, bool b_mn) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn ? 1u : 0u) << 16 | (uint32_t)(N >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}
// 16 bytes global -> shared under an L2 policy
__device__ __forceinline__ void pf_copy16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
// the barrier counts this thread's arrival once all its copies so far have landed
__device__ __forceinline__ void pf_arrive_landed(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// where chunk c (16 bytes) of row r is in a tile
__device__ __forceinline__ uint32_t pf_chunk(int r, int c) {
    return (uint32_t)((c >> 3) * kPfBox + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Two weights y (0, 2^-100 or more, or NaN) as bf16 parts: hi the upper 8 bits of y (1 - 2^-16), cut off, lo what is left of y, rounded.
// So the lower part of a positive weight is positive too, and an infinite value stays infinite under it.
__device__ __forceinline__ void pf_parts(float2 y, uint32_t& hi, uint32_t& lo) {
    const float2 z = __fmul2_rn(y, make_float2(1.0f - 0x1p-16f, 1.0f - 0x1p-16f));
    hi = __byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x7632);
    float x0, x1;                  // y - hi, exact
    asm("{\n\t.reg .b16 a, b, m;\n\t"
        "mov.b32 {a, b}, %4;\n\t"
        "mov.b16 m, 0xBF80;\n\t"
        "fma.rn.f32.bf16 %0, a, m, %2;\n\t"
        "fma.rn.f32.bf16 %1, b, m, %3;\n\t}"
        : "=f"(x0), "=f"(x1)
        : "f"(y.x), "f"(y.y), "r"(hi));
    lo = ptx::pack_bf16x2(x0, x1);
}

// A CTA's share of a unit: steps j0 .. j1 - 1.  Units of one K/V head are neighbours, row block by row block.
struct PfShare {
    int j0, j1, rb, kv;
};
struct PfWalk {                    // over the shares of a range u .. end - 1 of the line
    int u, end;
    __device__ __forceinline__ PfWalk(const PrefixParams& p) : u(p.start(blockIdx.x)), end(p.start(blockIdx.x + 1)) {}
    __device__ __forceinline__ bool next(const PrefixParams& p, PfShare& w) {
        const int places = p.steps + kPfEnd;
        int unit = p.by_places.of(u);
        w.j0 = u - unit * places;
        if (w.j0 >= p.steps) {         // (in the places behind a unit)
            w.j0 = 0;
            u = ++unit * places;
        }
        if (u >= end) return false;
        w.j1 = min(p.steps, w.j0 + end - u);
        w.kv = unit / p.row_blocks;
        w.rb = unit - w.kv * p.row_blocks;
        u = w.j1 == p.steps ? (unit + 1) * places : end;
        return true;
    }
};

template <int D, bool kSingle>
__global__ void __launch_bounds__(PfGeo<D, kSingle>::kThreads, 1) attn_prefix_kernel(const __grid_constant__ PrefixParams p) {
    using G = PfGeo<D, kSingle>;
    extern __shared__ __align__(1024) uint8_t pf_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)pf_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = ptx::smem_u32(smem);
    auto bar = [&](int i) { return sbase + (uint32_t)(G::kBars + 8 * i); };
    uint32_t* tmem_holder = (uint32_t*)(smem + G::kMisc);
    volatile uint32_t* abort_flag = (volatile uint32_t*)(smem + G::kMisc + 4);
    volatile uint32_t* bad_flag = (volatile uint32_t*)(smem + G::kMisc + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            ptx::mbar_init(bar(G::kFull + s), 32 * G::kLoaders);
            ptx::mbar_init(bar(G::kEmpty + s), 1);
        }
        ptx::mbar_init(bar(G::kQFull), 32 * G::kLoaders);
        ptx::mbar_init(bar(G::kQEmpty), 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(G::kSFull + i), 1);
            ptx::mbar_init(bar(G::kPFull + i), kPfTile);
            ptx::mbar_init(bar(G::kOFull + i), 1);
        }
        ptx::mbar_init(bar(G::kDrain), 1);
        *abort_flag = *bad_flag = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 9) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_holder), kPfTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const unsigned long long lim = p.wait_limit_ns;
    pdl_wait();
    pdl_launch();

    PfWalk walk(p);
    PfShare w = {};
    // tile of a unit's step j that warpgroup t's rows meet
    auto tile_of = [&](int j, int t) { return kSingle ? 2 * j + t : j; };

    if (warp >= 8) {
        ptx::reg_dealloc<G::kRegsOther>();
        if ((warp & 3) != 1) {
            // ------------------------------------------------------------------ loads
            // In the order in which the products take them: K0 V0 K1 V1 ..., or with two key tiles a step (a, b)
            // Ka0 Kb0, then Va0 Ka1 Vb0 Kb1, ..., and at the end Va Vb of every share.  A tile's 16 groups of 8 rows are dealt to
            // the loading warps; the pages of a tile of keys are looked up once, for its values too, and before the wait for a slot.
            const int who = (warp >= 12 ? 3 : 0) + ((warp & 3) == 0 ? 0 : (warp & 3) - 1);
            constexpr int kChunks = D / 8, kRowsPerCopy = 32 / kChunks, kCopies = 8 / kRowsPerCopy;
            const uint32_t key_stride = (uint32_t)p.Hkv * D * 2;   // (the host refuses more)
            const uint64_t policy = p.row_blocks > 1 ? ptx::policy_evict_last() : ptx::policy_evict_first();
            // Key i = lane + 32 * u of this warp's: row i % 8 of group who + loaders * (i / 8), as page and its slot (-1: behind
            // the prefix).
            constexpr int kGroups = (16 + G::kLoaders - 1) / G::kLoaders, kU = (8 * kGroups + 31) / 32;
            struct Rows { int page[kU], in[kU]; };
            auto lookup = [&](int tile) {
                Rows r;
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int i = lane + 32 * u, in_tile = (who + G::kLoaders * (i >> 3)) * 8 + (i & 7), key = tile * kPfTile + in_tile;
                    const bool there = in_tile < kPfTile && key < p.prefix_len;
                    const int pg = page_of(p.pages, there ? key : 0);
                    r.in[u] = there ? key - pg * p.pages.page_size : -1;
                    r.page[u] = there ? __ldg(p.pages.table + pg) : -1;
                }
                return r;
            };
            // where this lane's 16 bytes of each copy of a group go in a slot (its next group lies 8 * loaders rows on)
            uint32_t to[kCopies];
#pragma unroll
            for (int i = 0; i < kCopies; ++i) to[i] = pf_chunk(who * 8 + i * kRowsPerCopy + lane / kChunks, lane % kChunks);
            const int groups = (16 - who + G::kLoaders - 1) / G::kLoaders;
            uint32_t pos = 0;                                      // loads
            bool ok = true;
            auto load = [&](const char* base, const Rows& f) {
                const uint32_t slot = pos % G::kStages;
                if (pos >= G::kStages) {
                    ok = pf_wait(bar(G::kEmpty + slot), (pos / G::kStages - 1) & 1u, abort_flag, lim);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) return;
                }
                const uint32_t dst = sbase + (uint32_t)G::kRing + slot * G::kTileBytes;
                const char* src = base + (long long)w.kv * D * 2 + (lane % kChunks) * 16;
                bool there = true;
                int row[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const bool good = (unsigned)f.page[u] < (unsigned)p.pages.num_pages;
                    there &= good || lane + 32 * u >= groups * 8;
                    row[u] = good ? f.page[u] * p.pages.page_size + f.in[u] : -1;
                    if (!good && f.in[u] >= 0) {
                        *bad_flag = 1u;
                        report_invalid(ATTN_CACHE_SITE_PREFIX);
                    }
                }
                auto row_of = [&](int n, int i) {
                    return __shfl_sync(0xFFFFFFFFu, n < 4 ? row[0] : row[kU - 1], (n * 8 + i * kRowsPerCopy + lane / kChunks) & 31);
                };
                if (__all_sync(0xFFFFFFFFu, there)) {
                    // (a group's rows are handed over before its copies: one after another, each copy would wait for its own)
#pragma unroll
                    for (int n = 0; n < kGroups; ++n) {
                        if (n == kGroups - 1 && groups < kGroups) break;
                        const char* from[kCopies];
#pragma unroll
                        for (int i = 0; i < kCopies; ++i) from[i] = src + (unsigned long long)key_stride * (uint32_t)row_of(n, i);
#pragma unroll
                        for (int i = 0; i < kCopies; ++i) pf_copy16(dst + to[i] + n * (G::kLoaders * 8 * 128), from[i], policy);
                    }
                } else {
#pragma unroll 1
                    for (int n = 0; n < groups; ++n)
#pragma unroll
                        for (int i = 0; i < kCopies; ++i) {
                            const int x = row_of(n, i);
                            cp_async16(dst + to[i] + n * (G::kLoaders * 8 * 128), src + (unsigned long long)key_stride * (uint32_t)max(x, 0),
                                       x < 0 ? 0u : 16u, policy);
                        }
                }
                pf_arrive_landed(bar(G::kFull + slot));
                ++pos;
            };
#pragma unroll 1
            for (uint32_t n = 0; ok && walk.next(p, w); ++n) {
                {
                    constexpr int kRowsQ = G::kQTiles * kPfTile;
                    if (n > 0) {
                        ok = pf_wait(bar(G::kQEmpty), (n - 1) & 1u, abort_flag, lim);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                    }
                    const __nv_bfloat16* from = p.q + (long long)w.kv * p.group * D + lane % kChunks * 8;
#pragma unroll 4
                    for (int i = who; i < kRowsQ / kRowsPerCopy; i += G::kLoaders) {
                        const int r = i * kRowsPerCopy + lane / kChunks, x = w.rb * kRowsQ + r, b = p.by_group.of(x);
                        const bool there = x < p.rows;
                        cp_async16(sbase + (uint32_t)((r / kPfTile) * G::kTileBytes) + pf_chunk(r % kPfTile, lane % kChunks),
                                   from + (there ? ((long long)b * p.H + x - b * p.group) * D : 0), there ? 16u : 0u, policy);
                    }
                    pf_arrive_landed(bar(G::kQFull));
                }
                if constexpr (!kSingle) {
                    Rows next = lookup(w.j0);
#pragma unroll 1
                    for (int j = w.j0; j < w.j1 && ok; ++j) {
                        const Rows f = next;
                        if (j + 1 < w.j1) next = lookup(j + 1);
                        load(p.k, f);
                        if (ok) load(p.v, f);
                    }
                } else {
                    Rows f[2] = {lookup(2 * w.j0), lookup(2 * w.j0 + 1)};
                    load(p.k, f[0]);
                    if (ok) load(p.k, f[1]);
#pragma unroll 1
                    for (int j = w.j0; j < w.j1 && ok; ++j)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const Rows now = f[t];
                            if (j + 1 < w.j1) f[t] = lookup(2 * j + 2 + t);
                            if (ok) load(p.v, now);
                            if (ok && j + 1 < w.j1) load(p.k, f[t]);
                        }
                }
            }
            cp_async_commit();
            cp_async_wait<0>();                                    // (a block that gives up leaves no copy behind)
        } else if (warp == 9 && lane == 0) {
            // ------------------------------------------------------------------ products
            constexpr uint32_t idesc_s = pf_idesc(kPfTile, false), idesc_o = pf_idesc(D, true);
            // Q, K: rows of 128 bytes, 8-row swizzle atoms 1024 bytes apart, 16 elements 32 bytes on, the second 64
            // columns 16 KB on.  V: d contiguous, 64 columns 16 KB apart, 16 keys 2 KB on.
            const uint64_t dq = pf_desc(sbase, 16, 1024), dk = pf_desc(sbase + G::kRing, 16, 1024),
                           dv = pf_desc(sbase + G::kRing, kPfBox, 1024);
            auto issue_s = [&](int t, uint32_t slot) {
                const uint64_t a0 = dq + (uint64_t)(((kSingle ? 0 : t) * G::kTileBytes) >> 4);
                const uint64_t b0 = dk + (uint64_t)((slot * G::kTileBytes) >> 4);
                const uint32_t d = tmem + 128u * t;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = (uint64_t)(((kk >> 2) * kPfBox + (kk & 3) * 32) >> 4);
                    ptx::mma_ss(d, a0 + off, b0 + off, idesc_s, kk > 0 ? 1u : 0u);
                }
            };
            auto issue_o = [&](int t, uint32_t slot, bool first) {
                const uint64_t b0 = dv + (uint64_t)((slot * G::kTileBytes) >> 4);
                const uint32_t d = tmem + 256u + (uint32_t)(D * t), a = tmem + 128u * t, acc0 = first ? 0u : 1u;
#pragma unroll
                for (int kk = 0; kk < 2 * (kPfTile / 16); ++kk) {  // upper parts, then lower ones: of 32 keys 16 columns each, side by side
                    const int k = kk & 7;
                    ptx::mma_ts(d, a + (uint32_t)((k >> 1) * 32 + (kk >> 3) * 16 + (k & 1) * 8), b0 + (uint64_t)((k * 2048) >> 4), idesc_o,
                                kk > 0 ? 1u : acc0);
                }
            };
            uint32_t pos = 0, count = 0;                           // loads, and steps, before this share
            bool ok = true;
            // the slot of load `at`, once it has landed
            auto landed = [&](uint32_t at) {
                ok = ok && pf_wait(bar(G::kFull + at % G::kStages), (at / G::kStages) & 1u, abort_flag, lim);
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_after();
                return at % G::kStages;
            };
            auto release = [&](uint32_t at) { ptx::mma_commit(bar(G::kEmpty + at % G::kStages)); };
#pragma unroll 1
            for (uint32_t n = 0; ok && walk.next(p, w); ++n) {
                const int steps = w.j1 - w.j0;
                ok = pf_wait(bar(G::kQFull), n & 1u, abort_flag, lim);     // (its proxy fence: the next slot's)
                {
                    const uint32_t s0 = landed(pos);
                    if (!ok) break;
                    issue_s(0, s0);
                    ptx::mma_commit(bar(G::kSFull));
                    if (kSingle) release(pos++);
                    const uint32_t s1 = kSingle ? landed(pos) : s0;
                    if (!ok) break;
                    issue_s(1, s1);
                    ptx::mma_commit(bar(G::kSFull + 1));
                    release(pos++);
                    if (steps == 1) ptx::mma_commit(bar(G::kQEmpty));
                }
#pragma unroll 1
                for (int jj = 0; jj < steps && ok; ++jj) {
                    const bool more = jj + 1 < steps;
                    // loads of this step: value tile(s), key tile(s) of the next step
                    const uint32_t v0 = pos, k0 = pos + 1, v1 = kSingle ? pos + (more ? 2 : 1) : pos, k1 = kSingle ? pos + 3 : pos + 1;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t vt = t ? v1 : v0, kt = t ? k1 : k0;
                        const uint32_t vs = kSingle || t == 0 ? landed(vt) : vt % G::kStages;
                        ok = ok && pf_wait(bar(G::kPFull + t), (count + jj) & 1u, abort_flag, lim);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        issue_o(t, vs, jj == 0);
                        if (!more && !(p.test_hooks && n == 0 && t == 0 && blockIdx.x == 0)) ptx::mma_commit(bar(G::kOFull + t));
                        if (kSingle || t == 1) release(vt);
                        if (more) {
                            const uint32_t ks = kSingle || t == 0 ? landed(kt) : kt % G::kStages;
                            if (!ok) break;
                            issue_s(t, ks);
                            ptx::mma_commit(bar(G::kSFull + t));
                            if (kSingle || t == 1) release(kt);
                            if (t == 1 && jj + 2 == steps) ptx::mma_commit(bar(G::kQEmpty));
                        }
                    }
                    pos += (kSingle ? 2 : 1) * (more ? 2 : 1);
                }
                count += steps;
            }
            // every product has finished before TMEM goes back
            ptx::mma_commit(bar(G::kDrain));
            const uint64_t start = ptx::globaltimer_ns();
            while (!ptx::mbar_try_wait(bar(G::kDrain), 0) && ptx::globaltimer_ns() - start < lim) {
            }
        }
    } else {
        ptx::reg_alloc<G::kRegsSoftmax>();
        // ---------------------------------------------------------------------- softmax
        const int t = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off + 128u * t, tO = tmem + lane_off + 256u + (uint32_t)(D * t);
        const float c = p.scale_log2, tau = 8.0f;                  // a reference may lag by 2^8
        // A tile's logits are read from TMEM twice, a piece at a time in short loops: for their maximum, then for the weights, which
        // go where they were.  (Unrolled over all 128 the step was longer than the schedulers' instruction caches and waited for its
        // code: 24 sequences of 32 heads, 65,500 keys: 64 us, unrolled 79; 512 of 40, 4,133: 111 and 113.)
        constexpr int kLook = kSingle ? 32 : 64;                   // columns of a piece for the maximum
        uint32_t count = 0;                                        // steps before this share
        bool ok = true;
#pragma unroll 1
        for (uint32_t n = 0; walk.next(p, w); ++n) {               // (once a wait has given up: only to mark the parts that are owed)
        const int at = w.rb * (kSingle ? kPfTile : 2 * kPfTile) + (kSingle ? row : t * kPfTile + row);
        // warps without a row keep every wait and arrival, and skip the rest: a row is its own lane of TMEM
        const bool live = at - lane < p.rows;
        float m = -INFINITY, l = 0.0f;
        if (ok && !live) {
#pragma unroll 1
            for (int j = w.j0; j < w.j1; ++j, ++count) {
                ok = pf_wait(bar(G::kSFull + t), count & 1u, abort_flag, lim);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                ptx::tc_fence_after();
                ptx::tc_fence_before();
                ptx::mbar_arrive(bar(G::kPFull + t));
            }
        } else if (ok) {
#pragma unroll 1
            for (int j = w.j0; j < w.j1; ++j, ++count) {
                ok = pf_wait(bar(G::kSFull + t), count & 1u, abort_flag, lim);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                ptx::tc_fence_after();
                const int valid = p.prefix_len - tile_of(j, t) * kPfTile;      // keys of the tile (the same for every row)
                float mxa[4], mna[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mxa[i] = -INFINITY;
                    mna[i] = INFINITY;
                }
#pragma unroll 1
                for (int ch = 0; ch < kPfTile / kLook; ++ch) {
                    uint32_t s[kLook];
                    if constexpr (kLook == 32) ptx::tmem_ld32(tS + kLook * ch, s);
                    else ptx::tmem_ld64(tS + kLook * ch, s);
                    if (valid < kPfTile) {
#pragma unroll
                        for (int e = 0; e < kLook; ++e)
                            if (kLook * ch + e >= valid) s[e] = __float_as_uint(-INFINITY);
                    }
#pragma unroll
                    for (int e = 0; e < kLook; e += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float a = __uint_as_float(s[e + i]), b = __uint_as_float(s[e + 4 + i]);
                            mxa[i] = ptx::fmax3(mxa[i], a, b);
                            mna[i] = ptx::fmin3(mna[i], a, b);
                        }
                }
                const float mx = ptx::fmax3(mxa[0], mxa[1], fmaxf(mxa[2], mxa[3]));
                const float mn = ptx::fmin3(mna[0], mna[1], fminf(mna[2], mna[3]));
                bool rescale_o = false;
                float alpha = 1.0f;
                if (mx > m && (mx - m) * c > tau) {
                    alpha = rescale(m, mx, c);
                    rescale_o = m != -INFINITY && j > w.j0;
                    l *= alpha;
                    m = mx;
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                // Plain: no logit of -inf, which weighs 0, none so low that its weight would need the lower bound of 2^-100 (a finite logit
                // weighs something, and both parts of its weight are normal numbers), and a reference of 2^10 at most: then
                // (s - ref) c is one fma with ref * c rounded, which takes every weight by the same 2^-15 of an exponent or less.
                const bool plain = __all_sync(0xFFFFFFFFu, mn > -INFINITY && (mn - ref) * c >= -100.0f && fabsf(ref) * c <= 1024.0f);
                const float least = ref - 100.0f / c, minus = plain ? -ref * c : 0.0f;
                const float2 c2 = make_float2(c, c), minus2 = make_float2(minus, minus);
                float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int ch = 0; ch < kPfTile / 32; ++ch) {
                    uint32_t s[32], hi[16], lo[16];
                    ptx::tmem_ld32(tS + 32 * ch, s);
                    if (!plain) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = 32 * ch + e < valid ? __uint_as_float(s[e]) : -INFINITY;
                            s[e] = __float_as_uint(x == -INFINITY ? x : ptx::fmax_nan(x, least) - ref);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, minus2);
                        const float2 y = make_float2(ptx::ex2_approx(x.x), ptx::ex2_approx(x.y));
                        sum[e & 3] = __fadd2_rn(sum[e & 3], y);
                        pf_parts(y, hi[e], lo[e]);
                    }
                    ptx::tmem_st16(tS + 32 * ch, hi);
                    ptx::tmem_st16(tS + 32 * ch + 16, lo);
                }
                const float2 ls = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
                l += ls.x + ls.y;
                if (__any_sync(0xFFFFFFFFu, rescale_o)) {
                    const float a = rescale_o ? alpha : 1.0f;
                    const float2 a2 = make_float2(a, a);
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t o[32];
                        ptx::tmem_ld32(tO + ch * 32, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), a2);
                            o[2 * e] = __float_as_uint(y.x);
                            o[2 * e + 1] = __float_as_uint(y.y);
                        }
                        ptx::tmem_st32(tO + ch * 32, o);
                    }
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                ptx::mbar_arrive(bar(G::kPFull + t));
            }
        }
        ok = ok && pf_wait(bar(G::kOFull + t), n & 1u, abort_flag, lim);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!live) continue;
        // the warp's 32 rows, 32 columns at a time, through its room: each store then takes four whole 128-byte lines
        // (a thread's own row in 16-byte pieces took 4 us more)
        const long long part0 = (((long long)blockIdx.x * p.slots + n) * 2 + t) * kPfTile + quarter * 32;
        const uint32_t room = sbase + (uint32_t)(G::kRoom + warp * 4096);
        const int rows = min(32, p.rows - (at - lane));
        if (!ok) {                     // a part that is not there: the join leaves its rows unwritten
            if (lane < rows) p.part_ml[part0 + lane] = make_float2(-INFINITY, kBadPart);
            continue;
        }
        ptx::tc_fence_after();
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t o[32];
            ptx::tmem_ld32(tO + ch * 32, o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ptx::st_shared_v4(room + lane * 128 + ((i ^ (lane & 7)) << 4), o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3), x = lane & 7;
                const float4 y = *reinterpret_cast<const float4*>(smem + G::kRoom + warp * 4096 + r * 128 + ((x ^ (r & 7)) << 4));
                if (r < rows) *reinterpret_cast<float4*>(p.part_o + (part0 + r) * D + ch * 32 + x * 4) = y;
            }
            __syncwarp();
        }
        if (lane < rows) p.part_ml[part0 + lane] = make_float2(m, *bad_flag ? kBadPart : l);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kPfTmemCols);
    }
}

struct PrefixJoin {
    PrefixParams x;                // of the prefix's kernel
    DecodeParams s;                // of the kernel of the own keys
    int single, warps;             // one tile of rows a unit; warps a row
};

// The join: a row's parts of the prefix and of its own keys.  `warps` warps take two rows (16 lanes each), each a share of the
// prefix's parts and of the own keys', and are joined through shared memory.  The prefix's parts lie where arithmetic says, so
// they are on their way while the row's length and span are read.
constexpr int kPfJoinWarps = 8;
// kU: parts in flight; 4 where a row has no more, for more rows on an SM.  20,480 rows of 1 or 2 parts of the prefix: 15 us, with 8
// in flight 19; 2,048 rows of 20: 7.
template <int D, int kU>
__global__ void __launch_bounds__(32 * kPfJoinWarps, kU > 4 ? 2 : 3) attn_prefix_join_kernel(const __grid_constant__ PrefixJoin p) {
    constexpr int kQ = D / 64, kC = 4 * kQ;            // a lane's elements: 4 of each 64
    struct V { float4 q[kQ]; };
    __shared__ V o_s[kPfJoinWarps][32];
    __shared__ float2 ml_s[kPfJoinWarps][2];
    __shared__ int bad_s[kPfJoinWarps][2];
    pdl_wait();
    pdl_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, W = p.warps, share = warp & (W - 1);
    // (W is a power of two; heads in y)
    const int b = blockIdx.x, half = lane >> 4, at = lane & 15, h = (blockIdx.y * (kPfJoinWarps / W) + warp / W) * 2 + half;
    const bool there = h < p.s.H;
    const long long out = (long long)b * p.s.H + h;
    const int kv = there ? p.x.by_group.of(h) : 0, g = there ? h - kv * p.s.group : 0, r = b * p.s.group + g;
    const int heads = p.s.block_heads, blk = g / heads, hh = g - blk * heads;      // (8, 16 or 32 heads)
    const int len = __ldg(p.s.seqlens_k + b);
    const int2 span = p.s.span[((long long)b * p.s.Hkv + kv) * p.s.head_blocks + blk];     // (of a row with own keys)
    // the prefix's parts: of each CTA that has steps of the row's unit, its first share but in the first of them
    const int in_shift = p.single ? 7 : 8, rb = r >> in_shift, in = r - (rb << in_shift), places = p.x.steps + kPfEnd;
    const int place0 = (kv * p.x.row_blocks + rb) * places, first = p.x.cta_of(place0);
    const int parts = (p.x.cta_of(place0 + p.x.steps - 1) - first + 1) << p.single;
    const int before = p.x.by_places.of(p.x.start(first));     // the unit in which that CTA's range begins
    const int skip = kv * p.x.row_blocks + rb - before - (p.x.start(first) - before * places >= p.x.steps);
    const long long first_part = (((long long)first * p.x.slots + skip) * 2) * kPfTile + (p.single ? in : (in >> 7) * kPfTile + (in & 127));
    const long long rest_part = first_part - (long long)skip * (2 * kPfTile);      // (as if every CTA had it as its first)
    const int step_part = p.x.slots * (2 * kPfTile);
    auto prefix_part = [&](int i) {
        const int c = i >> p.single;
        return (c == 0 ? first_part : rest_part + (long long)c * step_part) + (p.single ? (i & 1) * kPfTile : 0);
    };
    float mx = -INFINITY, sum = 0.0f, acc[kC];
    bool bad = false;
#pragma unroll
    for (int x = 0; x < kC; ++x) acc[x] = 0.0f;
    // (every lane has a part's m and l, and its own elements: nothing to hand over)
    auto row_of = [&](const float* row) {
        V v;
#pragma unroll
        for (int q = 0; q < kQ; ++q) v.q[q] = reinterpret_cast<const float4*>(row)[q * 16 + at];
        return v;
    };
    auto add = [&](const V& v, float down, float f) {
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            acc[4 * q] = acc[4 * q] * down + v.q[q].x * f;
            acc[4 * q + 1] = acc[4 * q + 1] * down + v.q[q].y * f;
            acc[4 * q + 2] = acc[4 * q + 2] * down + v.q[q].z * f;
            acc[4 * q + 3] = acc[4 * q + 3] * down + v.q[q].w * f;
        }
    };
    auto merge = [&](float2 ml, const V& v) {
        bad |= ml.y == kBadPart;
        const float top = fmaxf(mx, ml.x), down = rescale(mx, top, p.s.scale_log2), f = rescale(ml.x, top, p.s.scale_log2);
        mx = top;
        sum = sum * down + ml.y * f;
        add(v, down, f);
    };
    const int i0 = parts * share / W, i1 = parts * (share + 1) / W;
    V v[kU], own_v;
    float2 ml[kU], own_m;
    auto fetch = [&](int i) {
#pragma unroll
        for (int j = 0; j < kU; ++j)
            if (i + j < i1) {
                const long long part = prefix_part(i + j);
                ml[j] = p.x.part_ml[part];
                v[j] = row_of(p.x.part_o + part * D);
            }
    };
    fetch(i0);
    const bool good = there && len >= p.x.prefix_len && (long long)len <= (long long)p.s.pages.max_pages * p.s.pages.page_size;
    if (there && !good && len != 0 && h == 0 && share == 0 && at == 0) report_invalid(ATTN_CACHE_SITE_DECODE);
    // the own keys' parts: one of a whole row, or one of each warp of the span (its first in slot 1 of its warp, the others in 0)
    const bool whole = span.x < 0;
    const int own = good && len > p.x.prefix_len ? (whole ? 1 : span.y - span.x + 1) : 0;
    auto own_fetch = [&](int i) {
        const long long part = (2ll * (span.x + i) + (i == 0)) * heads + hh;
        own_m = whole ? p.s.own_ml[out] : p.s.part_ml[part];
        own_v = row_of(whole ? p.s.own_o + out * D : p.s.part_o + part * D);
    };
    if (share < own) own_fetch(share);
#pragma unroll 1
    for (int i = i0; i < i1; i += kU) {
        if (i > i0) fetch(i);
#pragma unroll
        for (int j = 0; j < kU; ++j)
            if (i + j < i1) merge(ml[j], v[j]);
    }
#pragma unroll 1
    for (int i = share; i < own; i += W) {
        if (i > share) own_fetch(i);
        merge(own_m, own_v);
    }
    if (W > 1) {
        if (at == 0) {
            ml_s[warp][half] = make_float2(mx, sum);
            bad_s[warp][half] = bad;
        }
        V mine;
#pragma unroll
        for (int q = 0; q < kQ; ++q) mine.q[q] = make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
        o_s[warp][lane] = mine;
        __syncthreads();
        if (share != 0) return;
        float top = mx;
        for (int w = 1; w < W; ++w) top = fmaxf(top, ml_s[warp + w][half].x);
        const float f0 = rescale(mx, top, p.s.scale_log2);
        sum *= f0;
#pragma unroll
        for (int x = 0; x < kC; ++x) acc[x] *= f0;
        for (int w = 1; w < W; ++w) {
            const float2 ml = ml_s[warp + w][half];
            const float f = rescale(ml.x, top, p.s.scale_log2);
            sum += ml.y * f;
            bad |= bad_s[warp + w][half] != 0;
            add(o_s[warp + w][lane], 1.0f, f);
        }
        mx = top;
    }
    const bool ended = there && len == 0;              // without keys: NaN and -inf
    if (!(good || ended) || bad) return;
    const float inv = good && sum > 0.0f ? 1.0f / sum : NAN;       // no weight at all, or a NaN one: the row is NaN
    auto pair = [&](float x, float y) { return round_bf16(x * inv, p.s.round_mode) | round_bf16(y * inv, p.s.round_mode) << 16; };
#pragma unroll
    for (int q = 0; q < kQ; ++q)
        reinterpret_cast<uint2*>(p.s.o + out * D)[q * 16 + at] = make_uint2(pair(acc[4 * q], acc[4 * q + 1]), pair(acc[4 * q + 2], acc[4 * q + 3]));
    if (p.s.lse && at == 0) p.s.lse[out] = ended || sum == 0.0f ? -INFINITY : mx * p.s.scale + logf(sum);
}

}  // namespace cache
