// prefix.cuh -- attention of one new token per sequence over keys that the whole batch shares: the shared part, and
// the join with each sequence's own keys (decode.cuh).
//
// Mathematics.  The prefix's keys are the same for all sequences, so the queries of a K/V head's group in all sequences,
// B * G rows (G = H / Hkv), form one matrix against them:
//   S = Q K^T,  m_i = max_j S_ij,  P_ij = exp((S_ij - m_i) / sqrt(d)),  l_i = sum_j P_ij,  O_i = sum_j P_ij v_j,
// with a running m and l over tiles of 128 keys.  The keys are dealt to CTAs in contiguous ranges; a row's parts
// (m, l, O in fp32) of all ranges and of its own keys are joined as in decode.cuh.
//
// Bound.  Every key of the prefix is read once for the batch (2 * d * 2 bytes) and costs 4 * d * B * G flops: with some
// 285 rows and more the tensor pipe bounds it, with fewer HBM.  So the products run on tcgen05, with queries as the 128
// rows of a tile, S and O in TMEM, P written over S.  Two tiles of P are in work at a time, one softmax warpgroup each,
// so that the products of one run beside the exponentials of the other:
//   more than 128 rows: two tiles of rows against one tile of keys;
//   128 rows and fewer (kSingle): one tile of rows against two tiles of keys, even and odd ones, which keep
//   an m, l and O each.
// P is rounded to bf16 for the second product (tcgen05 takes it in that type from TMEM; a second product
// with its lower bits, as in decode.cuh, would double the work that bounds the kernel), l sums the unrounded weights.
//
// Loads.  Two warps copy keys and values with cp.async, row by row, into the 128-byte-swizzled tiles that the
// tensor pipe reads: any page size, any number of heads, no tensor maps to make on the host.  Each load is signalled kLag
// loads later, when it has landed (cp.async.wait_group, a proxy fence, an mbarrier), so kLag + 1 are in flight.
#pragma once
#include "cache_common.cuh"
#include "decode.cuh"

namespace cache {

struct PrefixParams {
    const __nv_bfloat16* q;        // [B][H][d]
    const char* k;                 // [rows][Hkv][d]
    const char* v;
    Pages pages;                   // table: the first sequence's row
    int H, Hkv, group, rows;       // rows = B * group
    int prefix_len, tiles;         // keys, and tiles of 128 of them
    int row_blocks, splits;        // blocks of 256 rows (kSingle: 128), ranges of tiles
    float scale_log2;              // log2(e) / sqrt(d)
    float* part_o;                 // [CTAs][2][128][d]
    float2* part_ml;               // [CTAs][2][128]: (m in logits, l); l = -1: a bad page
    unsigned long long wait_limit_ns;
};

constexpr int kPfThreads = 384;    // warpgroups 0, 1: softmax; warps 8 and 10 load, warp 9 issues the products
constexpr int kPfTile = 128;
constexpr int kPfBox = kPfTile * 64 * 2;       // 64 columns of a tile: rows of 128 bytes
constexpr uint32_t kPfRegsSoftmax = 200, kPfRegsOther = 104;       // 256 * 200 + 128 * 104 = 384 * 168
constexpr uint32_t kPfTmemCols = 512;          // S0 | S1 | O0 | O1

template <int D, bool kSingle>
struct PfGeo {
    static constexpr int kTileBytes = kPfTile * D * 2;
    static constexpr int kQTiles = kSingle ? 1 : 2;
    static constexpr int kStages = 7 * 128 / D - kQTiles;          // all the shared memory that Q leaves
    static constexpr int kLag = D == 128 ? 2 : 5;                  // 96 KB in flight
    static constexpr int kRing = kQTiles * kTileBytes;
    static constexpr int kBars = kRing + kStages * kTileBytes;
    // barriers
    static constexpr int kFull = 0, kEmpty = kStages, kQFull = 2 * kStages, kSFull = kQFull + 1, kPFull = kSFull + 2,
                         kOFull = kPFull + 2, kDrain = kOFull + 2, kNumBars = kDrain + 1;
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
// where chunk c (16 bytes) of row r is in a tile
__device__ __forceinline__ uint32_t pf_chunk(int r, int c) {
    return (uint32_t)((c >> 3) * kPfBox + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The range of a CTA, and its row block: CTAs that read the same keys are neighbours.
struct PfWork {
    int rb, kv, t0, t1;
};
__device__ __forceinline__ PfWork pf_work(const PrefixParams& p, int cta) {
    PfWork w;
    w.rb = cta % p.row_blocks;
    const int rest = cta / p.row_blocks;
    w.kv = rest % p.Hkv;
    const int s = rest / p.Hkv, base = p.tiles / p.splits, more = p.tiles - base * p.splits;
    w.t0 = s * base + min(s, more);
    w.t1 = w.t0 + base + (s < more);
    return w;
}

template <int D, bool kSingle>
__global__ void __launch_bounds__(kPfThreads, 1) attn_prefix_kernel(const __grid_constant__ PrefixParams p) {
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
            ptx::mbar_init(bar(G::kFull + s), 64);
            ptx::mbar_init(bar(G::kEmpty + s), 1);
        }
        ptx::mbar_init(bar(G::kQFull), 256);
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

    const PfWork w = pf_work(p, blockIdx.x);
    const int steps = kSingle ? (w.t1 - w.t0 + 1) / 2 : w.t1 - w.t0;
    const int key_end = min(p.prefix_len, w.t1 * kPfTile);         // behind the range's last key
    // tile of step jj that warpgroup t's rows meet
    auto tile_of = [&](int jj, int t) { return kSingle ? w.t0 + 2 * jj + t : w.t0 + jj; };

    if (warp >= 8) {
        ptx::reg_dealloc<kPfRegsOther>();
        if (warp == 8 || warp == 10) {
            // ------------------------------------------------------------------ loads
            // In the order in which the products take them: K0 V0 K1 V1 ..., or with two key tiles a step (a, b)
            // Ka0 Kb0, then Va0 Ka1 Vb0 Kb1, ..., and at the end Va Vb.
            const int half = warp == 8 ? 0 : 64, total = (kSingle ? 4 : 2) * steps;
            constexpr int kChunks = D / 8, kRowsPerCopy = 32 / kChunks;
            const long long key_stride = (long long)p.Hkv * D * 2;
            const uint64_t policy = p.row_blocks > 1 ? ptx::policy_evict_last() : ptx::policy_evict_first();
            struct Found { int tile_v, row[2]; };                  // value tile? ; rows of keys half + lane and + 32 (-1: none)
            auto find = [&](int pos) {
                int jj, t = 0, v;
                if (!kSingle) {
                    jj = pos >> 1;
                    v = pos & 1;
                } else if (pos < 2) {
                    jj = 0; t = pos; v = 0;
                } else {
                    const int g = (pos - 2) >> 2, r = (pos - 2) & 3;
                    if (g < steps - 1) {
                        t = r >> 1;
                        v = !(r & 1);
                        jj = v ? g : g + 1;
                    } else {
                        t = r; v = 1; jj = g;
                    }
                }
                Found f;
                f.tile_v = v;
                const int j0 = tile_of(jj, t) * kPfTile + half + lane;
                bool bad = false;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int j = j0 + 32 * u;
                    f.row[u] = j < key_end ? page_row(p.pages, p.pages.table, j) : -1;
                    bad |= j < key_end && f.row[u] < 0;
                }
                if (bad) {
                    *bad_flag = 1u;
                    report_invalid(ATTN_CACHE_SITE_PREFIX);
                }
                return f;
            };
            Found next = find(0);
            bool ok = true;
            int pos = 0;
#pragma unroll 1
            for (; pos < total; ++pos) {
                const Found f = next;
                if (pos + 1 < total) next = find(pos + 1);
                const int slot = pos % G::kStages;
                if (pos >= G::kStages) {
                    ok = pf_wait(bar(G::kEmpty + slot), (uint32_t)(pos / G::kStages - 1) & 1u, abort_flag, lim);
                    if (!__all_sync(0xFFFFFFFFu, ok)) break;
                }
                const char* src = (f.tile_v ? p.v : p.k) + (long long)w.kv * D * 2 + (lane % kChunks) * 16;
                const uint32_t dst = sbase + (uint32_t)(G::kRing + slot * G::kTileBytes);
#pragma unroll
                for (int i = 0; i < 64 / kRowsPerCopy; ++i) {
                    const int r = i * kRowsPerCopy + lane / kChunks;           // of this warp's 64
                    const int row = __shfl_sync(0xFFFFFFFFu, i * kRowsPerCopy < 32 ? f.row[0] : f.row[1], r & 31);
                    cp_async16(dst + pf_chunk(half + r, lane % kChunks), src + (long long)max(row, 0) * key_stride,
                               row < 0 ? 0u : 16u, policy);
                }
                cp_async_commit();
                if (pos >= G::kLag) {
                    cp_async_wait<G::kLag>();
                    ptx::fence_proxy_async_smem();
                    ptx::mbar_arrive(bar(G::kFull + (pos - G::kLag) % G::kStages));
                }
            }
            cp_async_wait<0>();
            ptx::fence_proxy_async_smem();
            if (pos == total)
                for (int q = max(total - G::kLag, 0); q < total; ++q) ptx::mbar_arrive(bar(G::kFull + q % G::kStages));
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
                for (int kk = 0; kk < kPfTile / 16; ++kk)
                    ptx::mma_ts(d, a + (uint32_t)kk * 8u, b0 + (uint64_t)((kk * 2048) >> 4), idesc_o, kk > 0 ? 1u : acc0);
            };
            uint32_t pos = 0;
            bool ok = pf_wait(bar(G::kQFull), 0, abort_flag, lim);
            // the slot of the next load in order, once it has landed
            auto landed = [&](uint32_t at) {
                ok = ok && pf_wait(bar(G::kFull + at % G::kStages), (at / G::kStages) & 1u, abort_flag, lim);
                ptx::tc_fence_after();
                return at % G::kStages;
            };
            auto release = [&](uint32_t at) { ptx::mma_commit(bar(G::kEmpty + at % G::kStages)); };
            {
                const uint32_t s0 = landed(0);
                if (ok) {
                    issue_s(0, s0);
                    ptx::mma_commit(bar(G::kSFull));
                    if (kSingle) release(0);
                }
                const uint32_t s1 = kSingle ? landed(1) : s0;
                if (ok) {
                    issue_s(1, s1);
                    ptx::mma_commit(bar(G::kSFull + 1));
                    release(kSingle ? 1 : 0);
                }
                pos = kSingle ? 2 : 1;
            }
#pragma unroll 1
            for (int jj = 0; jj < steps && ok; ++jj) {
                const bool more = jj + 1 < steps;
                // loads of this step: value tile(s) vt, key tile(s) of the next step kt
                const uint32_t v0 = pos, k0 = pos + 1, v1 = kSingle ? pos + (more ? 2 : 1) : pos, k1 = kSingle ? pos + 3 : pos + 1;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t vt = t ? v1 : v0, kt = t ? k1 : k0;
                    const uint32_t vs = landed(vt);
                    ok = ok && pf_wait(bar(G::kPFull + t), (uint32_t)jj & 1u, abort_flag, lim);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    issue_o(t, vs, jj == 0);
                    if (!more) ptx::mma_commit(bar(G::kOFull + t));
                    if (kSingle || t == 1) release(vt);
                    if (more) {
                        const uint32_t ks = landed(kt);
                        if (!ok) break;
                        issue_s(t, ks);
                        ptx::mma_commit(bar(G::kSFull + t));
                        if (kSingle || t == 1) release(kt);
                    }
                }
                pos += (kSingle ? 2 : 1) * (more ? 2 : 1);
            }
            // every product has finished before TMEM goes back
            ptx::mma_commit(bar(G::kDrain));
            const uint64_t start = ptx::globaltimer_ns();
            while (!ptx::mbar_try_wait(bar(G::kDrain), 0) && ptx::globaltimer_ns() - start < lim) {
            }
        }
    } else {
        ptx::reg_alloc<kPfRegsSoftmax>();
        // ---------------------------------------------------------------------- queries, softmax
        const int t = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const int block0 = w.rb * (kSingle ? kPfTile : 2 * kPfTile);           // first row of the CTA
        {
            constexpr int kChunks = D / 8, kRowsQ = kSingle ? kPfTile : 2 * kPfTile;
#pragma unroll 4
            for (int i = threadIdx.x; i < kRowsQ * kChunks; i += 256) {
                const int r = i / kChunks, c = i % kChunks, at = block0 + r;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (at < p.rows) {
                    const int b = at / p.group, g = at - b * p.group;
                    x = *reinterpret_cast<const uint4*>(p.q + ((long long)b * p.H + w.kv * p.group + g) * D + c * 8);
                }
                ptx::st_shared_v4(sbase + (uint32_t)((r / kPfTile) * G::kTileBytes) + pf_chunk(r % kPfTile, c), x.x, x.y, x.z, x.w);
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(bar(G::kQFull));
        }
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off + 128u * t, tO = tmem + lane_off + 256u + (uint32_t)(D * t);
        const float c = p.scale_log2, tau = 8.0f;                  // a reference may lag by 2^8
        const int at = block0 + (kSingle ? row : t * kPfTile + row);
        // warps without a row keep every wait and arrival, and skip the rest: a row is its own lane of TMEM
        const bool live = at - lane < p.rows;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        if (!live) {
#pragma unroll 1
            for (int jj = 0; jj < steps; ++jj) {
                ok = pf_wait(bar(G::kSFull + t), (uint32_t)jj & 1u, abort_flag, lim);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                ptx::tc_fence_after();
                ptx::tc_fence_before();
                ptx::mbar_arrive(bar(G::kPFull + t));
            }
        } else {
#pragma unroll 1
            for (int jj = 0; jj < steps; ++jj) {
                ok = pf_wait(bar(G::kSFull + t), (uint32_t)jj & 1u, abort_flag, lim);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                ptx::tc_fence_after();
                uint32_t s[128];
                ptx::tmem_ld128(tS, s);
                const int valid = key_end - tile_of(jj, t) * kPfTile;          // keys of the tile (the same for every row)
                if (valid < kPfTile) {
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (e >= valid) s[e] = __float_as_uint(-INFINITY);
                }
                float mxa[4], mna[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mxa[i] = mna[i] = __uint_as_float(s[i]);
#pragma unroll
                for (int e = 4; e < 124; e += 8)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = __uint_as_float(s[e + i]), b = __uint_as_float(s[e + 4 + i]);
                        mxa[i] = ptx::fmax3(mxa[i], a, b);
                        mna[i] = ptx::fmin3(mna[i], a, b);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mxa[i] = fmaxf(mxa[i], __uint_as_float(s[124 + i]));
                    mna[i] = fminf(mna[i], __uint_as_float(s[124 + i]));
                }
                const float mx = ptx::fmax3(mxa[0], mxa[1], fmaxf(mxa[2], mxa[3]));
                const float mn = ptx::fmin3(mna[0], mna[1], fminf(mna[2], mna[3]));
                bool rescale_o = false;
                float alpha = 1.0f;
                if (mx > m && (mx - m) * c > tau) {
                    alpha = rescale(m, mx, c);
                    rescale_o = m != -INFINITY && jj > 0;
                    l *= alpha;
                    m = mx;
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                // no exponent so low that its weight would need weight_of's lower bound, none of -inf
                const bool plain = mn > -INFINITY && (mn - ref) * c >= -125.0f;
                const float2 c2 = make_float2(c, c), nm2 = make_float2(-ref, -ref);
                float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t pk[64];
                if (__all_sync(0xFFFFFFFFu, plain)) {
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        const float2 x = __fmul2_rn(
                            __fadd2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), nm2), c2);
                        const float2 y = make_float2(ptx::ex2_approx(x.x), ptx::ex2_approx(x.y));
                        sum[e & 3] = __fadd2_rn(sum[e & 3], y);
                        pk[e] = ptx::pack_bf16x2(y.x, y.y);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        const float y0 = weight_of(__uint_as_float(s[2 * e]), ref, c);
                        const float y1 = weight_of(__uint_as_float(s[2 * e + 1]), ref, c);
                        sum[e & 3] = __fadd2_rn(sum[e & 3], make_float2(y0, y1));
                        pk[e] = ptx::pack_bf16x2(y0, y1);
                    }
                }
                ptx::tmem_st32(tS, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
                ptx::tmem_st32(tS + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
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
        if (ok) ok = pf_wait(bar(G::kOFull + t), 0, abort_flag, lim);
        if (__all_sync(0xFFFFFFFFu, ok) && live) {
            ptx::tc_fence_after();
            uint32_t o[D];
            if constexpr (D == 128) ptx::tmem_ld128(tO, o);
            else ptx::tmem_ld64(tO, o);
            if (at < p.rows) {
                const long long part = ((long long)blockIdx.x * 2 + t) * kPfTile + row;
                float4* to = reinterpret_cast<float4*>(p.part_o + part * D);
#pragma unroll
                for (int i = 0; i < D / 4; ++i)
                    to[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                                        __uint_as_float(o[4 * i + 3]));
                p.part_ml[part] = make_float2(m, *bad_flag ? kBadPart : l);
            }
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
    int single, warps;             // one tile of rows a CTA; warps a row
};

// The join: a row's parts of the prefix and of its own keys.  `warps` warps take a row, a contiguous share of its parts
// each, and are joined through shared memory.
constexpr int kPfJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kPfJoinWarps) attn_prefix_join_kernel(const __grid_constant__ PrefixJoin p) {
    constexpr int kC = D / 32;
    __shared__ float o_s[kPfJoinWarps][D];
    __shared__ float2 ml_s[kPfJoinWarps];
    __shared__ int bad_s[kPfJoinWarps];
    pdl_wait();
    pdl_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, W = p.warps, share = warp % W;
    const long long out = (long long)blockIdx.x * (kPfJoinWarps / W) + warp / W;       // (b, h)
    const bool there = out < (long long)p.s.B * p.s.H;
    const int b = there ? (int)(out / p.s.H) : 0, h = there ? (int)(out - (long long)b * p.s.H) : 0;
    const int kv = h / p.s.group, g = h - kv * p.s.group, r = b * p.s.group + g;
    const int len = __ldg(p.s.seqlens_k + b);
    const bool good = there && len >= p.x.prefix_len && (long long)len <= (long long)p.s.pages.max_pages * p.s.pages.page_size;
    if (there && !good && h == 0 && share == 0 && lane == 0) report_invalid(ATTN_CACHE_SITE_DECODE);
    // parts: the prefix's, then those of the own keys
    const int block_rows = p.single ? kPfTile : 2 * kPfTile, rb = r / block_rows, in = r - rb * block_rows;
    const int shared_parts = p.x.splits * (p.single ? 2 : 1);
    int c0 = -1, own = 0;                              // first CTA (-1: the row is whole) and number of the own parts
    const int heads = p.s.block_heads, blk = g / heads, hh = g - blk * heads;
    if (good && len > p.x.prefix_len) {
        const int2 span = p.s.span[((long long)b * p.s.Hkv + kv) * p.s.head_blocks + blk];
        c0 = span.x;
        own = c0 < 0 ? 1 : span.y - c0 + 1;
    }
    const int parts = good ? shared_parts + own : 0;
    auto where = [&](int i, const float2*& ml, const float*& o) {
        if (i < shared_parts) {
            const int s = p.single ? i >> 1 : i, t = p.single ? i & 1 : in / kPfTile;
            const long long cta = ((long long)s * p.x.Hkv + kv) * p.x.row_blocks + rb;
            const long long part = (cta * 2 + t) * kPfTile + in % kPfTile;
            ml = p.x.part_ml + part;
            o = p.x.part_o + part * D;
        } else if (c0 < 0) {
            ml = p.s.own_ml + out;
            o = p.s.own_o + out * D;
        } else {
            const int c = c0 + i - shared_parts;       // a row's first part is in slot 1 of its CTA, the others in slot 0
            const long long part = (long long)(2 * c + (c == c0)) * heads + hh;
            ml = p.s.part_ml + part;
            o = p.s.part_o + part * D;
        }
    };
    const int i0 = parts * share / W, i1 = parts * (share + 1) / W;
    float mx = -INFINITY, sum = 0.0f, acc[kC];
    bool bad = false;
#pragma unroll
    for (int x = 0; x < kC; ++x) acc[x] = 0.0f;
    // 32 parts at a time: a lane has one's m and l, then the warp adds up their rows, eight in flight
#pragma unroll 1
    for (int base = i0; base < i1; base += 32) {
        const int n = min(32, i1 - base);
        const float2* mlp = nullptr;
        const float* op = nullptr;
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < n) {
            where(base + lane, mlp, op);
            ml = *mlp;
        }
        bad |= ml.y == kBadPart;
        float top = ml.x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
        top = fmaxf(top, mx);
        const float down = rescale(mx, top, p.s.scale_log2);
        mx = top;
        sum *= down;
#pragma unroll
        for (int x = 0; x < kC; ++x) acc[x] *= down;
        const float f = rescale(ml.x, top, p.s.scale_log2);
        float add = ml.y * f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) add += __shfl_xor_sync(0xFFFFFFFFu, add, off);
        sum += add;
        constexpr int kU = 8;
#pragma unroll 1
        for (int j0 = 0; j0 < n; j0 += kU) {
            float v[kU][kC];
#pragma unroll
            for (int j = 0; j < kU; ++j) {
                const float* from = reinterpret_cast<const float*>(
                    __shfl_sync(0xFFFFFFFFu, (unsigned long long)reinterpret_cast<uintptr_t>(op), (j0 + j) & 31));
#pragma unroll
                for (int x = 0; x < kC; ++x) v[j][x] = j0 + j < n ? from[x * 32 + lane] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kU; ++j) {
                const float fj = __shfl_sync(0xFFFFFFFFu, f, (j0 + j) & 31);
#pragma unroll
                for (int x = 0; x < kC; ++x)
                    if (j0 + j < n) acc[x] += v[j][x] * fj;
            }
        }
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (W > 1) {
        if (lane == 0) {
            ml_s[warp] = make_float2(mx, sum);
            bad_s[warp] = bad;
        }
#pragma unroll
        for (int x = 0; x < kC; ++x) o_s[warp][x * 32 + lane] = acc[x];
        __syncthreads();
        if (share != 0) return;
        float top = mx;
        for (int w = 1; w < W; ++w) top = fmaxf(top, ml_s[warp + w].x);
        const float f0 = rescale(mx, top, p.s.scale_log2);
        sum *= f0;
#pragma unroll
        for (int x = 0; x < kC; ++x) acc[x] *= f0;
        for (int w = 1; w < W; ++w) {
            const float f = rescale(ml_s[warp + w].x, top, p.s.scale_log2);
            sum += ml_s[warp + w].y * f;
            bad |= bad_s[warp + w] != 0;
#pragma unroll
            for (int x = 0; x < kC; ++x) acc[x] += o_s[warp + w][x * 32 + lane] * f;
        }
        mx = top;
    }
    if (!good || bad) return;
    const float inv = sum > 0.0f ? 1.0f / sum : NAN;   // no weight at all, or a NaN one: the row is NaN
#pragma unroll
    for (int x = 0; x < kC; ++x)
        p.s.o[out * D + x * 32 + lane] = __ushort_as_bfloat16((unsigned short)round_bf16(acc[x] * inv, p.s.round_mode));
    if (p.s.lse && lane == 0) p.s.lse[out] = sum == 0.0f ? -INFINITY : mx * p.s.scale + logf(sum);
}

}  // namespace cache
