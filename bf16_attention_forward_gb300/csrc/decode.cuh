// decode.cuh -- attention of one new token per sequence over a paged K/V cache.
//
// Mathematics.  For every sequence b and query head h over K/V head g = h / (H / Hkv):
//   s_j = q_h . k_j / sqrt(d),  m = max s_j,  l = sum exp(s_j - m),  o_h = sum exp(s_j - m) v_j / l,
// in one pass over the keys with a running m and l; parts of a sequence's keys are joined by
// m = max m_i, l = sum l_i exp(m_i - m), and the same for o.  With `weights` the softmax weight
// of each key, summed over the query heads of its K/V head, is added to a running fp32 weight.
//
// Bound: HBM bytes; every key and value is read once (2 * d * 2 bytes for 4 * d * G flops, G =
// H / Hkv query heads).  The products run on mma.sync with the KEYS as the M rows and the
// query heads as the N columns (S^T = K Q^T, O^T = V^T P^T): N is 8, so a K/V head's 4 to 8 query
// heads waste at most half of it.  tcgen05 would need 128 rows of one operand and a trip through
// TMEM for a product that takes a few percent of the time.
//
// Work.  A CTA of 8 warps per SM.  The tiles (128 keys) of all (sequence, K/V head) rows form
// one line, which the CTAs divide evenly: a CTA takes a contiguous range, so every CTA
// reads the same bytes whatever the lengths are, and a row is split only where a range
// ends inside it.  Each warp streams 16 keys of a tile through a ring of its own (cp.async, no
// barrier between warps) and keeps its own m, l and o; the warps are joined at the end of a row.
// A range holds at most one part that begins before it and one that ends behind it, so two part
// slots per CTA suffice; attn_decode_join_kernel merges a split row's parts.
#pragma once
#include "cache_common.cuh"

namespace cache {

struct DecodeParams {
    const __nv_bfloat16* q;        // [B][H][d]
    const char* k;                 // [rows][Hkv][d]
    const char* v;
    __nv_bfloat16* o;              // [B][H][d]
    float* lse;                    // [B][H] or null
    float* weights;                // [B][Hkv][max_pages * page_size] or null
    const int32_t* seqlens_k;
    Pages pages;
    int B, H, Hkv, group;          // group = H / Hkv
    int head_blocks;               // blocks of 8 * NH query heads that a K/V head's group takes
    int round_mode;
    int grid;                      // CTAs of the attention kernel (the join kernel derives the parts)
    float scale_log2;              // log2(e) / sqrt(d)
    float scale;
    // workspace
    float* part_o;                 // [2 * grid][heads of a block][d]
    float2* part_ml;               // [2 * grid][heads of a block]: (m in logits, l); l = -1: a bad page
    float2* row_ml;                // [B][Hkv][head_blocks][heads of a block] (weights only)
    float* scores;                 // [B][Hkv][max_pages * page_size][group] logits (weights only)
};

constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecKeys = 16;                       // keys of a warp's part of a tile
constexpr int kDecTile = kDecWarps * kDecKeys;     // 128
constexpr float kBadPart = -1.0f;

template <int D>
struct DecGeo {
    static constexpr int kRow = 2 * D;                            // bytes of a key
    static constexpr int kStageBytes = 2 * kDecKeys * kRow;       // K then V of 16 keys: 8 KB or 4 KB
    static constexpr int kStages = D == 128 ? 3 : 6;              // 24 KB of ring per warp
    static constexpr int kRing = kDecWarps * kStages * kStageBytes;
    static constexpr int kRed = kDecWarps * 8 * (D / 2) * 4;      // 8 heads, half of d, per warp
    static constexpr int kSmem = kRing + kRed;
};

// tiles of a sequence; 0 for a length that the table has no room for (the join kernel reports it)
__device__ __forceinline__ int seq_tiles(const DecodeParams& p, int b) {
    const int n = __ldg(p.seqlens_k + b);
    return n > 0 && (long long)n <= (long long)p.pages.max_pages * p.pages.page_size ? (n - 1) / kDecTile + 1 : 0;
}

// The line of tiles: sequence by sequence, row by row, tile by tile.
struct Line {
    long long units;               // tiles of all rows
    int ctas;                      // CTAs that get any: min(grid, units)
    __device__ __forceinline__ long long start(int c) const { return units * c / ctas; }
    __device__ __forceinline__ int cta_of(long long u) const { return (int)(((u + 1) * ctas - 1) / units); }
};

__device__ __forceinline__ Line make_line(const DecodeParams& p) {   // every lane of a warp calls it
    long long n = 0;
    for (int b = threadIdx.x & 31; b < p.B; b += 32) n += seq_tiles(p, b);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
    Line l;
    l.units = n * p.Hkv * p.head_blocks;
    l.ctas = (int)(l.units < p.grid ? l.units : p.grid);
    return l;
}

struct Cursor {
    int b, row, tile, tiles, len;  // row: K/V head * head_blocks + block of query heads
};

// the tile at place u of the line (u < units); *first: the place of its row's first tile
__device__ __forceinline__ Cursor seek(const DecodeParams& p, long long u, long long* first) {
    const int lane = threadIdx.x & 31;
    const int rows = p.Hkv * p.head_blocks;
    long long done = 0;
    Cursor c{0, 0, 0, 1, 0};
    for (int base = 0; base < p.B; base += 32) {
        const int mine = base + lane < p.B ? seq_tiles(p, base + lane) : 0;
        long long incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, off);
            if (lane >= off) incl += x;
        }
        const unsigned past = __ballot_sync(0xFFFFFFFFu, (done + incl) * rows > u);
        if (past) {
            const int w = __ffs(past) - 1;
            c.tiles = __shfl_sync(0xFFFFFFFFu, mine, w);
            const long long before = (done + __shfl_sync(0xFFFFFFFFu, incl, w) - c.tiles) * rows;
            c.b = base + w;
            c.row = (int)((u - before) / c.tiles);
            c.tile = (int)((u - before) - (long long)c.row * c.tiles);
            *first = u - c.tile;
            break;
        }
        done += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    c.len = __ldg(p.seqlens_k + c.b);
    return c;
}

// to the next tile of the line (there is one)
__device__ __forceinline__ void advance(const DecodeParams& p, Cursor& c) {
    if (++c.tile < c.tiles) return;
    c.tile = 0;
    if (++c.row < p.Hkv * p.head_blocks) return;
    c.row = 0;
    while (c.b + 1 < p.B) {
        ++c.b;
        c.tiles = seq_tiles(p, c.b);
        if (c.tiles > 0) break;
    }
    c.len = __ldg(p.seqlens_k + c.b);
}

// softmax weight of logit s against the reference m, in base 2: exactly 1 for the logit that set m, a
// positive normal number for every other finite one, 0 for -inf, NaN for NaN
__device__ __forceinline__ float weight_of(float s, float m, float c) {
    const float x = ptx::fmax_nan((s - m) * c, -125.0f);
    return s == -INFINITY ? 0.0f : ptx::ex2_approx(x);
}
// factor that takes sums against reference m to reference to (m <= to)
__device__ __forceinline__ float rescale(float m, float to, float c) {
    return m == -INFINITY ? 0.0f : ptx::ex2_approx(ptx::fmax_nan((m - to) * c, -125.0f));
}

template <int D, int NH, bool kWeights>
__global__ void __launch_bounds__(kDecThreads, 1) attn_decode_kernel(const __grid_constant__ DecodeParams p) {
    using G = DecGeo<D>;
    constexpr int kHeads = 8 * NH;
    constexpr int kChunks = G::kRow / 16;              // 16-byte chunks of a key
    constexpr int kRowsPerCopy = 32 / kChunks;         // keys that one cp.async of the warp takes
    extern __shared__ __align__(128) char smem[];
    __shared__ float2 ml_s[kDecWarps][kHeads];
    __shared__ int bad_s[kDecWarps][G::kStages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = ptx::smem_u32(smem) + warp * (G::kStages * G::kStageBytes);
    float* red = reinterpret_cast<float*>(smem + G::kRing);

    pdl_wait();
    pdl_launch();
    const Line line = make_line(p);
    if ((int)blockIdx.x >= line.ctas) return;
    const long long u0 = line.start(blockIdx.x), u1 = line.start(blockIdx.x + 1);
    long long row_first;
    Cursor cur = seek(p, u0, &row_first), ahead = cur;
    int to_load = (int)(u1 - u0);
    const long long key_stride = (long long)p.Hkv * G::kRow;

    // loads this warp's 16 keys of the tile at `ahead` into a stage (rows past the length, and rows
    // of a page that does not exist, become zeros) and moves on
    auto load = [&](int stage) {
        if (to_load > 0) {
            const int j0 = ahead.tile * kDecTile + warp * kDecKeys;
            int row = -1;
            bool bad = false;
            if (lane < kDecKeys && j0 + lane < ahead.len) {
                row = page_row(p.pages, p.pages.table + (long long)ahead.b * p.pages.max_pages, j0 + lane);
                bad = row < 0;
            }
            const bool any_bad = __any_sync(0xFFFFFFFFu, bad);
            if (lane == 0) {
                bad_s[warp][stage] = any_bad;
                if (any_bad) report_invalid(ATTN_CACHE_SITE_DECODE);
            }
            const int chunk = lane % kChunks;
            const long long col = (long long)(ahead.row / p.head_blocks) * G::kRow + chunk * 16;
            const uint32_t dst = ring + stage * G::kStageBytes;
#pragma unroll
            for (int i = 0; i < kDecKeys / kRowsPerCopy; ++i) {
                const int r = i * kRowsPerCopy + lane / kChunks;
                const int src_row = __shfl_sync(0xFFFFFFFFu, row, r);
                const long long off = (long long)max(src_row, 0) * key_stride + col;
                const uint32_t at = dst + r * G::kRow + ((chunk ^ (r & 7)) * 16);
                const uint32_t bytes = src_row < 0 ? 0u : 16u;
                cp_async16(at, p.k + off, bytes);
                cp_async16(at + kDecKeys * G::kRow, p.v + off, bytes);
            }
            --to_load;
            if (to_load > 0) advance(p, ahead);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < G::kStages - 1; ++s) load(s);

    // ldmatrix addresses inside a stage: lane i gives row i % 8 of 8x8 matrix i / 8
    const int mat = lane >> 3, mrow = lane & 7;
    const int krow = mrow + (mat & 1) * 8, kchunk = mat >> 1;          // K: rows 0-7, 8-15, then the next chunk
    const int vrow = mrow + (mat >> 1) * 8, vchunk = mat & 1;          // V (transposed): chunks, then rows 8-15
    const float tau = 8.0f / p.scale_log2;                             // a reference may lag by 2^8
    int stage = 0;

    for (long long u = u0; u < u1;) {
        const int kv_head = cur.row / p.head_blocks, head0 = (cur.row - kv_head * p.head_blocks) * kHeads;
        const long long row_end = row_first + cur.tiles;
        const int n = (int)((row_end < u1 ? row_end : u1) - u);        // tiles of this row in the range
        const int b = cur.b, len = cur.len;
        // Q as the B operand: head lane / 4, elements 2 * (lane % 4) and + 8 of each 16
        uint32_t qf[NH][D / 16][2];
#pragma unroll
        for (int t = 0; t < NH; ++t) {
            const int h = head0 + t * 8 + (lane >> 2);
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                p.q + ((long long)b * p.H + kv_head * p.group + h) * D + (lane & 3) * 2);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                qf[t][ks][0] = h < p.group ? src[ks * 8] : 0u;
                qf[t][ks][1] = h < p.group ? src[ks * 8 + 4] : 0u;
            }
        }
        float m[NH][2], l[NH][2], acc[NH][D / 16][4];
#pragma unroll
        for (int t = 0; t < NH; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][mt][e] = 0.0f;
        }
        bool bad = false;
        for (int i = 0; i < n; ++i) {
            cp_async_wait<G::kStages - 2>();
            __syncwarp();
            bad |= bad_s[warp][stage] != 0;
            const uint32_t ks_base = ring + stage * G::kStageBytes, vs_base = ks_base + kDecKeys * G::kRow;
            float s[NH][4];
#pragma unroll
            for (int t = 0; t < NH; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t a[4];
                ldmatrix_x4(ks_base + krow * G::kRow + (((ks * 2 + kchunk) ^ (krow & 7)) * 16), a);
#pragma unroll
                for (int t = 0; t < NH; ++t) mma_16816(s[t], a, qf[t][ks][0], qf[t][ks][1]);
            }
            // s[t][0..1]: key j0, heads 2 * (lane % 4) and + 1; s[t][2..3]: key j0 + 8
            const int j0 = (cur.tile + i) * kDecTile + warp * kDecKeys + (lane >> 2);
            bool grow = false;
#pragma unroll
            for (int t = 0; t < NH; ++t) {
                if (j0 >= len) s[t][0] = s[t][1] = -INFINITY;
                if (j0 + 8 >= len) s[t][2] = s[t][3] = -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) grow |= s[t][e] > m[t][e & 1] + tau;
            }
            if constexpr (kWeights) {
                float* to = p.scores +
                            ((long long)(b * p.Hkv + kv_head) * ((long long)p.pages.max_pages * p.pages.page_size) + j0) *
                                p.group + head0 + (lane & 3) * 2;
#pragma unroll
                for (int t = 0; t < NH; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j0 + (e >> 1) * 8 < len && head0 + t * 8 + (lane & 3) * 2 + (e & 1) < p.group)
                            to[(e >> 1) * 8 * p.group + t * 8 + (e & 1)] = s[t][e];
            }
            if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
                for (int t = 0; t < NH; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(s[t][c], s[t][c + 2]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
                        mx = fmaxf(mx, m[t][c]);
                        const float f = rescale(m[t][c], mx, p.scale_log2);
                        m[t][c] = mx;
                        l[t][c] *= f;
#pragma unroll
                        for (int mt = 0; mt < D / 16; ++mt) {
                            acc[t][mt][c] *= f;
                            acc[t][mt][c + 2] *= f;
                        }
                    }
            }
            uint32_t pb[NH][2];
#pragma unroll
            for (int t = 0; t < NH; ++t) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = weight_of(s[t][e], m[t][e & 1], p.scale_log2);
                l[t][0] += w[0] + w[2];
                l[t][1] += w[1] + w[3];
                // the weights go to the second product as bf16 (nearest even): an error of at most 2^-8
                // relative in each, independent from key to key
                pb[t][0] = movmatrix_trans(ptx::pack_bf16x2(w[0], w[1]));
                pb[t][1] = movmatrix_trans(ptx::pack_bf16x2(w[2], w[3]));
            }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                uint32_t a[4];
                ldmatrix_x4_trans(vs_base + vrow * G::kRow + (((mt * 2 + vchunk) ^ (vrow & 7)) * 16), a);
#pragma unroll
                for (int t = 0; t < NH; ++t) mma_16816(acc[t][mt], a, pb[t][0], pb[t][1]);
            }
            __syncwarp();                               // every lane has read the stage that is filled next
            int next = stage + G::kStages - 1;
            if (next >= G::kStages) next -= G::kStages;
            load(next);
            stage = stage + 1 == G::kStages ? 0 : stage + 1;
        }

        // join the warps: m and l through ml_s, o in halves of d through red
#pragma unroll
        for (int t = 0; t < NH; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[t][c] += __shfl_xor_sync(0xFFFFFFFFu, l[t][c], off);
                if (lane < 4) ml_s[warp][t * 8 + lane * 2 + c] = make_float2(m[t][c], l[t][c]);
            }
        bad = __syncthreads_or(bad);
        const bool whole = row_first >= u0 && row_end <= u1;
        const int slot = 2 * blockIdx.x + (row_first >= u0 ? 1 : 0);
        const long long row_id = ((long long)b * p.Hkv + kv_head) * p.head_blocks + (head0 / kHeads);
#pragma unroll
        for (int t = 0; t < NH; ++t) {
            float f[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float mx = -INFINITY;
                for (int w = 0; w < kDecWarps; ++w) mx = fmaxf(mx, ml_s[w][t * 8 + (lane & 3) * 2 + c].x);
                f[c] = rescale(m[t][c], mx, p.scale_log2);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // red[warp][d / 2][8 heads]
#pragma unroll
                for (int mt = 0; mt < D / 32; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float* a = acc[t][half * (D / 32) + mt];
                        *reinterpret_cast<float2*>(
                            red + (warp * (D / 2) + mt * 16 + e * 8 + (lane >> 2)) * 8 + (lane & 3) * 2) =
                            make_float2(a[2 * e] * f[0], a[2 * e + 1] * f[1]);
                    }
                __syncthreads();
                for (int i = threadIdx.x; i < 8 * (D / 2); i += kDecThreads) {
                    const int hh = i / (D / 2), x = i % (D / 2), h = head0 + t * 8 + hh;
                    float mx = -INFINITY, sum = 0.0f, o = 0.0f;
                    for (int w = 0; w < kDecWarps; ++w) mx = fmaxf(mx, ml_s[w][t * 8 + hh].x);
                    for (int w = 0; w < kDecWarps; ++w) {
                        const float2 ml = ml_s[w][t * 8 + hh];
                        sum += ml.y * rescale(ml.x, mx, p.scale_log2);
                        o += red[(w * (D / 2) + x) * 8 + hh];
                    }
                    const int xd = half * (D / 2) + x;
                    if (whole) {
                        if (h < p.group && !bad) {
                            const long long at = (long long)b * p.H + kv_head * p.group + h;
                            // no weight at all (every logit -inf), or a NaN one: the row is NaN
                            p.o[at * D + xd] = __ushort_as_bfloat16(
                                (unsigned short)round_bf16(sum > 0.0f ? o / sum : NAN, p.round_mode));
                            if (p.lse && xd == 0) p.lse[at] = sum == 0.0f ? -INFINITY : mx * p.scale + logf(sum);
                        }
                        if (kWeights && xd == 0) p.row_ml[row_id * kHeads + t * 8 + hh] = make_float2(mx, bad ? kBadPart : sum);
                    } else {
                        p.part_o[((long long)slot * kHeads + t * 8 + hh) * D + xd] = o;
                        if (xd == 0) p.part_ml[(long long)slot * kHeads + t * 8 + hh] = make_float2(mx, bad ? kBadPart : sum);
                    }
                }
                __syncthreads();
            }
        }
        u += n;
        if (u < u1) {
            cur.tile += n - 1;
            advance(p, cur);
            row_first = u;
        }
    }
}

// One block per CTA boundary of the line: the block of the first boundary inside a row merges the row's
// parts.  It also writes the rows of sequences without keys and reports bad lengths.
template <int D, int NH, bool kWeights>
__global__ void __launch_bounds__(256) attn_decode_join_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int kHeads = 8 * NH, kC = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch();
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const int n = __ldg(p.seqlens_k + b);
        if (n < 0 || (long long)n > (long long)p.pages.max_pages * p.pages.page_size) {
            if (threadIdx.x == 0) report_invalid(ATTN_CACHE_SITE_DECODE);
        } else if (n == 0) {
            for (long long i = threadIdx.x; i < (long long)p.H * D; i += 256)
                p.o[(long long)b * p.H * D + i] = __ushort_as_bfloat16((unsigned short)0x7FC0u);
            if (p.lse)
                for (int h = threadIdx.x; h < p.H; h += 256) p.lse[(long long)b * p.H + h] = -INFINITY;
        }
    }
    const Line line = make_line(p);
    const int c = blockIdx.x;
    if (c < 1 || c >= line.ctas) return;
    const long long u = line.start(c);
    long long first;
    const Cursor cur = seek(p, u, &first);
    if (first == u) return;                            // a row begins here: nothing is split
    const int c0 = line.cta_of(first), c1 = line.cta_of(first + cur.tiles - 1);
    if (c != c0 + 1) return;
    const int kv_head = cur.row / p.head_blocks, block = cur.row - kv_head * p.head_blocks, head0 = block * kHeads;
    for (int hh = warp; hh < kHeads; hh += 8) {
        const int h = head0 + hh;
        if (h >= p.group) break;
        float mx = -INFINITY;
        bool bad = false;
        for (int i = c0 + lane; i <= c1; i += 32) {
            const float2 ml = p.part_ml[(long long)(2 * i + (i == c0)) * kHeads + hh];
            mx = fmaxf(mx, ml.x);
            bad |= ml.y == kBadPart;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        bad = __any_sync(0xFFFFFFFFu, bad);
        float sum = 0.0f, o[kC];
#pragma unroll
        for (int x = 0; x < kC; ++x) o[x] = 0.0f;
        for (int i = c0; i <= c1; ++i) {
            const long long at = (long long)(2 * i + (i == c0)) * kHeads + hh;
            const float2 ml = p.part_ml[at];
            const float f = rescale(ml.x, mx, p.scale_log2);
            sum += ml.y * f;
#pragma unroll
            for (int x = 0; x < kC; ++x) o[x] += p.part_o[at * D + x * 32 + lane] * f;
        }
        if (!bad) {
            const long long at = (long long)cur.b * p.H + kv_head * p.group + h;
#pragma unroll
            for (int x = 0; x < kC; ++x)
                p.o[at * D + x * 32 + lane] = __ushort_as_bfloat16(
                    (unsigned short)round_bf16(sum > 0.0f ? o[x] / sum : NAN, p.round_mode));
            if (p.lse && lane == 0) p.lse[at] = sum == 0.0f ? -INFINITY : mx * p.scale + logf(sum);
        }
        if (kWeights && lane == 0)
            p.row_ml[(((long long)cur.b * p.Hkv + kv_head) * p.head_blocks + block) * kHeads + hh] =
                make_float2(mx, bad ? kBadPart : sum);
    }
}

// Adds every key's softmax weights to its running weight: reads the logits that the attention kernel wrote
// and the rows' final (m, l).  The tiles are divided as there, over (sequence, K/V head) rows.
template <int NH>
__global__ void __launch_bounds__(256) attn_decode_weights_kernel(DecodeParams p) {
    constexpr int kHeads = 8 * NH;
    pdl_wait();
    pdl_launch();
    const int blocks = p.head_blocks;
    p.head_blocks = 1;                                 // a row is a K/V head here
    p.grid = gridDim.x;
    const Line line = make_line(p);
    if ((int)blockIdx.x >= line.ctas) return;
    const long long u1 = line.start(blockIdx.x + 1);
    long long u = line.start(blockIdx.x), first;
    Cursor cur = seek(p, u, &first);
    const long long room = (long long)p.pages.max_pages * p.pages.page_size;
    while (u < u1) {
        const long long left = u1 - u;
        const int n = left < cur.tiles - cur.tile ? (int)left : cur.tiles - cur.tile;
        const int end = min(cur.len, (cur.tile + n) * kDecTile);
        const long long row = (long long)cur.b * p.Hkv + cur.row;
        const float2* ml = p.row_ml + row * blocks * kHeads;     // head g of the group is at g: blocks are full but the last
        for (int j = cur.tile * kDecTile + threadIdx.x; j < end; j += 256) {
            const float* s = p.scores + (row * room + j) * p.group;
            float w = 0.0f;
            bool bad = false;
            for (int g = 0; g < p.group; ++g) {
                const float2 x = ml[g];
                bad |= x.y == kBadPart;
                const float e = s[g] == -INFINITY ? 0.0f : exp2f((s[g] - x.x) * p.scale_log2);
                w += e / x.y;
            }
            if (!bad) p.weights[row * room + j] += w;
        }
        u += n;
        if (u < u1) {
            cur.tile += n - 1;
            advance(p, cur);
        }
    }
}

}  // namespace cache
