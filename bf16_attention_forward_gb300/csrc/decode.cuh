// decode.cuh -- attention of one new token per sequence over a paged K/V cache.
//
// Mathematics.  For every sequence b and query head h over K/V head g = h / (H / Hkv):
//   s_j = q_h . k_j / sqrt(d),  m = max s_j,  l = sum exp(s_j - m),  o_h = sum exp(s_j - m) v_j / l,
// in one pass over the keys with a running m and l; parts of a sequence's keys are joined by
// m = max m_i, l = sum l_i exp(m_i - m), and the same for o.  With `weights` the softmax weight
// of each key, summed over the query heads of its K/V head, is added to a running fp32 weight.
//
// Bound: HBM bytes; every key and value is read once (2 * d * 2 bytes for 4 * d * G flops, G =
// H / Hkv query heads).  64 caches, 2.7 GB of keys and values: 383 to 397 us over boxes, 6.8 to 7.0 TB/s, the
// tensor pipe 10 % busy.  The products run on mma.sync with the KEYS as the M rows and the query heads as the
// N columns (S^T = K Q^T, O^T = V^T P^T): N is 8, so a K/V head's 4 to 8 query heads waste at most
// half of it.  tcgen05 would need 128 rows of one operand and a trip through TMEM for a product
// that takes a few percent of the time.
//
// Work.  A CTA of 8 warps per SM.  The tiles (128 keys) of all (sequence, K/V head) rows form
// one line, which the CTAs divide evenly: a CTA takes a contiguous range, so every CTA reads the
// same bytes whatever the lengths are, and a row is split only where a range ends inside it.
// Behind each row's tiles the line has one more place, which stands for the row's end (loading its
// queries and joining the warps take about as long as a tile).  Each warp streams 16 keys of a tile
// through a ring of its own (cp.async, no barrier between warps) and keeps its own m, l and o; the
// warps are joined at the end of a row.
// Keys and values are read once and leave the L2 first: the logits kept for the weights stay there
// until the join has read them (24 caches, 240,000 keys: 178 -> 171 us), and of caches near the
// L2's size a part stays for the next step (4 caches, 181 MB: 35.5 -> 33.8 us).
// A range holds at most one part that begins before it and one that ends behind it, so two part
// slots per CTA suffice.  A few short rows go to a CTA each instead: one launch, no parts.
// attn_decode_join_kernel merges a split row's parts, and beside that adds the
// weights from the logits that the attention kernel kept.
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
    int whole;                     // 1: a CTA per row, nothing is split, no workspace, no join
    float scale_log2;              // log2(e) / sqrt(d)
    float scale;
    // workspace
    float* part_o;                 // [2 * grid][heads of a block][d]
    float2* part_ml;               // [2 * grid][heads of a block]: (m in logits, l); l = -1: a bad page
    int4* split;                   // [grid]: (b, row, first and last CTA) of a row whose second part is the CTA's, else b = -1
    float2* row_ml;                // [B][Hkv][head_blocks][heads of a block] of unsplit rows (weights only)
    float* scores;                 // [B][H][score_room] logits (weights only)
    long long score_room;          // max_pages * page_size rounded up to 16 bytes
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
    static constexpr int kRedRow = D / 2 + 4;                     // floats of a head's half row, padded against bank conflicts
    static constexpr int kRed = kDecWarps * 8 * kRedRow * 4;      // 8 heads, half of d, per warp
    static constexpr int kSmem = kRing + kRed;
};

// tiles of a sequence; 0 for a length that the table has no room for (the join kernel reports it)
__device__ __forceinline__ int seq_tiles(const DecodeParams& p, int n) {
    return n > 0 && (long long)n <= (long long)p.pages.max_pages * p.pages.page_size ? (n - 1) / kDecTile + 1 : 0;
}

// The line: sequence by sequence, row by row, a row's tiles and its end.  (The host refuses sizes whose
// line could have 2^31 places.)
struct Line {
    int units;                     // places
    int ctas;                      // CTAs that get any: min(grid, units)
    int per, more;                 // units / ctas, and how many CTAs have one more
    __device__ __forceinline__ int start(int c) const { return per * c + min(c, more); }
    __device__ __forceinline__ int cta_of(int u) const {
        return u < more * (per + 1) ? u / (per + 1) : more + (u - more * (per + 1)) / per;
    }
};

// rows: of a sequence
__device__ __forceinline__ Line make_line(const DecodeParams& p, int rows) {   // every lane of a warp calls it
    int n = 0;
#pragma unroll 2
    for (int b = threadIdx.x & 31; b < p.B; b += 32) {
        const int t = seq_tiles(p, __ldg(p.seqlens_k + b));
        n += t > 0 ? t + 1 : 0;
    }
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    Line l;
    l.units = n * rows;
    l.ctas = min(l.units, p.grid);
    l.per = l.ctas ? l.units / l.ctas : 1;
    l.more = l.units - l.per * l.ctas;
    return l;
}

struct Cursor {
    int u, b, row, tile, tiles, len;   // place; row: K/V head * head_blocks + block of query heads; tile == tiles: its end
};

// what is at place u of the line (u < units)
__device__ __forceinline__ Cursor seek(const DecodeParams& p, int rows, int u) {
    const int lane = threadIdx.x & 31;
    int done = 0;                      // places of a row, of the sequences before
    Cursor c{u, 0, 0, 0, 1, 0};
#pragma unroll 1
    for (int base = 0; base < p.B; base += 32) {
        const int len = base + lane < p.B ? __ldg(p.seqlens_k + base + lane) : 0, tiles = seq_tiles(p, len);
        const int mine = tiles > 0 ? tiles + 1 : 0;
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, incl, off);
            if (lane >= off) incl += x;
        }
        const unsigned past = __ballot_sync(0xFFFFFFFFu, (done + incl) * rows > u);
        if (past) {
            const int w = __ffs(past) - 1;
            c.b = base + w;
            c.len = __shfl_sync(0xFFFFFFFFu, len, w);
            c.tiles = __shfl_sync(0xFFFFFFFFu, tiles, w);
            const int in = u - (done + __shfl_sync(0xFFFFFFFFu, incl, w) - (c.tiles + 1)) * rows;
            c.row = in / (c.tiles + 1);
            c.tile = in - c.row * (c.tiles + 1);
            break;
        }
        done += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    return c;
}

// to the first tile of the next row (past the last sequence's last row: any place behind the line)
__device__ __forceinline__ void next_row(const DecodeParams& p, int rows, Cursor& c) {
    c.u += c.tiles + 1 - c.tile;
    c.tile = 0;
    if (++c.row < rows) return;
    c.row = 0;
#pragma unroll 1
    while (c.b + 1 < p.B) {
        ++c.b;
        c.len = __ldg(p.seqlens_k + c.b);
        c.tiles = seq_tiles(p, c.len);
        if (c.tiles > 0) break;
    }
}

// The rows of a sequence without keys, and the report of a bad length; by the threads of a block.
__device__ __forceinline__ void keyless(const DecodeParams& p, int b, int n, int d) {
    if (n < 0 || (long long)n > (long long)p.pages.max_pages * p.pages.page_size) {
        if (threadIdx.x == 0) report_invalid(ATTN_CACHE_SITE_DECODE);
    } else if (n == 0) {
#pragma unroll 1
        for (long long i = threadIdx.x; i < (long long)p.H * d; i += blockDim.x)
            p.o[(long long)b * p.H * d + i] = __ushort_as_bfloat16((unsigned short)0x7FC0u);
        if (p.lse)
#pragma unroll 1
            for (int h = threadIdx.x; h < p.H; h += blockDim.x) p.lse[(long long)b * p.H + h] = -INFINITY;
    }
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
    __shared__ float2 ml_s[kDecWarps][kHeads], joined_s[kHeads];
    __shared__ int bad_s[kDecWarps][G::kStages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = ptx::smem_u32(smem) + warp * (G::kStages * G::kStageBytes);
    float* red = reinterpret_cast<float*>(smem + G::kRing);

    pdl_wait();
    pdl_launch();
    const int rows = p.Hkv * p.head_blocks;
    Line line;
    Cursor cur;
    int u0 = 0, u1;
    if (p.whole) {
        cur = Cursor{0, (int)blockIdx.x / rows, (int)blockIdx.x % rows, 0, 0, 0};
        cur.len = __ldg(p.seqlens_k + cur.b);
        u1 = cur.tiles = seq_tiles(p, cur.len);
        if (cur.row == 0) keyless(p, cur.b, cur.len, D);
        if (u1 == 0) return;
    } else {
        line = make_line(p, rows);
        if ((int)blockIdx.x >= line.ctas) {
            if (threadIdx.x == 0) p.split[blockIdx.x] = make_int4(-1, 0, 0, 0);
            return;
        }
        u0 = line.start(blockIdx.x);
        u1 = line.start(blockIdx.x + 1);
        cur = seek(p, rows, u0);
        if (cur.tile == cur.tiles) next_row(p, rows, cur);
    }
    Cursor ahead = cur;
    const Cursor at0 = cur;
    const long long key_stride = (long long)p.Hkv * G::kRow;
    const uint64_t stream_policy = ptx::policy_evict_first(), keep_policy = ptx::policy_evict_last();

    // Where the loads are: find() looks up the rows of this warp's 16 keys of the tile at `ahead` (-1: past the
    // length or on a page that does not exist) and moves on; load() copies the tile found before into a
    // stage, absent rows as zeros.  A tile is found one load ahead, so that the table's latency is hidden.
    struct Found { int row, kv_head; bool bad; };      // kv_head: -1 behind the range
    auto find = [&]() {
        Found f{-1, -1, false};
        if (ahead.u >= u1) return f;
        f.kv_head = ahead.row / p.head_blocks;
        const int j = ahead.tile * kDecTile + warp * kDecKeys + lane;
        if (lane < kDecKeys && j < ahead.len) {
            f.row = page_row(p.pages, p.pages.table + (long long)ahead.b * p.pages.max_pages, j);
            f.bad = f.row < 0;
        }
        ++ahead.u;
        if (++ahead.tile == ahead.tiles && ahead.u < u1) next_row(p, rows, ahead);
        return f;
    };
    auto load = [&](int stage, const Found& f) {
        if (f.kv_head >= 0) {
            const bool any_bad = __any_sync(0xFFFFFFFFu, f.bad);
            if (lane == 0) {
                bad_s[warp][stage] = any_bad;
                if (any_bad) report_invalid(ATTN_CACHE_SITE_DECODE);
            }
            const int chunk = lane % kChunks;
            const long long col = (long long)f.kv_head * G::kRow + chunk * 16;
            const uint32_t dst = ring + stage * G::kStageBytes;
#pragma unroll
            for (int i = 0; i < kDecKeys / kRowsPerCopy; ++i) {
                const int r = i * kRowsPerCopy + lane / kChunks;
                const int src_row = __shfl_sync(0xFFFFFFFFu, f.row, r);
                const long long off = (long long)max(src_row, 0) * key_stride + col;
                const uint32_t at = dst + r * G::kRow + ((chunk ^ (r & 7)) * 16);
                const uint32_t bytes = src_row < 0 ? 0u : 16u;
                cp_async16(at, p.k + off, bytes, stream_policy);
                cp_async16(at + kDecKeys * G::kRow, p.v + off, bytes, stream_policy);
            }
        }
        cp_async_commit();
    };
    // (code that runs once is kept short: every launch fetches it anew)
    Found next_tile = find();
#pragma unroll 1
    for (int s = 0; s < G::kStages - 1; ++s) {
        const Found f = next_tile;
        next_tile = find();
        load(s, f);
    }

    // ldmatrix addresses inside a stage: lane i gives row i % 8 of 8x8 matrix i / 8
    const int mat = lane >> 3, mrow = lane & 7;
    const int krow = mrow + (mat & 1) * 8, kchunk = mat >> 1;          // K: rows 0-7, 8-15, then the next chunk
    const int vrow = mrow + (mat >> 1) * 8, vchunk = mat & 1;          // V (transposed): chunks, then rows 8-15
    const float tau = 8.0f / p.scale_log2;                             // a reference may lag by 2^8
    int stage = 0;

    while (cur.u < u1) {
        const int kv_head = cur.row / p.head_blocks, head0 = (cur.row - kv_head * p.head_blocks) * kHeads;
        const int n = min(cur.tiles - cur.tile, u1 - cur.u);           // tiles of this row in the range
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
#pragma unroll 1
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
                const long long room = p.score_room;
                float* to = p.scores + ((long long)b * p.H + kv_head * p.group + head0 + (lane & 3) * 2) * room + j0;
#pragma unroll
                for (int t = 0; t < NH; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j0 + (e >> 1) * 8 < len && head0 + t * 8 + (lane & 3) * 2 + (e & 1) < p.group)
                            st_policy(to + (t * 8 + (e & 1)) * room + (e >> 1) * 8, s[t][e], keep_policy);
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
            // The weights go to the second product as two bf16 parts, the upper 8 bits and the next 8 (an error of 2^-16;
            // one part alone would add 2^-9 to every weight, as much as rounding the output).  Both parts of a
            // positive weight are positive, so that an infinite value stays infinite.
            uint32_t hi[NH][2], lo[NH][2];
#pragma unroll
            for (int t = 0; t < NH; ++t) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = weight_of(s[t][e], m[t][e & 1], p.scale_log2);
                l[t][0] += w[0] + w[2];
                l[t][1] += w[1] + w[3];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t h = ptx::pack_bf16x2_rz(w[2 * c], w[2 * c + 1]);
                    const float r0 = w[2 * c] - __uint_as_float(h << 16), r1 = w[2 * c + 1] - __uint_as_float(h & 0xFFFF0000u);
                    hi[t][c] = movmatrix_trans(h);
                    lo[t][c] = movmatrix_trans(ptx::pack_bf16x2(w[2 * c] > 0.0f ? fmaxf(r0, 0x1p-126f) : r0,
                                                                w[2 * c + 1] > 0.0f ? fmaxf(r1, 0x1p-126f) : r1));
                }
            }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                uint32_t a[4];
                ldmatrix_x4_trans(vs_base + vrow * G::kRow + (((mt * 2 + vchunk) ^ (vrow & 7)) * 16), a);
#pragma unroll
                for (int t = 0; t < NH; ++t) {
                    mma_16816(acc[t][mt], a, hi[t][0], hi[t][1]);
                    mma_16816(acc[t][mt], a, lo[t][0], lo[t][1]);
                }
            }
            __syncwarp();                               // every lane has read the stage that is filled next
            int next = stage + G::kStages - 1;
            if (next >= G::kStages) next -= G::kStages;
            load(next, next_tile);
            next_tile = find();
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
        const bool whole = n == cur.tiles;
        const long long slot = (2 * blockIdx.x + (cur.tile == 0 ? 1 : 0)) * kHeads;
        const long long out0 = (long long)b * p.H + kv_head * p.group + head0;
        if (threadIdx.x < kHeads) {
            const int h = threadIdx.x;
            float mx = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) mx = fmaxf(mx, ml_s[w][h].x);
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) sum += ml_s[w][h].y * rescale(ml_s[w][h].x, mx, p.scale_log2);
            // no weight at all (every logit -inf), or a NaN one: the row is NaN
            joined_s[h] = make_float2(mx, whole ? (sum > 0.0f ? 1.0f / sum : NAN) : 1.0f);
            const float2 ml = make_float2(mx, bad ? kBadPart : sum);
            if (!whole) p.part_ml[slot + h] = ml;
            else if (h < p.group - head0) {
                if (p.lse && !bad) p.lse[out0 + h] = sum == 0.0f ? -INFINITY : mx * p.scale + logf(sum);
                if (kWeights) p.row_ml[(((long long)b * p.Hkv + kv_head) * p.head_blocks + head0 / kHeads) * kHeads + h] = ml;
            }
        }
        // o in halves of d, 8 heads at a time: red[warp][head][d / 2]
#pragma unroll
        for (int t = 0; t < NH; ++t) {
            float f[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < kDecWarps; ++w) mx = fmaxf(mx, ml_s[w][t * 8 + (lane & 3) * 2 + c].x);
                f[c] = rescale(m[t][c], mx, p.scale_log2);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float* to = red + (warp * 8 + (lane & 3) * 2) * G::kRedRow + (lane >> 2);
#pragma unroll
                for (int mt = 0; mt < D / 32; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        to[(e & 1) * G::kRedRow + mt * 16 + (e >> 1) * 8] = acc[t][half * (D / 32) + mt][e] * f[e & 1];
                __syncthreads();
                // two neighbouring elements of a head a thread
                for (int i = threadIdx.x; i < 8 * (D / 4); i += kDecThreads) {
                    const int hh = i / (D / 4), x = i % (D / 4) * 2;
                    float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < kDecWarps; ++w) {
                        const float2 part = *reinterpret_cast<const float2*>(red + (w * 8 + hh) * G::kRedRow + x);
                        o.x += part.x;
                        o.y += part.y;
                    }
                    const int xd = half * (D / 2) + x, h = t * 8 + hh;
                    if (!whole) {
                        *reinterpret_cast<float2*>(p.part_o + (slot + h) * D + xd) = o;
                    } else if (head0 + h < p.group && !bad) {
                        const float inv = joined_s[h].y;
                        *reinterpret_cast<uint32_t*>(p.o + (out0 + h) * D + xd) =
                            round_bf16(o.x * inv, p.round_mode) | round_bf16(o.y * inv, p.round_mode) << 16;
                    }
                }
                __syncthreads();
            }
        }
        next_row(p, rows, cur);
    }
    if (!p.whole && threadIdx.x == 0) {
        // a row whose second part was this CTA's: for the join
        int4 d = make_int4(-1, 0, 0, 0);
        const int first = at0.u - at0.tile;
        if (at0.tile > 0 && line.cta_of(first) + 1 == (int)blockIdx.x)
            d = make_int4(at0.b, at0.row, blockIdx.x - 1, line.cta_of(first + at0.tiles - 1));
        p.split[blockIdx.x] = d;
    }
}

// The join.  Blocks 0 .. grid - 1: the block of the CTA that has a split row's second part merges the row's parts;
// they also write the rows of sequences without keys and report bad lengths.  With kWeights the blocks
// behind them add every key's softmax weights to its running weight, from the logits that the attention kernel
// kept and the rows' (m, l); they divide the tiles evenly over (sequence, K/V head) rows.
template <int D, int NH, bool kWeights>
__global__ void __launch_bounds__(256, 4) attn_decode_join_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int kHeads = 8 * NH, kC = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch();
    if ((int)blockIdx.x < p.grid) {
        const int4 row = p.split[blockIdx.x];
        const int b = row.x, c0 = row.z, c1 = row.w;
        const int kv_head = row.y / p.head_blocks, head0 = (row.y - kv_head * p.head_blocks) * kHeads;
#pragma unroll 1
        for (int hh = warp; b >= 0 && hh < kHeads && head0 + hh < p.group; hh += 8) {
            // a row's first part is in slot 1 of its CTA, the others in slot 0 of theirs
            auto part = [&](int i) { return (long long)(2 * i + (i == c0)) * kHeads + hh; };
            // the weight of part c0 + lane of the row, and of parts past the 31st later
            float2 ml = c0 + lane <= c1 ? p.part_ml[part(c0 + lane)] : make_float2(-INFINITY, 0.0f);
            constexpr int kU = 4;                      // parts in flight
            float v[kU][kC], sum = 0.0f, o[kC];
            auto load = [&](int i0) {
                const float* from = p.part_o + part(i0) * D + lane;
#pragma unroll
                for (int j = 0; j < kU; ++j) {
                    if (i0 + j <= c1)
#pragma unroll
                        for (int x = 0; x < kC; ++x) v[j][x] = from[x * 32];
                    from = p.part_o + part(i0 + j + 1) * D + lane;
                }
            };
            float mx = ml.x;
#pragma unroll 1
            for (int i = c0 + 32 + lane; i <= c1; i += 32) mx = fmaxf(mx, p.part_ml[part(i)].x);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
            bool bad = false;
#pragma unroll
            for (int x = 0; x < kC; ++x) o[x] = 0.0f;
#pragma unroll 1
            for (int i0 = c0; i0 <= c1; i0 += kU) {
                load(i0);
                const int j0 = (i0 - c0) & 31;
                if (j0 == 0 && i0 > c0) ml = i0 + lane <= c1 ? p.part_ml[part(i0 + lane)] : make_float2(-INFINITY, 0.0f);
                bad |= ml.y == kBadPart;
                const float f = rescale(ml.x, mx, p.scale_log2), s = ml.y * f;
#pragma unroll
                for (int j = 0; j < kU; ++j) {
                    const float fj = __shfl_sync(0xFFFFFFFFu, f, j0 + j), sj = __shfl_sync(0xFFFFFFFFu, s, j0 + j);
                    if (i0 + j > c1) continue;
                    sum += sj;
#pragma unroll
                    for (int x = 0; x < kC; ++x) o[x] += v[j][x] * fj;
                }
            }
            if (__any_sync(0xFFFFFFFFu, bad)) continue;
            const long long at = (long long)b * p.H + kv_head * p.group + head0 + hh;
            const float inv = sum > 0.0f ? 1.0f / sum : NAN;
#pragma unroll
            for (int x = 0; x < kC; ++x)
                p.o[at * D + x * 32 + lane] = __ushort_as_bfloat16((unsigned short)round_bf16(o[x] * inv, p.round_mode));
            if (p.lse && lane == 0) p.lse[at] = sum == 0.0f ? -INFINITY : mx * p.scale + logf(sum);
        }
#pragma unroll 1
        for (int s = blockIdx.x; s < p.B; s += p.grid) keyless(p, s, __ldg(p.seqlens_k + s), D);
        return;
    }
    if constexpr (kWeights) {
        constexpr int kG = 8;                          // query heads at a time
        __shared__ float2 ml_s[kG];                    // (m, 1 / l)
        __shared__ int bad_s;
        const Line line = make_line(p, p.Hkv * p.head_blocks);
        // this block's places on the line of K/V heads, which has one for head_blocks of the attention kernel's
        const int units = line.units / p.head_blocks, block = blockIdx.x - p.grid, blocks = gridDim.x - p.grid;
        const int per = units / blocks, more = units - per * blocks;
        const int t0 = per * block + min(block, more), t1 = t0 + per + (block < more);
        if (t0 >= t1) return;
        const long long room = (long long)p.pages.max_pages * p.pages.page_size;
        const bool vector = room % 4 == 0 && reinterpret_cast<uintptr_t>(p.weights) % 16 == 0;
        const uint64_t done_policy = ptx::policy_evict_first();
        Cursor cur = seek(p, p.Hkv, t0);
#pragma unroll 1
        for (; cur.u < t1; next_row(p, p.Hkv, cur)) {
            const int n = min(cur.tiles - cur.tile, t1 - cur.u);
            if (n == 0) continue;
            const int j1 = min(cur.len, (cur.tile + n) * kDecTile);
            const long long kv = (long long)cur.b * p.Hkv + cur.row;
            // the place of the head's first row on the attention kernel's line: the places of the heads before it
            // count there head_blocks times
            const int main0 = (cur.u - cur.tile) * p.head_blocks;
            float* out = p.weights + kv * room;
#pragma unroll 1
            for (int g0 = 0; g0 < p.group; g0 += kG) {
                __syncthreads();
                if (threadIdx.x == 0) bad_s = 0;
                __syncthreads();
                if (warp < kG && g0 + warp < p.group) {
                    const int g = g0 + warp, blk = g / kHeads, hh = g - blk * kHeads;
                    const int r0 = main0 + blk * (cur.tiles + 1);
                    const int c0 = line.cta_of(r0), c1 = line.cta_of(r0 + cur.tiles - 1);
                    float2 ml;
                    if (c0 == c1) {
                        ml = p.row_ml[(kv * p.head_blocks + blk) * kHeads + hh];
                    } else {
                        float mx = -INFINITY, sum = 0.0f;
                        bool bad = false;
#pragma unroll 1
                        for (int i = c0 + lane; i <= c1; i += 32) {
                            const float2 x = p.part_ml[(long long)(2 * i + (i == c0)) * kHeads + hh];
                            mx = fmaxf(mx, x.x);
                            bad |= x.y == kBadPart;
                        }
#pragma unroll
                        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
#pragma unroll 1
                        for (int i = c0; i <= c1; ++i) {
                            const float2 x = p.part_ml[(long long)(2 * i + (i == c0)) * kHeads + hh];
                            sum += x.y * rescale(x.x, mx, p.scale_log2);
                        }
                        ml = make_float2(mx, __any_sync(0xFFFFFFFFu, bad) ? kBadPart : sum);
                    }
                    if (lane == 0) {
                        ml_s[warp] = make_float2(ml.x, 1.0f / ml.y);
                        if (ml.y == kBadPart) bad_s = 1;
                    }
                }
                __syncthreads();
                if (bad_s) break;
                // four neighbouring keys a thread: 16-byte loads (4-byte ones left the loop at 2.5 TB/s)
#pragma unroll 1
                for (int j0 = cur.tile * kDecTile + threadIdx.x * 4; j0 < j1; j0 += 1024) {
                    const float* s =
                        p.scores + ((long long)cur.b * p.H + (long long)cur.row * p.group + g0) * p.score_room + j0;
                    float4 x[kG], w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int g = 0; g < kG; ++g)
                        if (g0 + g < p.group)
                            x[g] = ld_policy(reinterpret_cast<const float4*>(s + g * p.score_room), done_policy);
                    if (vector) {
                        w = *reinterpret_cast<const float4*>(out + j0);
                    } else {
                        w.x = out[j0];
                        if (j0 + 1 < j1) w.y = out[j0 + 1];
                        if (j0 + 2 < j1) w.z = out[j0 + 2];
                        if (j0 + 3 < j1) w.w = out[j0 + 3];
                    }
                    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int g = 0; g < kG; ++g) {
                        if (g0 + g >= p.group) continue;
                        const float2 ml = ml_s[g];
                        // (-inf logits weigh nothing, but in a row of nothing else, which is NaN: 0 / 0)
                        auto weight = [&](float v) {
                            return (v == -INFINITY ? 0.0f : ptx::ex2_approx((v - ml.x) * p.scale_log2)) * ml.y;
                        };
                        sum.x += weight(x[g].x);
                        sum.y += weight(x[g].y);
                        sum.z += weight(x[g].z);
                        sum.w += weight(x[g].w);
                    }
                    w.x += sum.x; w.y += sum.y; w.z += sum.z; w.w += sum.w;
                    if (vector && j0 + 3 < j1) {
                        *reinterpret_cast<float4*>(out + j0) = w;
                    } else {
                        out[j0] = w.x;
                        if (j0 + 1 < j1) out[j0 + 1] = w.y;
                        if (j0 + 2 < j1) out[j0 + 2] = w.z;
                        if (j0 + 3 < j1) out[j0 + 3] = w.w;
                    }
                }
            }
        }
    }
}

}  // namespace cache
