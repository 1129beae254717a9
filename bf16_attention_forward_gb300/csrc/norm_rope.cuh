// norm_rope.cuh -- norms of queries and keys for each head, with their rotary positions in the same pass; the
// gradient; and the form that writes the keys to a paged cache.
//
// Mathematics.  Of a head x of d elements, with weights w:
//   r = 1 / sqrt(sum x_i^2 / d + eps),  n = r x,  y = R(n * w),
// R the rotation of rope.cuh (pair p by pos[axis[p]] * freq[p]).  Of the gradient dy, with g = R^T dy:
//   dw = sum over heads and tokens of g * n,  dx = r (g * w - n (sum (g * w)_i n_i) / d).
// All of it in fp32, y and dx rounded once.  (The squares' sum is fp32 too: elements past 10^19 overflow it, r is 0.)
//
// Bound: HBM bytes; x read and y written once (backward: x and dy read, dx written).  The threads stand as in rope.cuh:
// a warp takes a token, whose angles it computes once; D / 16 lanes take a head, 16 elements each, so the sums over a
// head are 2 or 3 shuffles.  Weights are fp32 in shared memory: 64 bytes of it a thread and head beside 32 from HBM.
#pragma once
#include "rope.cuh"

namespace cache {

struct NormRopeParams {
    RopeTensor x[3];               // q, k, v (v is copied; only when appending); backward: x is read, dst = dx
    RopeTensor dy[2];              // backward: the gradients (src)
    const void* weight[2];         // [d] fp32 or bf16, or null (ones)
    int weight_bf16;
    float eps;
    const int32_t* positions;      // null with pairs = 0
    const double* freqs;
    const int32_t* axes;
    long long pos_axis, pos_b;     // element strides of positions
    long long S, tokens;           // tokens per batch entry, and in all
    int pairs, num_axes, heads_per_block, heads;
    // appending
    const int64_t* slots;          // [tokens] rows of the cache, -1: none
    long long rows;                // of the cache
    // backward
    float* part;                   // [blocks][D] sums of dw
    float* dw[2];                  // [d] or null
    int blocks[2];                 // of q and of k
};

constexpr int kNormThreads = 128;
constexpr int kNormWarps = kNormThreads / 32;

// The rotation's tables in shared memory, by the threads of a block; true (for all) when an axis is not there.
template <int D>
struct TurnTable {
    unsigned long long turn[D / 2];
    int axis[D / 2];
    __device__ __forceinline__ bool fill(const NormRopeParams& p) {
        int bad = 0;
        for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) {
            const double freq = p.freqs[i];
            const int a = p.axes[i];
            turn[i] = turn_of(freq);
            axis[i] = isfinite(freq) ? a : ~a;             // (an infinite frequency or NaN: the pair becomes NaN)
            bad |= (unsigned)a >= (unsigned)p.num_axes;
        }
        return __syncthreads_or(bad);
    }
    // cosines and sines of a token's pairs, by the lanes of a warp
    __device__ __forceinline__ void angles(const NormRopeParams& p, long long b, long long s, float2* cs) const {
        __syncwarp();                                      // (the token before is done with cs)
#pragma unroll 1
        for (int pr = threadIdx.x & 31; pr < p.pairs; pr += 32) {
            const int a = axis[pr];
            const long long pos = __ldg(p.positions + (a < 0 ? ~a : a) * p.pos_axis + b * p.pos_b + s);
            const long long at = (long long)(turn[pr] * (unsigned long long)pos);
            float sn, c;
            sincospif(a < 0 ? NAN : (float)at * 0x1p-63f, &sn, &c);
            cs[pr] = make_float2(c, sn);
        }
        __syncwarp();
    }
};

// Where a lane's 16 elements of a head are: two chunks of 8 (a pair has its elements in one thread), and the first pair
// of each half of them.
template <int D, bool kHalves>
struct Place {
    int ca, cb, pa, pb;
    __device__ __forceinline__ Place(int l, int pairs) {
        if constexpr (kHalves) {
            const int rot = pairs / 8;
            ca = l < rot ? l : 2 * rot + 2 * (l - rot);
            cb = l < rot ? l + rot : ca + 1;
            pa = l < rot ? 8 * l : pairs;
            pb = pa + 4;
        } else {
            ca = l;
            cb = l + D / 16;
            pa = 4 * ca;
            pb = 4 * cb;
        }
    }
    // cosines and sines of the thread's 8 pairs; returns which of them turn, a bit each
    __device__ __forceinline__ uint32_t take(const float2* cs, int pairs, float (&c)[8], float (&sn)[8]) const {
        uint32_t turns = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int pr = e < 4 ? pa + e : pb + e - 4;
            const bool t = pr < pairs;
            const float2 v = t ? cs[pr] : make_float2(1.0f, 0.0f);
            turns |= (uint32_t)t << e;
            c[e] = v.x;
            sn[e] = v.y;
        }
        return turns;
    }
    // the thread's elements (chunk a in x[0..7], chunk b in x[8..15]) turned by the angles, or by their negatives (a pair
    // that does not turn is left alone: a NaN in one of its elements stays there)
    template <bool kBack>
    static __device__ __forceinline__ void turn(float (&x)[16], const float (&c)[8], const float (&sn)[8], uint32_t turns) {
        if (turns == 0) return;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = kHalves ? e : 2 * e, j = kHalves ? e + 8 : 2 * e + 1;
            const float s = kBack ? -sn[e] : sn[e], x0 = x[i], x1 = x[j];
            if (!kHalves && !(turns >> e & 1u)) continue;      // (halves: all 8 or none)
            x[i] = x0 * c[e] - x1 * s;
            x[j] = x1 * c[e] + x0 * s;
        }
    }
};

__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&x)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void pack16(const float (&x)[16], uint4& a, uint4& b) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = ptx::pack_bf16x2(x[2 * i], x[2 * i + 1]);
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}
// a head's weights of the thread's two chunks
__device__ __forceinline__ void weights16(const float* w, int ca, int cb, float (&x)[16]) {
    *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(w + ca * 8);
    *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(w + ca * 8 + 4);
    *reinterpret_cast<float4*>(x + 8) = *reinterpret_cast<const float4*>(w + cb * 8);
    *reinterpret_cast<float4*>(x + 12) = *reinterpret_cast<const float4*>(w + cb * 8 + 4);
}
__device__ __forceinline__ float weight_at(const NormRopeParams& p, int t, int i) {
    if (!p.weight[t]) return 1.0f;
    return p.weight_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.weight[t])[i])
                         : reinterpret_cast<const float*>(p.weight[t])[i];
}
// the sum over the lanes of a head
template <int kL>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int off = 1; off < kL; off <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

template <int D, bool kHalves, bool kAppend>
__global__ void __launch_bounds__(kNormThreads, 5) attn_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int kL = D / 16;     // lanes of a head
    constexpr int kSub = 32 / kL;  // heads that a warp takes side by side
    __shared__ TurnTable<D> table;
    __shared__ __align__(16) float w_s[2][D];
    __shared__ float2 cs[kNormWarps][D / 2];
    pdl_wait();
    pdl_launch();
    for (int i = threadIdx.x; i < 2 * D; i += kNormThreads) w_s[i / D][i % D] = weight_at(p, i / D, i % D);
    if (table.fill(p)) {
        if (threadIdx.x == 0) report_invalid(ATTN_CACHE_SITE_AXES);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Place<D, kHalves> place(lane % kL, p.pairs);
    const int h_first = blockIdx.y * p.heads_per_block, h_begin = h_first + lane / kL;
    const int h_end = min(h_first + p.heads_per_block, p.heads);
    // which tensor head h of the token belongs to, and its number there
    auto tensor_of = [&](int& h) {
        int t = 0;
        if (h >= p.x[0].heads) { h -= p.x[0].heads; t = 1; }
        if (kAppend && t == 1 && h >= p.x[1].heads) { h -= p.x[1].heads; t = 2; }
        return t;
    };
#pragma unroll 1
    for (long long token = (long long)blockIdx.x * kNormWarps + warp; token < p.tokens;
         token += (long long)gridDim.x * kNormWarps) {
        const long long b = kAppend ? 0 : token / p.S, s = kAppend ? token : token - b * p.S;
        struct Heads { uint4 a[kRopeHeads], b[kRopeHeads]; };
        auto load = [&](int h0, Heads& x) {
#pragma unroll
            for (int u = 0; u < kRopeHeads; ++u) {
                int h = h0 + u * kSub;
                x.a[u] = x.b[u] = make_uint4(0u, 0u, 0u, 0u);
                if (h >= h_end) continue;
                const RopeTensor& t = p.x[tensor_of(h)];
                const char* src = t.src + b * t.src_b + s * t.src_t + h * t.src_h;
                x.a[u] = *reinterpret_cast<const uint4*>(src + place.ca * 16);
                x.b[u] = *reinterpret_cast<const uint4*>(src + place.cb * 16);
            }
        };
        Heads x, next;
        long long row = -1;        // the token's row of the cache
        if constexpr (kAppend) {
            row = __ldg(reinterpret_cast<const long long*>(p.slots) + token);
            load(h_begin, x);      // (beside the slot's read: a token without a slot is rare)
            if (row == -1) continue;
            if (row < 0 || row >= p.rows) {
                row = -1;
                if (lane == 0) report_invalid(ATTN_CACHE_SITE_SLOTS);
            }
        } else {
            load(h_begin, x);
        }
        table.angles(p, b, s, cs[warp]);
        float c[8], sn[8];
        const uint32_t turns = place.take(cs[warp], p.pairs, c, sn);
#pragma unroll 1
        for (int h0 = h_first; h0 < h_end; h0 += kRopeHeads * kSub) {      // (every lane of the warp)
            load(h0 + lane / kL + kRopeHeads * kSub, next);
#pragma unroll
            for (int u = 0; u < kRopeHeads; ++u) {
                int h = h0 + lane / kL + u * kSub;
                const bool there = h < h_end;
                float v[16];
                unpack16(x.a[u], x.b[u], v);
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e) ss += v[e] * v[e];
                const float r = rsqrtf(head_sum<kL>(ss) * (1.0f / D) + p.eps);
                if (!there) continue;
                const int t = tensor_of(h);
                if (kAppend && t > 0 && row < 0) continue;
                if (!kAppend || t < 2) {
                    float w[16];
                    weights16(w_s[t], place.ca, place.cb, w);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] *= r * w[e];
                    place.template turn<false>(v, c, sn, turns);
                    pack16(v, x.a[u], x.b[u]);
                }
                const RopeTensor& to = p.x[t];
                char* dst = to.dst + b * to.dst_b + (kAppend && t > 0 ? row : s) * to.dst_t + h * to.dst_h;
                *reinterpret_cast<uint4*>(dst + place.ca * 16) = x.a[u];
                *reinterpret_cast<uint4*>(dst + place.cb * 16) = x.b[u];
            }
            x = next;
        }
    }
}

// The gradient.  Blocks 0 .. blocks[0] - 1 take q, the others k, each tokens in turn; a thread sums its 16 elements of dw
// over all of its heads, a block adds up its threads' in a fixed order, and attn_norm_rope_dw_kernel the blocks'.
template <int D, bool kHalves>
__global__ void __launch_bounds__(kNormThreads, 4) attn_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int kL = D / 16, kSub = 32 / kL;
    __shared__ TurnTable<D> table;
    __shared__ __align__(16) float w_s[D];
    __shared__ float2 cs[kNormWarps][D / 2];
    __shared__ float sum_s[kNormWarps][D];
    pdl_wait();
    pdl_launch();
    const int t = (int)blockIdx.x >= p.blocks[0], block = blockIdx.x - t * p.blocks[0];
    for (int i = threadIdx.x; i < D; i += kNormThreads) w_s[i] = weight_at(p, t, i);
    if (table.fill(p)) {
        if (threadIdx.x == 0) report_invalid(ATTN_CACHE_SITE_AXES);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Place<D, kHalves> place(lane % kL, p.pairs);
    const RopeTensor &tx = p.x[t], &tg = p.dy[t];
    float dw[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) dw[e] = 0.0f;
#pragma unroll 1
    for (long long token = (long long)block * kNormWarps + warp; token < p.tokens;
         token += (long long)p.blocks[t] * kNormWarps) {
        const long long b = token / p.S, s = token - b * p.S;
        struct Head { uint4 xa, xb, ga, gb; };
        auto load = [&](int h) {
            Head y;
            y.xa = y.xb = y.ga = y.gb = make_uint4(0u, 0u, 0u, 0u);
            if (h < tx.heads) {
                const char* x = tx.src + b * tx.src_b + s * tx.src_t + h * tx.src_h;
                const char* g = tg.src + b * tg.src_b + s * tg.src_t + h * tg.src_h;
                y.xa = *reinterpret_cast<const uint4*>(x + place.ca * 16);
                y.xb = *reinterpret_cast<const uint4*>(x + place.cb * 16);
                y.ga = *reinterpret_cast<const uint4*>(g + place.ca * 16);
                y.gb = *reinterpret_cast<const uint4*>(g + place.cb * 16);
            }
            return y;
        };
        Head y = load(lane / kL);
        table.angles(p, b, s, cs[warp]);
        float c[8], sn[8];
        const uint32_t turns = place.take(cs[warp], p.pairs, c, sn);
#pragma unroll 1
        for (int h0 = 0; h0 < tx.heads; h0 += kSub) {
            const int h = h0 + lane / kL;
            const Head next = load(h + kSub);
            float x[16], g[16], w[16];
            unpack16(y.xa, y.xb, x);
            unpack16(y.ga, y.gb, g);
            place.template turn<true>(g, c, sn, turns);
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) ss += x[e] * x[e];
            const float r = rsqrtf(head_sum<kL>(ss) * (1.0f / D) + p.eps);
            weights16(w_s, place.ca, place.cb, w);
            float dot = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                x[e] *= r;
                if (h < tx.heads) dw[e] += g[e] * x[e];    // (an absent head's r may be infinite)
                g[e] *= w[e];
                dot += g[e] * x[e];
            }
            dot = head_sum<kL>(dot) * (1.0f / D);
            if (h < tx.heads) {
#pragma unroll
                for (int e = 0; e < 16; ++e) g[e] = r * (g[e] - x[e] * dot);
                char* dst = tx.dst + b * tx.dst_b + s * tx.dst_t + h * tx.dst_h;
                uint4 oa, ob;
                pack16(g, oa, ob);
                *reinterpret_cast<uint4*>(dst + place.ca * 16) = oa;
                *reinterpret_cast<uint4*>(dst + place.cb * 16) = ob;
            }
            y = next;
        }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int off = kL; off < 32; off <<= 1) dw[e] += __shfl_xor_sync(0xFFFFFFFFu, dw[e], off);
        if (lane < kL) sum_s[warp][(e < 8 ? place.ca : place.cb) * 8 + (e & 7)] = dw[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kNormThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kNormWarps; ++w) v += sum_s[w][i];
        p.part[(long long)blockIdx.x * D + i] = v;
    }
}

// dw: a block of 32 columns of a tensor; thread (y, x) sums column x of every 32nd block's sums, from y on.
constexpr int kDwRows = 32;
template <int D>
__global__ void __launch_bounds__(32 * kDwRows) attn_norm_rope_dw_kernel(const __grid_constant__ NormRopeParams p) {
    __shared__ float sum_s[kDwRows][32];
    pdl_wait();
    pdl_launch();
    const int t = blockIdx.x / (D / 32), col = blockIdx.x % (D / 32) * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    if (!p.dw[t]) return;
    // (with a bad axis the sums were not written, and neither is dw: the pass before has reported it)
    int bad = 0;
    for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) bad |= (unsigned)p.axes[i] >= (unsigned)p.num_axes;
    if (__syncthreads_or(bad)) return;
    const float* part = p.part + (t ? (long long)p.blocks[0] * D : 0) + col;
    float v = 0.0f;
#pragma unroll 8
    for (int i = y; i < p.blocks[t]; i += kDwRows) v += part[(long long)i * D];
    sum_s[y][threadIdx.x & 31] = v;
    __syncthreads();
    if (y == 0) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < kDwRows; ++i) v += sum_s[i][threadIdx.x];
        p.dw[t][col] = v;
    }
}

}  // namespace cache
