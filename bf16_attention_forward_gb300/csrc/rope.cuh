// rope.cuh -- rotary positions with several axes, and their form that writes a paged cache.
//
// Mathematics.  Pair p of a head's rotated dimensions turns by theta = pos[axis[p]] * freq[p]:
//   y0 = x0 cos(theta) - x1 sin(theta),  y1 = x1 cos(theta) + x0 sin(theta),
// with (x0, x1) = (x[2p], x[2p+1]) ("adjacent") or (x[p], x[p+P]) ("halves", P pairs); the
// backward is the rotation by -theta.  The remaining dimensions pass through bit for bit.
//
// Angles.  Positions reach 2^31, where pos * freq in fp32 has no correct digit left.  The
// kernel keeps freq / 2pi as a 64-bit binary fraction of a turn; an integer position times it,
// modulo 2^64, is the fraction of a turn (whole turns drop out of the high end), exact
// but for the fraction's own last bit: pos * 2^-64 turns.  The product, read as a signed number of
// half turns in [-1, 1) and rounded to fp32 as a whole (its upper 32 bits alone would leave an angle of
// 10^-7 rad 1 % off), goes to sincospi.
//
// Bound: HBM bytes (each element read and written once).  A warp takes a token: it computes each angle
// once, into shared memory; a thread then holds the cosines and sines of 16 elements and applies
// them to those elements of every 4th (d = 64: 8th) head, so that a warp reads 1 KB of a token at a time.
// (A thread per 16 elements of a token, which reads 256 bytes of four tokens at a time and computes its 8
// angles itself, took 55.7 us where this takes 51.7: 16,384 tokens of 40 heads, 336 MB at 6.5 TB/s.)
#pragma once
#include "cache_common.cuh"

namespace cache {

struct RopeTensor {       // byte strides
    const char* src;
    char* dst;
    long long src_b, src_t, src_h, dst_b, dst_t, dst_h;
    int heads;
};

struct RopeParams {
    RopeTensor x[3];               // q, k, v (v is copied; only when appending)
    const int32_t* positions;
    const double* freqs;
    const int32_t* axes;
    long long pos_axis, pos_b;     // element strides of positions
    long long S, tokens;           // tokens per batch entry, and in all
    int pairs, num_axes, inverse, heads_per_block, heads;
    // appending
    Pages pages;
    const int32_t* cu_new;
    const int32_t* seqlens_k;
    int B;
};

constexpr int kRopeThreads = 128;
constexpr int kRopeHeads = 2;       // heads that a thread turns at a time, while the next ones are on their way
constexpr int kCuStage = 1024;     // sequence offsets that a block searches in shared memory

// bf16 pair (x0 in the low half) turned by (c, s)
__device__ __forceinline__ uint32_t rotate_word(uint32_t w, float c, float s) {
    const float x0 = __uint_as_float(w << 16), x1 = __uint_as_float(w & 0xFFFF0000u);
    return ptx::pack_bf16x2(x0 * c - x1 * s, x1 * c + x0 * s);
}

// freq / 2pi without its whole turns, in units of 2^-64 turns (rounded towards zero): the 53-bit mantissa times
// 1 / 2pi in 128 bits, shifted by the exponent.  (In fp64 the product alone is off by 2^-53 of the frequency, 2^-22
// radians per radian of it at position 2^31, and a second part for its error took this kernel 0.6 us more.)
__device__ __forceinline__ unsigned long long turn_of(double freq) {
    constexpr unsigned long long kTurn1 = 0x28be60db9391054aull, kTurn0 = 0x7f09d5f47d4d3770ull;       // 2^128 / 2pi
    const unsigned long long u = (unsigned long long)__double_as_longlong(freq);
    const int e = (int)(u >> 52) & 2047;
    const unsigned long long m = (u & 0xFFFFFFFFFFFFFull) | (e ? 1ull << 52 : 0ull);       // freq = +-m * 2^(max(e, 1) - 1075)
    const unsigned __int128 x = (unsigned __int128)m * kTurn1 + __umul64hi(m, kTurn0);    // m / 2pi in units of 2^-64
    const int s = 1075 - max(e, 1);
    unsigned long long t = 0;
    if (s >= 0 && s < 128) t = (unsigned long long)(x >> s);
    else if (s < 0 && s > -64) t = (unsigned long long)x << -s;
    return u >> 63 ? 0ull - t : t;
}

template <int D, bool kHalves, bool kAppend>
__global__ void __launch_bounds__(kRopeThreads, 7) attn_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kL = D / 16;     // lanes of a head: 16 elements (two 16-byte chunks) each
    constexpr int kSub = 32 / kL;  // heads that a warp takes side by side
    constexpr int kWarps = kRopeThreads / 32;
    __shared__ unsigned long long turn[D / 2];
    __shared__ int axis[D / 2];
    __shared__ float2 cs[kWarps][D / 2];               // cosine and sine of a warp's token
    __shared__ int cu_s[kAppend ? kCuStage : 1];
    pdl_wait();
    pdl_launch();
    int bad = 0;
    for (int i = threadIdx.x; i < p.pairs; i += kRopeThreads) {
        const double freq = p.freqs[i];
        const int a = p.axes[i];
        turn[i] = turn_of(freq);
        axis[i] = isfinite(freq) ? a : ~a;                 // (an infinite frequency or NaN: the pair becomes NaN)
        bad |= (unsigned)a >= (unsigned)p.num_axes;
    }
    const bool staged = kAppend && p.B < kCuStage;
    if constexpr (kAppend)
        if (staged)
            for (int i = threadIdx.x; i <= p.B; i += kRopeThreads) cu_s[i] = __ldg(p.cu_new + i);
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) report_invalid(ATTN_CACHE_SITE_AXES);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % kL;
    const int h_begin = blockIdx.y * p.heads_per_block + lane / kL;
    const int h_end = min((int)(blockIdx.y + 1) * p.heads_per_block, p.heads);
    // the two chunks of this thread, and the first pair of each
    int ca, cb, pa, pb;
    if constexpr (kHalves) {
        const int rot = p.pairs / 8;
        ca = l < rot ? l : 2 * rot + 2 * (l - rot);
        cb = l < rot ? l + rot : ca + 1;
        pa = l < rot ? 8 * l : p.pairs;
        pb = pa + 4;
    } else {
        ca = l;
        cb = l + kL;
        pa = 4 * ca;
        pb = 4 * cb;
    }
    // which tensor head h of the token belongs to, and its number there
    auto tensor_of = [&](int& h) {
        int t = 0;
        if (h >= p.x[0].heads) { h -= p.x[0].heads; t = 1; }
        if (kAppend && t == 1 && h >= p.x[1].heads) { h -= p.x[1].heads; t = 2; }
        return t;
    };
    // a token a warp
#pragma unroll 1
    for (long long token = (long long)blockIdx.x * kWarps + warp; token < p.tokens; token += (long long)gridDim.x * kWarps) {
        const long long b = kAppend ? 0 : token / p.S, s = kAppend ? token : token - b * p.S;
        struct Heads { uint4 a[kRopeHeads], b[kRopeHeads]; };
        auto load = [&](int h0, Heads& x) {
#pragma unroll
            for (int u = 0; u < kRopeHeads; ++u) {
                int h = h0 + u * kSub;
                if (h >= h_end) continue;
                const RopeTensor& t = p.x[tensor_of(h)];
                const char* src = t.src + b * t.src_b + s * t.src_t + h * t.src_h;
                x.a[u] = *reinterpret_cast<const uint4*>(src + ca * 16);
                x.b[u] = *reinterpret_cast<const uint4*>(src + cb * 16);
            }
        };
        Heads x, next;
        long long row = -1;        // the token's row of the cache
        if constexpr (kAppend) {
            const int* cu = staged ? cu_s : p.cu_new;
            // the last sequence that starts at or before the token (a later one, empty, may start there too)
            int lo = 0, hi = p.B;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= token) lo = mid; else hi = mid - 1;
            }
            if (lo >= p.B || cu[lo] > token) continue;     // in front of the first sequence or behind the last
            load(h_begin, x);
            const int end = cu[lo + 1];
            const long long len = __ldg(p.seqlens_k + lo), first = len - ((long long)end - cu[lo]);
            const long long at = len - end + token;        // its slot in the sequence
            if (first >= 0 && at >= 0 && at < len && len <= (long long)p.pages.max_pages * p.pages.page_size)
                row = page_row(p.pages, p.pages.table + (long long)lo * p.pages.max_pages, (int)at);
            if (row < 0 && lane == 0) report_invalid(ATTN_CACHE_SITE_APPEND);
        } else {
            load(h_begin, x);
        }

        __syncwarp();              // (the token before is done with cs)
#pragma unroll 1
        for (int pr = lane; pr < p.pairs; pr += 32) {
            const int a = axis[pr];
            const long long pos = __ldg(p.positions + (a < 0 ? ~a : a) * p.pos_axis + b * p.pos_b + s);
            const long long at = (long long)(turn[pr] * (unsigned long long)pos);
            float sn, c;
            sincospif(a < 0 ? NAN : (float)at * 0x1p-63f, &sn, &c);
            cs[warp][pr] = make_float2(c, p.inverse ? -sn : sn);
        }
        __syncwarp();
        float c[8], sn[8];
        bool turned[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int pr = e < 4 ? pa + e : pb + e - 4;
            turned[e] = pr < p.pairs;
            const float2 v = turned[e] ? cs[warp][pr] : make_float2(1.0f, 0.0f);
            c[e] = v.x;
            sn[e] = v.y;
        }
#pragma unroll 1
        for (int h0 = h_begin; h0 < h_end; h0 += kRopeHeads * kSub) {
            load(h0 + kRopeHeads * kSub, next);
#pragma unroll
            for (int u = 0; u < kRopeHeads; ++u) {
                int h = h0 + u * kSub;
                if (h >= h_end) continue;
                const int t = tensor_of(h);
                if (kAppend && t > 0 && row < 0) continue;
                if (!kAppend || t < 2) {
                    uint32_t wa[4] = {x.a[u].x, x.a[u].y, x.a[u].z, x.a[u].w}, wb[4] = {x.b[u].x, x.b[u].y, x.b[u].z, x.b[u].w};
                    if constexpr (kHalves) {
                        if (turned[0]) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                // elements 2i and 2i + 1 of both chunks
                                const float a0 = __uint_as_float(wa[i] << 16), a1 = __uint_as_float(wa[i] & 0xFFFF0000u);
                                const float b0 = __uint_as_float(wb[i] << 16), b1 = __uint_as_float(wb[i] & 0xFFFF0000u);
                                wa[i] = ptx::pack_bf16x2(a0 * c[2 * i] - b0 * sn[2 * i],
                                                         a1 * c[2 * i + 1] - b1 * sn[2 * i + 1]);
                                wb[i] = ptx::pack_bf16x2(b0 * c[2 * i] + a0 * sn[2 * i],
                                                         b1 * c[2 * i + 1] + a1 * sn[2 * i + 1]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (turned[i]) wa[i] = rotate_word(wa[i], c[i], sn[i]);
                            if (turned[4 + i]) wb[i] = rotate_word(wb[i], c[4 + i], sn[4 + i]);
                        }
                    }
                    x.a[u] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
                    x.b[u] = make_uint4(wb[0], wb[1], wb[2], wb[3]);
                }
                const RopeTensor& to = p.x[t];
                char* dst = to.dst + b * to.dst_b + (kAppend && t > 0 ? row : s) * to.dst_t + h * to.dst_h;
                *reinterpret_cast<uint4*>(dst + ca * 16) = x.a[u];
                *reinterpret_cast<uint4*>(dst + cb * 16) = x.b[u];
            }
            x = next;
        }
    }
}

}  // namespace cache
