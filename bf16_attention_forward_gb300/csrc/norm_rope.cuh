// norm_rope.cuh -- norms of queries and keys for each head, with their rotary positions in the same pass; the
// gradient; and the form that writes the keys to a paged cache.
//
// Mathematics.  Of a head x of d elements, with weights w:
//   r = 1 / sqrt(sum x_i^2 / d + eps),  n = r x,  y = R(n * w),
// R the rotation of rope.cuh (pair p by pos[axis[p]] * freq[p]).  Of the gradient dy, with g = R^T dy:
//   dw = sum over heads and tokens of g * n,  dx = r (g * w - n (sum (g * w)_i n_i) / d).
// All of it in fp32, y and dx rounded once.  (The squares' sum is fp32 too: elements past 10^18 may overflow it, then r is 0 and
// so are n, y and dx.  Squares that underflow are taken of 2^80 x.)
//
// Bound: HBM bytes; x read and y written once (backward: x and dy read, dx written).  A warp takes a token, whose angles it
// computes once; D / 16 lanes take a head, 16 elements each (two 16-byte chunks, so that a pair's elements meet in one thread),
// and the sums over a head are 2 or 3 shuffles.  Weights stand in shared memory as fp32; the forward multiplies them into
// the cosines and sines once a token.
#pragma once
#include <type_traits>

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
    float* part;                   // [2][blocks][D] sums of q's and k's dw
    float* dw[2];                  // [d] or null
    int blocks;
};

constexpr int kNormThreads = 128;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kNormBwdBlocks = 4;  // of the gradient's kernel an SM: one wave, since each block leaves sums to be added up

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
    // cosines and sines of a token's pairs, by the lanes of a warp: positions first (they wait for memory)
    __device__ __forceinline__ void angles(const NormRopeParams& p, int b, int s, float2* cs) const {
        constexpr int kPairs = (D / 2 + 31) / 32;          // of a lane
        int pos[kPairs];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int pr = (threadIdx.x & 31) + 32 * i;
            pos[i] = 0;
            if (pr < p.pairs) {
                const int a = axis[pr];
                pos[i] = __ldg(p.positions + (a < 0 ? ~a : a) * p.pos_axis + b * p.pos_b + s);
            }
        }
        __syncwarp();                                      // (the token before is done with cs)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int pr = (threadIdx.x & 31) + 32 * i;
            if (pr >= p.pairs) break;
            const long long at = (long long)(turn[pr] * (unsigned long long)(long long)pos[i]);
            float sn, c;
            sincospif(axis[pr] < 0 ? NAN : (float)at * 0x1p-63f, &sn, &c);
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
    // which of the thread's 8 pairs turn, a bit each
    __device__ __forceinline__ uint32_t turning(int pairs) const {
        uint32_t turns = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) turns |= (uint32_t)((e < 4 ? pa + e : pb + e - 4) < pairs) << e;
        return turns;
    }
    // their cosines and sines (1 and 0 where they do not turn: see still())
    __device__ __forceinline__ void take(const float2* cs, float (&c)[8], float (&sn)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float4 v = *reinterpret_cast<const float4*>(cs + (e < 4 ? pa + e : pb + e - 4));
            c[e] = v.x; sn[e] = v.y;
            c[e + 1] = v.z; sn[e + 1] = v.w;
        }
    }
    // a warp's cosines and sines of pairs that do not turn; behind the last pair halves read 8 more
    static constexpr int kAngles = D / 2 + 8;
    static __device__ __forceinline__ void still(float2* cs, int pairs) {
        for (int i = pairs + (threadIdx.x & 31); i < kAngles; i += 32) cs[i] = make_float2(1.0f, 0.0f);
        __syncwarp();
    }
    // Of weights, cosines and sines the factors of a word: y = x * A + (its partners) * B.  Adjacent: a word is a pair and its
    // partners its own elements, swapped; halves: the word of the other chunk.
    static __device__ __forceinline__ void factors(const float2 (&w)[8], const float (&c)[8], const float (&sn)[8], float2 (&A)[8],
                                                   float2 (&B)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (kHalves) {
                const int e = 2 * (i & 3);
                const float2 cc = make_float2(c[e], c[e + 1]), ss = make_float2(sn[e], sn[e + 1]);
                A[i] = __fmul2_rn(w[i], cc);
                B[i] = __fmul2_rn(w[i ^ 4], i < 4 ? make_float2(-ss.x, -ss.y) : ss);
            } else {
                A[i] = __fmul2_rn(w[i], make_float2(c[i], c[i]));
                B[i] = __fmul2_rn(make_float2(w[i].y, w[i].x), make_float2(-sn[i], sn[i]));
            }
        }
    }
    static __device__ __forceinline__ float2 partners(const float2 (&x)[8], int i) {
        return kHalves ? x[i ^ 4] : make_float2(x[i].y, x[i].x);
    }
    // whether word i turns (a pair that does not is left alone: a NaN in one of its elements stays there)
    static __device__ __forceinline__ bool turned(uint32_t turns, int i) { return kHalves ? turns != 0 : turns >> i & 1u; }
    // the thread's elements, two by two (chunk a in x[0..3], chunk b in x[4..7]), turned by the angles, or by their negatives (a
    // pair that does not turn is left alone: a NaN in one of its elements stays there)
    template <bool kBack>
    static __device__ __forceinline__ void turn(float2 (&x)[8], const float (&c)[8], const float (&sn)[8], uint32_t turns) {
        if (turns == 0) return;
        if constexpr (kHalves) {           // (all 8 or none)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 cc = make_float2(c[2 * e], c[2 * e + 1]), v = make_float2(sn[2 * e], sn[2 * e + 1]);
                const float2 s = kBack ? make_float2(-v.x, -v.y) : v, m = make_float2(-s.x, -s.y), x0 = x[e], x1 = x[e + 4];
                x[e] = __ffma2_rn(x0, cc, __fmul2_rn(x1, m));
                x[e + 4] = __ffma2_rn(x1, cc, __fmul2_rn(x0, s));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!(turns >> e & 1u)) continue;
                const float s = kBack ? -sn[e] : sn[e];
                const float2 v = x[e];
                x[e] = make_float2(v.x * c[e] - v.y * s, v.y * c[e] + v.x * s);
            }
        }
    }
};

__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float2 (&x)[8]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void pack16(const float2 (&x)[8], uint4& a, uint4& b) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = ptx::pack_bf16x2(x[i].x, x[i].y);
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}
// a head's weights of the thread's two chunks
__device__ __forceinline__ void weights16(const float* w, int ca, int cb, float2 (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(w + (i < 2 ? ca : cb) * 8 + (i & 1) * 4);
        x[2 * i] = make_float2(v.x, v.y);
        x[2 * i + 1] = make_float2(v.z, v.w);
    }
}
__device__ __forceinline__ float weight_at(const NormRopeParams& p, int t, int i) {
    if (!p.weight[t]) return 1.0f;
    return p.weight_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.weight[t])[i])
                         : reinterpret_cast<const float*>(p.weight[t])[i];
}
// sum of a thread's products over the lanes of a head
template <int kL>
__device__ __forceinline__ float head_dot(const float2 (&x)[8], const float2 (&y)[8]) {
    float2 s = __fmul2_rn(x[0], y[0]), t = __fmul2_rn(x[1], y[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        s = __ffma2_rn(x[i], y[i], s);
        t = __ffma2_rn(x[i + 1], y[i + 1], t);
    }
    s = __fadd2_rn(s, t);
    float v = s.x + s.y;
#pragma unroll
    for (int off = 1; off < kL; off <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}
// r of a head.  kSmall: where the mean and eps are below 2^-80, the squares may have underflowed: x comes back times `up` = 2^80 (else 1),
// and so does 1 / r, whose squares then lie between 2^-106 and 2^94.  there: whether the head is one (others' numbers count for nothing).
// Looked for only where eps allows such heads: the vote keeps the heads of a step from running side by side (32,760 tokens of 24
// heads: 65.7 us, without 63.8).
constexpr float kNormSmall = 0x1p-80f;
template <int D, bool kSmall>
__device__ __forceinline__ float head_root(float2 (&x)[8], float eps, bool there, float& up) {
    float mean = head_dot<D / 16>(x, x) * (1.0f / D) + eps;
    up = 1.0f;
    if (kSmall && __any_sync(0xFFFFFFFFu, there && mean < kNormSmall)) {
        up = mean < kNormSmall ? 0x1p80f : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], make_float2(up, up));
        mean = head_dot<D / 16>(x, x) * (1.0f / D) + eps * up * up;
    }
    return rsqrtf(mean);
}
// 16 bytes global -> shared
__device__ __forceinline__ void cp_async16_plain(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A token, and where it is in its batch entry; the next one of a warp lies `tokens` on.  (The host refuses 2^30 of them.)
struct NormToken {
    int token, b, s;
};
struct NormStride {
    int tokens, b, s, S;
    __device__ __forceinline__ explicit NormStride(const NormRopeParams& p)
        : tokens(gridDim.x * kNormWarps), b((int)(tokens / p.S)), s((int)(tokens - b * p.S)), S((int)p.S) {}
    __device__ __forceinline__ NormToken first() const {
        const int t = blockIdx.x * kNormWarps + (threadIdx.x >> 5);
        return {t, t / S, t % S};
    }
    __device__ __forceinline__ void next(NormToken& t) const {
        t.token += tokens;
        t.b += b;
        t.s += s;
        if (t.s >= S) { t.s -= S; ++t.b; }
    }
};

// Each thread copies its own 16-byte chunks into shared memory two steps ahead and reads only those back: nothing but its own
// wait_group stands between.  At HBM's rate the SMs have 350 instructions for a warp's kSub heads, so the loop is kept
// short: weights, cosines and sines multiplied once a token, two products an instruction, addresses by addition.
// 32,760 tokens of 24 heads (403 MB): 63.6 us, 95 % of a copy; with the next heads in registers 72, with more steps ahead or more
// blocks 64 to 75 (more rows of the memory are open then).
constexpr int kNormStages = 3;
constexpr int kNormHeads = 2;      // of a thread at a time
constexpr int kNormBlocks = 4;     // an SM, one wave: a block's tables and weights take as long as some tokens
template <int D, bool kHalves, bool kAppend>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks) attn_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int kL = D / 16;     // lanes of a head
    constexpr int kSub = 32 / kL;  // heads that a warp takes side by side
    constexpr int kTensors = kAppend ? 3 : 2;
    __shared__ TurnTable<D> table;
    __shared__ __align__(16) float w_s[2][D];
    __shared__ __align__(16) float2 cs[kNormWarps][Place<D, kHalves>::kAngles];
    __shared__ uint4 ring[kNormStages][2 * kNormHeads][kNormThreads];
    pdl_wait();
    pdl_launch();
    for (int i = threadIdx.x; i < 2 * D; i += kNormThreads) w_s[i / D][i % D] = weight_at(p, i / D, i % D);
    if (table.fill(p)) {
        if (threadIdx.x == 0) report_invalid(ATTN_CACHE_SITE_AXES);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / kL;
    const Place<D, kHalves> place(lane % kL, p.pairs);
    const uint32_t ring_at = ptx::smem_u32(&ring[0][0][threadIdx.x]);
    // this block's heads of tensor t
    const int block_h = blockIdx.y * p.heads_per_block;
    auto first_head = [&](int t) { return max(block_h - (t > 0 ? p.x[0].heads : 0) - (t > 1 ? p.x[1].heads : 0), 0); };
    auto last_head = [&](int t) {
        return min(block_h + p.heads_per_block - (t > 0 ? p.x[0].heads : 0) - (t > 1 ? p.x[1].heads : 0), p.x[t].heads);
    };
    place.still(cs[warp], p.pairs);
    const uint32_t turns = place.turning(p.pairs);
    const bool all_turn = __all_sync(0xFFFFFFFFu, turns == 0xFFu);
    // the loads ahead: tensor, heads left of it, where the next ones are
    const NormStride stride(p);
    NormToken at = stride.first(), ahead = at;
    const int tokens = (int)p.tokens;
    int ta = -1, left = 0;
    const char* from = nullptr;
    auto slot_of = [&](int token) {
        return token < tokens ? __ldg(reinterpret_cast<const long long*>(p.slots) + token) : 0;
    };
    // appending: the slots of the token ahead and of the next one (a token without a slot is passed over)
    long long slot = kAppend ? slot_of(ahead.token) : 0, next_slot = kAppend ? slot_of(ahead.token + stride.tokens) : 0;
    auto pass = [&]() {
        stride.next(ahead);
        slot = next_slot;
        if (kAppend) next_slot = slot_of(ahead.token + stride.tokens);
    };
    auto load = [&](int stage) {
        while (left <= 0 && ahead.token < tokens) {
            if (kAppend && slot == -1) {
                pass();
                continue;
            }
            if (++ta == kTensors) {
                ta = -1;
                pass();
                continue;
            }
            const int h = first_head(ta);
            left = last_head(ta) - h;
            from = p.x[ta].src + (long long)ahead.b * p.x[ta].src_b + (long long)ahead.s * p.x[ta].src_t + (h + sub) * p.x[ta].src_h;
        }
#pragma unroll
        for (int u = 0; u < kNormHeads; ++u) {
            if (left > sub) {
                cp_async16_plain(ring_at + ((stage * kNormHeads + u) * 2) * (kNormThreads * 16), from + place.ca * 16);
                cp_async16_plain(ring_at + ((stage * kNormHeads + u) * 2 + 1) * (kNormThreads * 16), from + place.cb * 16);
            }
            if (left > 0) from += kSub * p.x[ta].src_h;
            left -= kSub;
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kNormStages - 1; ++i) load(i);
    int stage = 0;
#pragma unroll 1
    for (; at.token < tokens; stride.next(at)) {
        long long row = -1;        // the token's row of the cache
        if constexpr (kAppend) {
            row = slot_of(at.token);
            if (row == -1) continue;
            if (row < 0 || row >= p.rows) {
                row = -1;
                if (lane == 0) report_invalid(ATTN_CACHE_SITE_SLOTS);
            }
        }
        table.angles(p, at.b, at.s, cs[warp]);
#pragma unroll 1
        for (int t = 0; t < kTensors; ++t) {
            const int h0 = first_head(t), h1 = last_head(t);
            if (h0 >= h1) continue;
            const bool out = !(kAppend && t > 0 && row < 0);
            char* dst = p.x[t].dst + (long long)at.b * p.x[t].dst_b + (kAppend && t > 0 ? row : (long long)at.s) * p.x[t].dst_t + (h0 + sub) * p.x[t].dst_h;
            const long long step = kSub * p.x[t].dst_h;
            float2 A[8], B[8];
            if (!kAppend || t < 2) {
                float2 w[8];
                float c[8], sn[8];
                weights16(w_s[t & 1], place.ca, place.cb, w);
                place.take(cs[warp], c, sn);
                place.factors(w, c, sn, A, B);
            }
            auto heads = [&](auto all, auto small) {       // all: every word of the warp turns; small: see head_root
#pragma unroll 1
                for (int h = h0 + sub; h - sub < h1; h += kNormHeads * kSub) {
                    cp_async_wait<kNormStages - 2>();
                    uint4 xa[kNormHeads], xb[kNormHeads];
#pragma unroll
                    for (int u = 0; u < kNormHeads; ++u) {
                        xa[u] = ring[stage][2 * u][threadIdx.x];
                        xb[u] = ring[stage][2 * u + 1][threadIdx.x];
                    }
                    load(stage == 0 ? kNormStages - 1 : stage - 1);        // (the stage read in the step before)
                    stage = stage + 1 == kNormStages ? 0 : stage + 1;
#pragma unroll
                    for (int u = 0; u < kNormHeads; ++u) {
                        if (!kAppend || t < 2) {
                            float2 x[8], y[8];
                            unpack16(xa[u], xb[u], x);
                            float up;
                            const float r = head_root<D, small.value>(x, p.eps, h + u * kSub < h1, up);
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], both(r));      // (before the factors, which may be large)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                y[i] = __fmul2_rn(x[i], A[i]);
                                if (all.value || place.turned(turns, i)) y[i] = __ffma2_rn(place.partners(x, i), B[i], y[i]);
                            }
                            pack16(y, xa[u], xb[u]);
                        }
                        if (out && h + u * kSub < h1) {
                            *reinterpret_cast<uint4*>(dst + place.ca * 16) = xa[u];
                            *reinterpret_cast<uint4*>(dst + place.cb * 16) = xb[u];
                        }
                        dst += step;
                    }
                }
            };
            if (p.eps < kNormSmall) heads(std::false_type(), std::true_type());
            else if (all_turn) heads(std::true_type(), std::false_type());
            else heads(std::false_type(), std::false_type());
        }
    }
    cp_async_wait<0>();
}

// The gradient.  A warp takes a token's q heads, then its k heads; a thread sums its 16 elements of q's dw over all of its heads
// in registers, of k's in shared memory, a block adds up its threads' in a fixed order, and attn_norm_rope_dw_kernel the blocks'.
// 16,384 tokens of 40 heads (503 MB): 83 us both kernels, 91 % of a copy's rate; q and k in blocks of their own took 93 (a token's
// angles, which wait for its position, take as long as some heads' steps), the next head in registers 105.
constexpr int kNormBwdStages = 3;
template <int D, bool kHalves>
__global__ void __launch_bounds__(kNormThreads, kNormBwdBlocks) attn_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int kL = D / 16, kSub = 32 / kL;
    __shared__ TurnTable<D> table;
    __shared__ __align__(16) float w_s[2][D];
    __shared__ __align__(16) float2 cs[kNormWarps][Place<D, kHalves>::kAngles];
    __shared__ uint4 ring[kNormBwdStages][4][kNormThreads];
    __shared__ float4 dk_s[4][kNormThreads];           // a thread's sums of k's dw
    float(*sum_s)[D] = reinterpret_cast<float(*)[D]>(ring);        // (at the end)
    pdl_wait();
    pdl_launch();
    for (int i = threadIdx.x; i < 2 * D; i += kNormThreads) w_s[i / D][i % D] = weight_at(p, i / D, i % D);
#pragma unroll
    for (int i = 0; i < 4; ++i) dk_s[i][threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (table.fill(p)) {
        if (threadIdx.x == 0) report_invalid(ATTN_CACHE_SITE_AXES);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / kL;
    const Place<D, kHalves> place(lane % kL, p.pairs);
    const NormStride stride(p);
    NormToken at = stride.first(), ahead = at;
    const int tokens = (int)p.tokens;
    const uint32_t ring_at = ptx::smem_u32(&ring[0][0][threadIdx.x]);
    place.still(cs[warp], p.pairs);
    const uint32_t turns = place.turning(p.pairs);
    // the loads ahead: tensor, heads left of it, where the next ones are
    int ta = -1, left = 0;
    const char *from_x = nullptr, *from_g = nullptr;
    auto load = [&](int stage) {
        while (left <= 0 && ahead.token < tokens) {
            if (++ta == 2) {
                ta = -1;
                stride.next(ahead);
                continue;
            }
            left = p.x[ta].heads;
            from_x = p.x[ta].src + (long long)ahead.b * p.x[ta].src_b + (long long)ahead.s * p.x[ta].src_t + sub * p.x[ta].src_h;
            from_g = p.dy[ta].src + (long long)ahead.b * p.dy[ta].src_b + (long long)ahead.s * p.dy[ta].src_t + sub * p.dy[ta].src_h;
        }
        if (left > sub) {
            const uint32_t to = ring_at + stage * (4 * kNormThreads * 16);
            cp_async16_plain(to, from_x + place.ca * 16);
            cp_async16_plain(to + kNormThreads * 16, from_x + place.cb * 16);
            cp_async16_plain(to + 2 * kNormThreads * 16, from_g + place.ca * 16);
            cp_async16_plain(to + 3 * kNormThreads * 16, from_g + place.cb * 16);
        }
        if (left > 0) {
            from_x += kSub * p.x[ta].src_h;
            from_g += kSub * p.dy[ta].src_h;
        }
        left -= kSub;
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kNormBwdStages - 1; ++i) load(i);
    float2 dq[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dq[e] = make_float2(0.0f, 0.0f);
    int stage = 0;
#pragma unroll 1
    for (; at.token < tokens; stride.next(at)) {
        table.angles(p, at.b, at.s, cs[warp]);
        float c[8], sn[8];
        place.take(cs[warp], c, sn);
        auto tensor = [&](int t, float2 (&dw)[8], auto small) {
            char* dst = p.x[t].dst + (long long)at.b * p.x[t].dst_b + (long long)at.s * p.x[t].dst_t + sub * p.x[t].dst_h;
            const long long step = kSub * p.x[t].dst_h;
            const int heads = p.x[t].heads;
#pragma unroll 1
            for (int h = sub; h - sub < heads; h += kSub) {
                cp_async_wait<kNormBwdStages - 2>();
                float2 x[8], g[8], w[8];
                unpack16(ring[stage][0][threadIdx.x], ring[stage][1][threadIdx.x], x);
                unpack16(ring[stage][2][threadIdx.x], ring[stage][3][threadIdx.x], g);
                load(stage == 0 ? kNormBwdStages - 1 : stage - 1);     // (the stage read in the step before)
                place.template turn<true>(g, c, sn, turns);
                const bool there = h < heads;                          // (what an absent head's place holds is another's)
                float up;
                const float r = head_root<D, small.value>(x, p.eps, there, up);
                weights16(w_s[t], place.ca, place.cb, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = __fmul2_rn(x[e], both(r));
                    if (there) dw[e] = __ffma2_rn(g[e], x[e], dw[e]);
                    g[e] = __fmul2_rn(g[e], w[e]);
                }
                const float dot = head_dot<kL>(g, x) * (1.0f / D);
                if (there) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = __fmul2_rn(__ffma2_rn(x[e], both(-dot), g[e]), both(r));
                    if (small.value && up != 1.0f)
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[e] = __fmul2_rn(g[e], both(up));
                    uint4 oa, ob;
                    pack16(g, oa, ob);
                    *reinterpret_cast<uint4*>(dst + place.ca * 16) = oa;
                    *reinterpret_cast<uint4*>(dst + place.cb * 16) = ob;
                }
                dst += step;
                stage = stage + 1 == kNormBwdStages ? 0 : stage + 1;
            }
        };
        const bool small = p.eps < kNormSmall;
        if (small) tensor(0, dq, std::true_type());
        else tensor(0, dq, std::false_type());
        if (p.x[1].heads > 0) {
            float2 dk[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) dk[e] = make_float2(0.0f, 0.0f);
            if (small) tensor(1, dk, std::true_type());
            else tensor(1, dk, std::false_type());
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4 v = dk_s[i][threadIdx.x];
                v.x += dk[2 * i].x; v.y += dk[2 * i].y; v.z += dk[2 * i + 1].x; v.w += dk[2 * i + 1].y;
                dk_s[i][threadIdx.x] = v;
            }
        }
    }
    cp_async_wait<0>();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float4 k = dk_s[e >> 2][threadIdx.x];
            float v = t ? ((e & 3) == 0 ? k.x : (e & 3) == 1 ? k.y : (e & 3) == 2 ? k.z : k.w) : e & 1 ? dq[e / 2].y : dq[e / 2].x;
#pragma unroll
            for (int off = kL; off < 32; off <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
            if (lane < kL) sum_s[warp][(e < 8 ? place.ca : place.cb) * 8 + (e & 7)] = v;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < D; i += kNormThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kNormWarps; ++w) v += sum_s[w][i];
            p.part[((long long)t * gridDim.x + blockIdx.x) * D + i] = v;
        }
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
    const float* part = p.part + (long long)t * p.blocks * D + col;
    float v = 0.0f;
#pragma unroll 8
    for (int i = y; i < p.blocks; i += kDwRows) v += part[(long long)i * D];
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
