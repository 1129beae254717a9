// attn_cache.cu -- host side of the calls around the paged K/V cache: rotary positions (rope.cuh),
// appending (rope.cuh), attention of one new token (decode.cuh) and eviction (evict.cuh).
#include <cuda_runtime.h>
#include <string.h>

#include <cmath>
#include <mutex>
#include <type_traits>

#include "cache_common.cuh"
#include "decode.cuh"
#include "evict.cuh"
#include "rope.cuh"

namespace {
using namespace cache;

constexpr int kMaxDevices = 64;
constexpr int64_t kLim = (int64_t)1 << 30;      // sizes: row and slot indices are int32
struct Device {
    bool init = false;
    int sms = 0, major = 0, minor = 0;
};
std::mutex g_mutex;
Device g_dev[kMaxDevices];

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

template <int D, int NH>
cudaError_t set_decode_attr() {
    cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<D, NH, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         DecGeo<D>::kSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attn_decode_kernel<D, NH, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 DecGeo<D>::kSmem);
    return e;
}

int device(int* sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return ATTN_ERR_NO_DEVICE; }
    if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_NO_DEVICE;
    std::lock_guard<std::mutex> g(g_mutex);
    Device& d = g_dev[dev];
    if (!d.init) {
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
            cudaGetLastError();
            return ATTN_ERR_NO_DEVICE;
        }
        if (d.major == 10 && d.minor == 3 &&
            (set_decode_attr<128, 1>() != cudaSuccess || set_decode_attr<128, 2>() != cudaSuccess ||
             set_decode_attr<128, 4>() != cudaSuccess || set_decode_attr<64, 1>() != cudaSuccess ||
             set_decode_attr<64, 2>() != cudaSuccess || set_decode_attr<64, 4>() != cudaSuccess)) {
            cudaGetLastError();
            return ATTN_ERR_CUDA;
        }
        d.init = true;
    }
    if (d.major != 10 || d.minor != 3) return ATTN_ERR_NO_DEVICE;
    *sms = d.sms;
    return ATTN_OK;
}

// Each kernel is launched as the programmatic dependent of the one before it in the stream, waits for that one before
// it touches global memory and before it ends, and only then lets the next one start.  One reads earlier: eviction's
// select kernel reads lengths and weights while the prepare kernel runs, which only reads them too; what ran before that
// is complete by then, because the prepare kernel's CTAs let select start behind their own wait.
// cluster: CTAs of a cluster.
template <class P>
int launch_clusters(void (*kernel)(P), int64_t grid, int cluster, int threads, size_t smem, cudaStream_t stream,
                    const std::remove_const_t<P>& args, int grid_y = 1) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)grid, (unsigned)grid_y);
    lc.blockDim = dim3((unsigned)threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    lc.attrs = at;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&lc, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return ATTN_OK;
}
template <class P>
int launch(void (*kernel)(P), int64_t grid, int grid_y, int threads, size_t smem, cudaStream_t stream,
           const std::remove_const_t<P>& args) {
    return launch_clusters(kernel, grid, 1, threads, smem, stream, args, grid_y);
}

// ------------------------------------------------------------------------------ memory ranges
// A strided bf16 tensor [n0][n1][n2][d] (elements).
struct View {
    uintptr_t at;
    int64_t n[3], st[3], d;
    int64_t span() const {       // elements from the first to behind the last; 0 when empty
        int64_t s = d;
        for (int i = 0; i < 3; ++i) {
            if (n[i] < 1) return 0;
            s += (n[i] - 1) * st[i];
        }
        return s;
    }
    uintptr_t end() const { return at + 2 * (uintptr_t)span(); }
};

View view(const void* p, int64_t n0, int64_t n1, int64_t n2, int64_t d, int64_t s0, int64_t s1, int64_t s2) {
    View v;
    v.at = (uintptr_t)p;
    v.n[0] = n0; v.n[1] = n1; v.n[2] = n2;
    v.st[0] = s0; v.st[1] = s1; v.st[2] = s2;
    v.d = d;
    return v;
}

bool same(const View& a, const View& b) {
    if (a.at != b.at) return false;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.st[i] != b.st[i])) return false;
    return true;
}

bool overlap(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) { return a0 < b1 && b0 < a1; }

// Two views as sums of multiples of common strides, largest first: 0 .. n - 1 times each, and an extent behind the
// last (an extent of one entry, or of stride zero, adds nothing; two of one stride add up).
struct Lattice {
    int levels = 0;
    int64_t st[6], n[2][6], d[2];
    void add(int64_t stride) {
        int i = 0;
        while (i < levels && st[i] > stride) ++i;
        if (i < levels && st[i] == stride) return;
        for (int j = levels++; j > i; --j) st[j] = st[j - 1];
        st[i] = stride;
    }
    int64_t width(int v, int level) const {        // of what the levels from `level` on span
        int64_t w = d[v];
        for (int i = level; i < levels; ++i) w += (n[v][i] - 1) * st[i];
        return w;
    }
    // whether the two share an element from `level` on, the second `diff` elements behind the first: the multiples
    // i of the first and j of the second leave diff - (i - j) * st for the levels behind, so only i - j for which
    // those still reach each other count: three at most where extents nest (more: taken to meet)
    bool meet(int level, int64_t diff) const {
        const int64_t wa = width(0, level), wb = width(1, level);
        if (diff >= wa || -diff >= wb) return false;
        if (level == levels) return true;
        const int64_t t = st[level], ra = width(0, level + 1), rb = width(1, level + 1);
        auto floor_div = [&](int64_t x) { return x / t - (x % t < 0); };
        int64_t k0 = floor_div(diff - ra) + 1, k1 = -floor_div(-(diff + rb)) - 1;
        if (k0 < 1 - n[1][level]) k0 = 1 - n[1][level];
        if (k1 > n[0][level] - 1) k1 = n[0][level] - 1;
        if (k1 - k0 > 3) return true;
        for (int64_t k = k0; k <= k1; ++k)
            if (meet(level + 1, diff - k * t)) return true;
        return false;
    }
};

// whether two views share an element: slices of one buffer, side by side in any of their extents, do not
bool meet(const View& a, const View& b) {
    if (!a.span() || !b.span() || !overlap(a.at, a.end(), b.at, b.end())) return false;
    const View* v[2] = {&a, &b};
    Lattice l;
    for (int x = 0; x < 2; ++x)
        for (int i = 0; i < 3; ++i)
            if (v[x]->n[i] > 1 && v[x]->st[i] > 0) l.add(v[x]->st[i]);
    for (int x = 0; x < 2; ++x) {
        l.d[x] = v[x]->d;
        for (int j = 0; j < l.levels; ++j) {
            l.n[x][j] = 1;
            for (int i = 0; i < 3; ++i)
                if (v[x]->n[i] > 1 && v[x]->st[i] == l.st[j]) l.n[x][j] += v[x]->n[i] - 1;
        }
    }
    return l.meet(0, (int64_t)(b.at - a.at) / 2);
}

// no two elements of a view on one address: its extents nest
bool nested(const View& v) {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (v.st[order[j]] > v.st[order[j + 1]]) { const int t = order[j]; order[j] = order[j + 1]; order[j + 1] = t; }
    int64_t width = v.d;
    for (int i = 0; i < 3; ++i) {
        const int a = order[i];
        if (v.n[a] < 2) continue;
        if (v.st[a] < width) return false;
        width = (v.n[a] - 1) * v.st[a] + width;
    }
    return true;
}

// extents n[i] of strides st[i]: no negative one, and no view of more than 2^40 elements a dimension
bool strides_ok(const int64_t* st, const int64_t* n, int dims) {
    for (int i = 0; i < dims; ++i)
        if (st[i] < 0 || (n[i] > 1 && st[i] > ((int64_t)1 << 40) / (n[i] - 1))) return false;
    return true;
}
bool strides_aligned(const int64_t* st, const int64_t* n, int dims) {
    for (int i = 0; i < dims; ++i)
        if (n[i] > 1 && st[i] % 8 != 0) return false;
    return true;
}

bool head_dim(int64_t d) { return d == 128 || d == 64; }

int check_pairs(int32_t pairs, int32_t num_axes, int32_t pairing, int64_t d) {
    if (pairs < 0 || pairs > d / 2 || num_axes < 1) return ATTN_ERR_INVALID_ARG;
    if (pairing != ATTN_ROPE_ADJACENT && pairing != ATTN_ROPE_HALVES) return ATTN_ERR_INVALID_ARG;
    if (pairing == ATTN_ROPE_HALVES && pairs % 8 != 0) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

int check_cache(int64_t B, int64_t Hkv, int64_t num_pages, int64_t page_size, int64_t max_pages, int64_t d) {
    if (B < 1 || Hkv < 1 || num_pages < 1 || page_size < 1 || max_pages < 1 || d < 1) return ATTN_ERR_INVALID_ARG;
    if (!head_dim(d)) return ATTN_ERR_UNSUPPORTED;
    if (B > kLim || Hkv > kLim || num_pages > kLim || page_size > kLim || max_pages > kLim) return ATTN_ERR_UNSUPPORTED;
    if (num_pages * page_size > kLim || max_pages * page_size > kLim || B * max_pages > kLim || B * Hkv > kLim)
        return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

Pages make_pages(const int32_t* table, int64_t num_pages, int64_t page_size, int64_t max_pages) {
    Pages c;
    c.table = table;
    c.num_pages = (int)num_pages;
    c.page_size = (int)page_size;
    c.max_pages = (int)max_pages;
    uint32_t log2 = 0;
    while (((int64_t)1 << log2) < page_size) ++log2;
    c.shift = 30 + log2;
    c.mul = (uint32_t)(((((uint64_t)1 << c.shift) - 1) / (uint64_t)page_size) + 1);
    return c;
}

// ------------------------------------------------------------------------------ rope, append
RopeTensor rope_tensor(const void* src, void* dst, const int64_t* ss, const int64_t* ds, int64_t heads) {
    RopeTensor t;
    memset(&t, 0, sizeof t);
    t.src = reinterpret_cast<const char*>(src);
    t.dst = reinterpret_cast<char*>(dst);
    t.src_b = 2 * ss[0]; t.src_t = 2 * ss[1]; t.src_h = 2 * ss[2];
    t.dst_b = 2 * ds[0]; t.dst_t = 2 * ds[1]; t.dst_h = 2 * ds[2];
    t.heads = (int)heads;
    return t;
}

int launch_rope(RopeParams& p, int64_t d, bool halves, bool append, int sms, cudaStream_t stream) {
    // Heads of a block: all of its tokens', which computes each angle once, unless that leaves the SMs short
    // of threads (2048 each); then the heads are dealt out evenly, in the pieces that a warp turns at a time.
    const int64_t lanes = p.tokens * 32, full = (int64_t)sms * 2048, piece = kRopeHeads * (32 / (d / 16));
    int64_t splits = lanes < full ? cdiv(full, lanes) : 1;
    if (splits > cdiv(p.heads, piece)) splits = cdiv(p.heads, piece);
    p.heads_per_block = (int)(cdiv(cdiv(p.heads, splits), piece) * piece);
    // 28 blocks an SM at most, 4 waves of the 7 that fit; longer lines give a warp several tokens (32,760 tokens of
    // 24 heads: 63.1 us with a block per 4 tokens, 61.7 so; 16,384 of 40: 51.8 either way)
    const int64_t most = cdiv(p.tokens, kRopeThreads / 32), grid = most < 28 * sms ? most : 28 * sms;
    const int gy = (int)cdiv(p.heads, p.heads_per_block);
    if (gy > 65535) return ATTN_ERR_UNSUPPORTED;
    if (d == 128)
        return append ? (halves ? launch(attn_rope_kernel<128, true, true>, grid, gy, kRopeThreads, 0, stream, p)
                                : launch(attn_rope_kernel<128, false, true>, grid, gy, kRopeThreads, 0, stream, p))
                      : (halves ? launch(attn_rope_kernel<128, true, false>, grid, gy, kRopeThreads, 0, stream, p)
                                : launch(attn_rope_kernel<128, false, false>, grid, gy, kRopeThreads, 0, stream, p));
    return append ? (halves ? launch(attn_rope_kernel<64, true, true>, grid, gy, kRopeThreads, 0, stream, p)
                            : launch(attn_rope_kernel<64, false, true>, grid, gy, kRopeThreads, 0, stream, p))
                  : (halves ? launch(attn_rope_kernel<64, true, false>, grid, gy, kRopeThreads, 0, stream, p)
                            : launch(attn_rope_kernel<64, false, false>, grid, gy, kRopeThreads, 0, stream, p));
}

int run_rope(const attn_rope_args_t& a, cudaStream_t stream) {
    const int64_t Hkv = a.k ? a.Hkv : 0;
    if (!a.q || !a.q_out || (a.k && !a.k_out) || !a.positions || !a.freqs || !a.axes) return ATTN_ERR_INVALID_ARG;
    if (a.B < 1 || a.S < 0 || a.H < 1 || (a.k && Hkv < 1) || a.pairs < 1) return ATTN_ERR_INVALID_ARG;
    if (a.inverse != 0 && a.inverse != 1) return ATTN_ERR_INVALID_ARG;
    int st = check_pairs(a.pairs, a.num_axes, a.pairing, head_dim(a.d) ? a.d : 128);
    if (st != ATTN_OK) return st;
    if (!head_dim(a.d)) return ATTN_ERR_UNSUPPORTED;
    if (a.B > kLim || a.S > kLim || a.H > kLim || Hkv > kLim || a.B * a.S > kLim || a.H + Hkv > kLim)
        return ATTN_ERR_UNSUPPORTED;
    const int64_t nq[3] = {a.B, a.S, a.H}, nk[3] = {a.B, a.S, Hkv};
    const int64_t np[2] = {a.num_axes, a.B}, ps[2] = {a.pos_axis_stride, a.pos_batch_stride};
    if (!strides_ok(a.q_stride, nq, 3) || !strides_ok(a.q_out_stride, nq, 3) || !strides_ok(ps, np, 2)) return ATTN_ERR_INVALID_ARG;
    if (a.k && (!strides_ok(a.k_stride, nk, 3) || !strides_ok(a.k_out_stride, nk, 3))) return ATTN_ERR_INVALID_ARG;
    if (((uintptr_t)a.q | (uintptr_t)a.q_out | (uintptr_t)a.k | (a.k ? (uintptr_t)a.k_out : 0)) & 15u)
        return ATTN_ERR_MISALIGNED;
    if (((uintptr_t)a.positions | (uintptr_t)a.axes) & 3u || (uintptr_t)a.freqs & 7u) return ATTN_ERR_MISALIGNED;
    if (!strides_aligned(a.q_stride, nq, 3) || !strides_aligned(a.q_out_stride, nq, 3)) return ATTN_ERR_MISALIGNED;
    if (a.k && (!strides_aligned(a.k_stride, nk, 3) || !strides_aligned(a.k_out_stride, nk, 3))) return ATTN_ERR_MISALIGNED;
    auto v = [&](const void* p, int64_t H, const int64_t* s) { return view(p, a.B, a.S, H, a.d, s[0], s[1], s[2]); };
    const View q = v(a.q, a.H, a.q_stride), qo = v(a.q_out, a.H, a.q_out_stride);
    if (!nested(qo) || (!same(q, qo) && meet(q, qo))) return ATTN_ERR_ALIAS;
    if (a.k) {
        const View k = v(a.k, Hkv, a.k_stride), ko = v(a.k_out, Hkv, a.k_out_stride);
        if (!nested(ko) || (!same(k, ko) && meet(k, ko)) || meet(qo, ko) || meet(qo, k) || meet(ko, q)) return ATTN_ERR_ALIAS;
    }
    if (a.S == 0) return ATTN_OK;
    int sms = 0;
    if ((st = device(&sms)) != ATTN_OK) return st;
    RopeParams p;
    memset(&p, 0, sizeof p);
    p.x[0] = rope_tensor(a.q, a.q_out, a.q_stride, a.q_out_stride, a.H);
    if (a.k) p.x[1] = rope_tensor(a.k, a.k_out, a.k_stride, a.k_out_stride, Hkv);
    p.positions = a.positions;
    p.freqs = a.freqs;
    p.axes = a.axes;
    p.pos_axis = a.pos_axis_stride;
    p.pos_b = a.pos_batch_stride;
    p.S = a.S;
    p.tokens = a.B * a.S;
    p.pairs = a.pairs;
    p.num_axes = a.num_axes;
    p.inverse = a.inverse;
    p.heads = (int)(a.H + Hkv);
    return launch_rope(p, a.d, a.pairing == ATTN_ROPE_HALVES, false, sms, stream);
}

int run_append(const attn_append_args_t& a, cudaStream_t stream) {
    const int64_t H = a.q ? a.H : 0;
    if (!a.k || !a.v || !a.k_cache || !a.v_cache || (a.q && !a.q_out)) return ATTN_ERR_INVALID_ARG;
    if (!a.cu_seqlens_new || !a.seqlens_k || !a.block_table) return ATTN_ERR_INVALID_ARG;
    if (a.pairs != 0 && (!a.positions || !a.freqs || !a.axes)) return ATTN_ERR_INVALID_ARG;
    int st = check_cache(a.B, a.Hkv, a.num_pages, a.page_size, a.max_pages, a.d);
    if (st != ATTN_OK) return st;
    if (a.total < 0 || (a.q && H < 1) || a.reserved != 0 || a.pos_axis_stride < 0 ||
        a.pos_axis_stride > ((int64_t)1 << 40))
        return ATTN_ERR_INVALID_ARG;
    if (a.pairs != 0 && (st = check_pairs(a.pairs, a.num_axes, a.pairing, a.d)) != ATTN_OK) return st;
    if (a.total > kLim || H > kLim || H + 2 * a.Hkv > kLim) return ATTN_ERR_UNSUPPORTED;
    const int64_t nk[2] = {a.total, a.Hkv}, nq[2] = {a.total, H};
    if (!strides_ok(a.k_stride, nk, 2) || !strides_ok(a.v_stride, nk, 2) || (a.q && !strides_ok(a.q_stride, nq, 2)))
        return ATTN_ERR_INVALID_ARG;
    if (((uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache | (uintptr_t)a.q |
         (a.q ? (uintptr_t)a.q_out : 0)) & 15u)
        return ATTN_ERR_MISALIGNED;
    if (((uintptr_t)a.cu_seqlens_new | (uintptr_t)a.seqlens_k | (uintptr_t)a.block_table) & 3u) return ATTN_ERR_MISALIGNED;
    if (a.pairs && (((uintptr_t)a.positions | (uintptr_t)a.axes) & 3u || (uintptr_t)a.freqs & 7u)) return ATTN_ERR_MISALIGNED;
    if (!strides_aligned(a.k_stride, nk, 2) || !strides_aligned(a.v_stride, nk, 2) ||
        (a.q && !strides_aligned(a.q_stride, nq, 2)))
        return ATTN_ERR_MISALIGNED;
    auto v = [&](const void* p, int64_t heads, const int64_t* s) { return view(p, 1, a.total, heads, a.d, 0, s[0], s[1]); };
    const int64_t dense[2] = {H * a.d, a.d}, cs[2] = {a.Hkv * a.d, a.d};
    const View k = v(a.k, a.Hkv, a.k_stride), val = v(a.v, a.Hkv, a.v_stride);
    const View kc = view(a.k_cache, 1, a.num_pages * a.page_size, a.Hkv, a.d, 0, cs[0], cs[1]);
    const View vc = view(a.v_cache, 1, a.num_pages * a.page_size, a.Hkv, a.d, 0, cs[0], cs[1]);
    auto hits = [](const View& x, const View& y) { return x.span() && y.span() && overlap(x.at, x.end(), y.at, y.end()); };
    if (hits(kc, vc) || hits(kc, k) || hits(kc, val) || hits(vc, k) || hits(vc, val)) return ATTN_ERR_ALIAS;
    if (a.q) {
        const View q = v(a.q, H, a.q_stride), qo = v(a.q_out, H, dense);
        if ((!same(q, qo) && meet(q, qo)) || meet(qo, k) || meet(qo, val)) return ATTN_ERR_ALIAS;
        if (hits(qo, kc) || hits(qo, vc) || hits(q, kc) || hits(q, vc)) return ATTN_ERR_ALIAS;
    }
    if (a.total == 0) return ATTN_OK;
    int sms = 0;
    if ((st = device(&sms)) != ATTN_OK) return st;
    RopeParams p;
    memset(&p, 0, sizeof p);
    const int64_t qs[3] = {0, a.q_stride[0], a.q_stride[1]}, qo[3] = {0, dense[0], dense[1]};
    const int64_t ks[3] = {0, a.k_stride[0], a.k_stride[1]}, vs[3] = {0, a.v_stride[0], a.v_stride[1]};
    const int64_t co[3] = {0, cs[0], cs[1]};
    if (a.q) p.x[0] = rope_tensor(a.q, a.q_out, qs, qo, H);
    p.x[1] = rope_tensor(a.k, a.k_cache, ks, co, a.Hkv);
    p.x[2] = rope_tensor(a.v, a.v_cache, vs, co, a.Hkv);
    p.positions = a.positions;
    p.freqs = a.freqs;
    p.axes = a.axes;
    p.pos_axis = a.pos_axis_stride;
    p.S = p.tokens = a.total;
    p.pairs = a.pairs;
    p.num_axes = a.pairs ? a.num_axes : 1;
    p.heads = (int)(H + 2 * a.Hkv);
    p.pages = make_pages(a.block_table, a.num_pages, a.page_size, a.max_pages);
    p.cu_new = a.cu_seqlens_new;
    p.seqlens_k = a.seqlens_k;
    p.B = (int)a.B;
    return launch_rope(p, a.d, a.pairs && a.pairing == ATTN_ROPE_HALVES, true, sms, stream);
}

// ------------------------------------------------------------------------------ decode
// blocks of 8 query heads that a warp takes of a K/V head's group: the whole group up to 32, in
// powers of two (the instances); larger groups read the keys once per 32 heads
int head_tiles(int64_t group) { return group <= 8 ? 1 : group <= 16 ? 2 : 4; }

// Few short rows go to a CTA each: one launch, no parts to join.  A tile costs such a CTA 0.5 to 0.9 us, and
// the split path 3 us more to begin with, so rows of up to 5 tiles are not split; where the rows nearly fill
// the SMs a split gains little, and up to 10 tiles are not.  By the table's room (lengths are on the device).
// us a call in a graph, d = 128, split / whole:  8 rows of 2 tiles 7.0 / 4.8, 5 tiles 7.0 / 7.1, 8 tiles 7.2 / 9.4;
// 16 x 8 rows of 2 tiles 7.8 / 5.2, 5 tiles 11.8 / 8.0, 8 tiles 14.5 / 10.8.
// (Short rows in a wide table are split: 2 rows of 513 keys, d = 64, 5.9 in a table of 528 slots, 6.2 in one of 32,768.)
bool decode_whole(const attn_decode_args_t& a, int sms) {
    const int64_t group = a.H / a.Hkv, rows = a.B * a.Hkv * cdiv(group, 8 * head_tiles(group));
    const int64_t tiles = cdiv(a.max_pages * a.page_size, kDecTile);
    return !a.weights && rows <= sms && (tiles <= 5 || (tiles <= 10 && tiles * (sms - rows) <= 5 * sms));
}

struct DecodeLayout {
    size_t part_o, part_ml, split, row_ml, scores, bytes;
};
int64_t score_room(const attn_decode_args_t& a) { return cdiv(a.max_pages * a.page_size, 4) * 4; }
DecodeLayout decode_layout(const attn_decode_args_t& a, int sms) {
    const int64_t heads = 8 * head_tiles(a.H / a.Hkv), blocks = cdiv(a.H / a.Hkv, heads);
    DecodeLayout l;
    l.part_o = 0;
    l.part_ml = align256((size_t)(2 * sms * heads * a.d) * 4);
    l.split = l.part_ml + align256((size_t)(2 * sms * heads) * 8);
    l.row_ml = l.split + align256((size_t)sms * 16);
    l.scores = l.row_ml + (a.weights ? align256((size_t)(a.B * a.Hkv * blocks * heads) * 8) : 0);
    l.bytes = decode_whole(a, sms) ? 0 : l.scores + (a.weights ? (size_t)(a.B * a.H) * (size_t)score_room(a) * 4 : 0);
    return l;
}

int check_decode_shape(const attn_decode_args_t& a) {
    if (a.H < 1 || a.Hkv < 1) return ATTN_ERR_INVALID_ARG;
    int st = check_cache(a.B, a.Hkv, a.num_pages, a.page_size, a.max_pages, a.d);
    if (st != ATTN_OK) return st;
    if (a.H % a.Hkv != 0 || a.round_mode < ATTN_ROUND_RTNE || a.round_mode > ATTN_ROUND_RTZ || a.reserved != 0)
        return ATTN_ERR_INVALID_ARG;
    if (a.H > kLim || a.B * a.H > kLim) return ATTN_ERR_UNSUPPORTED;
    // places on the attention kernel's line are int32
    const int64_t group = a.H / a.Hkv, rows = a.B * a.Hkv * cdiv(group, 8 * head_tiles(group));
    if (cdiv(a.max_pages * a.page_size, kDecTile) + 1 > (2 * kLim - 1) / rows) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

template <int D, int NH>
int launch_decode(const DecodeParams& p, cudaStream_t stream) {
    int st;
    // the weights' blocks: three an SM, beside one that joins
    if (p.weights) {
        st = launch(attn_decode_kernel<D, NH, true>, p.grid, 1, kDecThreads, DecGeo<D>::kSmem, stream, p);
        if (st != ATTN_OK) return st;
        return launch(attn_decode_join_kernel<D, NH, true>, 4 * p.grid, 1, 256, 0, stream, p);
    }
    st = launch(attn_decode_kernel<D, NH, false>, p.grid, 1, kDecThreads, DecGeo<D>::kSmem, stream, p);
    if (st != ATTN_OK || p.whole) return st;
    return launch(attn_decode_join_kernel<D, NH, false>, p.grid, 1, 256, 0, stream, p);
}

int run_decode(const attn_decode_args_t& a, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_decode_shape(a);
    if (st != ATTN_OK) return st;
    if (!a.q || !a.k_cache || !a.v_cache || !a.o || !a.seqlens_k || !a.block_table) return ATTN_ERR_INVALID_ARG;
    if (((uintptr_t)a.q | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache | (uintptr_t)a.o) & 15u) return ATTN_ERR_MISALIGNED;
    if (((uintptr_t)a.lse | (uintptr_t)a.weights | (uintptr_t)a.seqlens_k | (uintptr_t)a.block_table) & 3u)
        return ATTN_ERR_MISALIGNED;
    const uintptr_t cb = (uintptr_t)(a.num_pages * a.page_size * a.Hkv * a.d * 2), qb = (uintptr_t)(a.B * a.H * a.d * 2);
    const uintptr_t wb = (uintptr_t)(a.B * a.Hkv) * (uintptr_t)(a.max_pages * a.page_size) * 4;
    struct { uintptr_t at, bytes; } in[] = {{(uintptr_t)a.q, qb}, {(uintptr_t)a.k_cache, cb}, {(uintptr_t)a.v_cache, cb},
                                            {(uintptr_t)a.seqlens_k, (uintptr_t)a.B * 4},
                                            {(uintptr_t)a.block_table, (uintptr_t)(a.B * a.max_pages) * 4}},
      out[4] = {{(uintptr_t)a.o, qb}, {(uintptr_t)a.lse, a.lse ? (uintptr_t)(a.B * a.H) * 4 : 0},
                {(uintptr_t)a.weights, a.weights ? wb : 0}, {0, 0}};
    int sms = 0;
    for (int pass = 0; pass < 2; ++pass) {
        if (pass == 1) {       // the workspace, once its size is known
            if ((st = device(&sms)) != ATTN_OK) return st;
            const DecodeLayout l = decode_layout(a, sms);
            if (l.bytes && (!workspace || workspace_bytes < l.bytes)) return ATTN_ERR_WORKSPACE;
            if (l.bytes && (uintptr_t)workspace & 15u) return ATTN_ERR_MISALIGNED;
            out[3].at = (uintptr_t)workspace;
            out[3].bytes = l.bytes;
        }
        for (int i = 0; i < 4; ++i) {
            if (!out[i].bytes) continue;
            for (const auto& x : in)
                if (overlap(out[i].at, out[i].at + out[i].bytes, x.at, x.at + x.bytes)) return ATTN_ERR_ALIAS;
            for (int j = 0; j < i; ++j)
                if (out[j].bytes && overlap(out[i].at, out[i].at + out[i].bytes, out[j].at, out[j].at + out[j].bytes))
                    return ATTN_ERR_ALIAS;
        }
    }
    const DecodeLayout l = decode_layout(a, sms);
    char* ws = reinterpret_cast<char*>(workspace);
    DecodeParams p;
    memset(&p, 0, sizeof p);
    p.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
    p.k = reinterpret_cast<const char*>(a.k_cache);
    p.v = reinterpret_cast<const char*>(a.v_cache);
    p.o = reinterpret_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    p.weights = a.weights;
    p.seqlens_k = a.seqlens_k;
    p.pages = make_pages(a.block_table, a.num_pages, a.page_size, a.max_pages);
    p.B = (int)a.B;
    p.H = (int)a.H;
    p.Hkv = (int)a.Hkv;
    p.group = (int)(a.H / a.Hkv);
    const int nh = head_tiles(p.group);
    p.head_blocks = (int)cdiv(p.group, 8 * nh);
    p.round_mode = a.round_mode;
    p.whole = decode_whole(a, sms);
    p.grid = p.whole ? p.B * p.Hkv * p.head_blocks : sms;
    p.scale = (float)(1.0 / std::sqrt((double)a.d));
    p.scale_log2 = (float)((1.0 / std::sqrt((double)a.d)) * 1.4426950408889634);
    p.part_o = reinterpret_cast<float*>(ws + l.part_o);
    p.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
    p.split = reinterpret_cast<int4*>(ws + l.split);
    p.row_ml = reinterpret_cast<float2*>(ws + l.row_ml);
    p.scores = reinterpret_cast<float*>(ws + l.scores);
    p.score_room = score_room(a);
    if (a.d == 128)
        return nh == 1   ? launch_decode<128, 1>(p, stream)
               : nh == 2 ? launch_decode<128, 2>(p, stream)
                         : launch_decode<128, 4>(p, stream);
    return nh == 1   ? launch_decode<64, 1>(p, stream)
           : nh == 2 ? launch_decode<64, 2>(p, stream)
                     : launch_decode<64, 4>(p, stream);
}

// ------------------------------------------------------------------------------ evict
int check_evict_shape(const attn_evict_args_t& a) {
    int st = check_cache(a.B, a.Hkv, a.num_pages, a.page_size, a.max_pages, a.d);
    if (st != ATTN_OK) return st;
    if (a.budget < 1 || a.sinks < 0 || a.recent < 0 || a.sinks > a.budget || a.recent > a.budget ||
        a.sinks + a.recent > a.budget)
        return ATTN_ERR_INVALID_ARG;
    // 17 tasks a head at most; moves are counted, and rows of a head numbered, in int32
    if (a.budget > kLim || a.B * a.Hkv > kLim / 32 || a.num_pages * a.page_size > 2 * kLim / a.Hkv ||
        a.max_pages * a.page_size > 2 * kLim / (a.B * a.Hkv))
        return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

struct EvictLayout {
    size_t uses, cut, lens, total, list, each, bytes;
    int64_t most_moves;
};
EvictLayout evict_layout(const attn_evict_args_t& a) {
    const int64_t keep = a.budget - a.sinks - a.recent, over = a.max_pages * a.page_size - a.budget;
    EvictLayout l;
    l.most_moves = over < 0 ? 0 : keep < over ? keep : over;
    const size_t all = (size_t)(a.B * a.Hkv) * (size_t)l.most_moves;
    l.uses = 0;
    l.cut = align256((size_t)a.num_pages * 4);
    l.lens = l.cut + align256((size_t)a.B * 4);
    l.total = l.lens + align256((size_t)a.B * 4);
    l.list = l.total + 256;
    l.each = align256(all * 4);
    l.bytes = l.list + 4 * l.each;
    return l;
}

int run_evict(const attn_evict_args_t& a, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_evict_shape(a);
    if (st != ATTN_OK) return st;
    if (!a.k_cache || !a.v_cache || !a.weights || !a.weights_out || !a.seqlens_k || !a.seqlens_out || !a.block_table)
        return ATTN_ERR_INVALID_ARG;
    if (((uintptr_t)a.k_cache | (uintptr_t)a.v_cache) & 15u) return ATTN_ERR_MISALIGNED;
    if (((uintptr_t)a.weights | (uintptr_t)a.weights_out | (uintptr_t)a.seqlens_k | (uintptr_t)a.seqlens_out |
         (uintptr_t)a.block_table) & 3u)
        return ATTN_ERR_MISALIGNED;
    const EvictLayout l = evict_layout(a);
    const uintptr_t cb = (uintptr_t)(a.num_pages * a.page_size * a.Hkv * a.d * 2);
    const uintptr_t wb = (uintptr_t)(a.B * a.Hkv) * (uintptr_t)(a.max_pages * a.page_size) * 4, nb = (uintptr_t)a.B * 4;
    struct Range { uintptr_t at, bytes; };
    const Range all[] = {{(uintptr_t)a.k_cache, cb}, {(uintptr_t)a.v_cache, cb}, {(uintptr_t)a.weights, wb},
                         {(uintptr_t)a.block_table, (uintptr_t)(a.B * a.max_pages) * 4}, {(uintptr_t)a.seqlens_k, nb},
                         {(uintptr_t)a.weights_out, a.weights_out != a.weights ? wb : 0},
                         {(uintptr_t)a.seqlens_out, a.seqlens_out != a.seqlens_k ? nb : 0},
                         {(uintptr_t)workspace, workspace ? l.bytes : 0}};
    for (const Range& x : all)
        for (const Range& y : all)
            if (&x != &y && x.bytes && y.bytes && overlap(x.at, x.at + x.bytes, y.at, y.at + y.bytes))
                return ATTN_ERR_ALIAS;
    if (!workspace || workspace_bytes < l.bytes) return ATTN_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15u) return ATTN_ERR_MISALIGNED;
    int sms = 0;
    if ((st = device(&sms)) != ATTN_OK) return st;
    char* ws = reinterpret_cast<char*>(workspace);
    EvictParams p;
    memset(&p, 0, sizeof p);
    p.k = reinterpret_cast<char*>(a.k_cache);
    p.v = reinterpret_cast<char*>(a.v_cache);
    p.weights = a.weights;
    p.weights_out = a.weights_out;
    p.seqlens_k = a.seqlens_k;
    p.seqlens_out = a.seqlens_out;
    p.pages = make_pages(a.block_table, a.num_pages, a.page_size, a.max_pages);
    p.B = (int)a.B;
    p.Hkv = (int)a.Hkv;
    p.row_bytes = (int)a.d * 2;
    p.budget = (int)a.budget;
    p.sinks = (int)a.sinks;
    p.recent = (int)a.recent;
    p.uses = reinterpret_cast<int32_t*>(ws + l.uses);
    p.cut = reinterpret_cast<int32_t*>(ws + l.cut);
    p.lens = reinterpret_cast<int32_t*>(ws + l.lens);
    p.total = reinterpret_cast<int32_t*>(ws + l.total);
    p.to = reinterpret_cast<int32_t*>(ws + l.list);
    p.from = reinterpret_cast<int32_t*>(ws + l.list + l.each);
    p.w_to = reinterpret_cast<uint32_t*>(ws + l.list + 2 * l.each);
    p.w_from = reinterpret_cast<uint32_t*>(ws + l.list + 3 * l.each);
    const int64_t rows = a.B * a.Hkv, room = a.max_pages * a.page_size;
    // select: the CTAs of a row hold its keys in registers where 8 of 1024 threads can (else the keys are read again for
    // each pass), and more of them share a row while every CTA has an SM and 2048 keys
    p.cluster = 1;
    while (p.cluster < kMostCluster &&
           (room > (int64_t)p.cluster * 1024 * kHeldMost || (2 * rows * p.cluster <= sms && room > p.cluster * 2048)))
        p.cluster *= 2;
    const bool wide = room > (int64_t)p.cluster * 2048;      // 1024 threads, else 512: four keys a thread
    // column pieces of 32 bytes at least (a DRAM sector), until there are three CTAs for every SM
    p.pieces = 1;
    while (2 * rows * p.pieces < 3 * sms && p.row_bytes / p.pieces > 32) p.pieces *= 2;
    if ((st = launch_clusters(attn_evict_prep_kernel, kPrepCtas, kPrepCtas, kPrepThreads, 0, stream, p)) != ATTN_OK) return st;
    const int64_t ctas = rows * p.cluster;
    if (p.cluster == 1 && l.most_moves <= kMostWhole && a.recent <= kMostWhole) {
        st = wide ? launch(attn_evict_select_kernel<1024, true>, ctas, 1, 1024, 0, stream, p)
                  : launch(attn_evict_select_kernel<512, true>, ctas, 1, 512, 0, stream, p);
        if (st != ATTN_OK || p.seqlens_out != p.seqlens_k) return st;
        return launch(attn_evict_lens_kernel, 1, 1, 256, 0, stream, p);
    }
    st = wide ? launch_clusters(attn_evict_select_kernel<1024, false>, ctas, p.cluster, 1024, 0, stream, p)
              : launch_clusters(attn_evict_select_kernel<512, false>, ctas, p.cluster, 512, 0, stream, p);
    if (st != ATTN_OK) return st;
    if (l.most_moves > 0) {
        st = a.d == 128 ? launch(attn_evict_fill_kernel<128>, 16 * sms, 1, kFillThreads, 0, stream, p)
                        : launch(attn_evict_fill_kernel<64>, 16 * sms, 1, kFillThreads, 0, stream, p);
        if (st != ATTN_OK) return st;
    }
    return launch(attn_evict_shift_kernel, rows * (2 * p.pieces + 1), 1, kShiftThreads, 0, stream, p);
}

}  // namespace

extern "C" {

int attn_rope(const attn_rope_args_t* args, attn_stream_t stream) {
    return args ? run_rope(*args, (cudaStream_t)stream) : ATTN_ERR_INVALID_ARG;
}

int attn_paged_append(const attn_append_args_t* args, attn_stream_t stream) {
    return args ? run_append(*args, (cudaStream_t)stream) : ATTN_ERR_INVALID_ARG;
}

size_t attn_paged_decode_workspace_size(const attn_decode_args_t* args) {
    int sms = 0;
    if (!args || check_decode_shape(*args) != ATTN_OK || device(&sms) != ATTN_OK) return 0;
    return decode_layout(*args, sms).bytes;
}

int attn_paged_decode(const attn_decode_args_t* args, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
    return args ? run_decode(*args, workspace, workspace_bytes, (cudaStream_t)stream) : ATTN_ERR_INVALID_ARG;
}

size_t attn_paged_evict_workspace_size(const attn_evict_args_t* args) {
    return args && check_evict_shape(*args) == ATTN_OK ? evict_layout(*args).bytes : 0;
}

int attn_paged_evict(const attn_evict_args_t* args, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
    return args ? run_evict(*args, workspace, workspace_bytes, (cudaStream_t)stream) : ATTN_ERR_INVALID_ARG;
}

int attn_cache_get_device_status(attn_stream_t stream, int32_t* site) {
    if (site) *site = 0;
    uint32_t h[2] = {0u, 0u};
    const uint32_t zero[2] = {0u, 0u};
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess ||
        cudaMemcpyFromSymbol(h, g_status, sizeof h) != cudaSuccess ||
        cudaMemcpyToSymbol(g_status, zero, sizeof zero) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    if (site) *site = (int32_t)h[1];
    return (int)h[0];
}

}  // extern "C"
