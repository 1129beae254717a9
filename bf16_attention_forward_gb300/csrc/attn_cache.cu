// attn_cache.cu -- host side of the calls around the paged K/V cache: rotary positions (rope.cuh),
// appending (rope.cuh), attention of one new token (decode.cuh) and eviction (evict.cuh); norms with positions
// (norm_rope.cuh), pages and slots (reserve.cuh), and one new token behind a shared prefix (prefix.cuh).
#include <cuda_runtime.h>
#include <string.h>

#include <cmath>
#include <mutex>
#include <type_traits>

#include "cache_common.cuh"
#include "decode.cuh"
#include "evict.cuh"
#include "norm_rope.cuh"
#include "prefix.cuh"
#include "reserve.cuh"
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

template <int D, bool kSingle>
cudaError_t set_prefix_attr() {
    return cudaFuncSetAttribute(attn_prefix_kernel<D, kSingle>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                PfGeo<D, kSingle>::kSmem);
}
template <int D, int NH>
cudaError_t set_decode_attr() {
    cudaError_t e = cudaSuccess;
    for (auto kernel : {attn_decode_kernel<D, NH, false>, attn_decode_kernel<D, NH, true>, attn_decode_kernel<D, NH, false, kCommonKeys>,
                        attn_decode_kernel<D, NH, false, kOwnKeys>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, DecGeo<D>::kSmem);
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
             set_decode_attr<64, 2>() != cudaSuccess || set_decode_attr<64, 4>() != cudaSuccess ||
             set_prefix_attr<128, false>() != cudaSuccess || set_prefix_attr<128, true>() != cudaSuccess ||
             set_prefix_attr<64, false>() != cudaSuccess || set_prefix_attr<64, true>() != cudaSuccess)) {
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
// it touches global memory and before it ends, and only then lets the next one start.  Two differ.
// Eviction's select kernel reads lengths and weights while the prepare kernel runs, which only reads them too; what ran before that
// is complete by then, because the prepare kernel's CTAs let select start behind their own wait.
// The own keys' kernel behind a shared prefix (attn_decode_kernel<.., kOwnKeys>) lets the join start at once, reads lengths, table, queries and
// caches and writes its parts of the workspace, all before its wait.  That holds as long as the prefix's kernel is the launch directly before it
// and lets it start only behind a wait of its own (so that what ran before is complete, the last call's join among it, which read
// that workspace), writes nothing of what it reads or writes, and as long as each of its exits passes its wait (so that the join, which waits
// for this kernel, has the prefix's parts too).
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
    if (!v.span()) return true;
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
    if (p.common) {
        st = launch(attn_decode_kernel<D, NH, false, kCommonKeys>, p.grid, 1, kDecThreads, DecGeo<D>::kSmem, stream, p);
        if (st != ATTN_OK || p.whole) return st;
        return launch(attn_decode_join_kernel<D, NH, false, kCommonKeys>, p.grid, 1, 256, 0, stream, p);
    }
    st = launch(attn_decode_kernel<D, NH, false>, p.grid, 1, kDecThreads, DecGeo<D>::kSmem, stream, p);
    if (st != ATTN_OK || p.whole) return st;
    return launch(attn_decode_join_kernel<D, NH, false>, p.grid, 1, 256, 0, stream, p);
}

// all but the workspace
void fill_decode(DecodeParams& p, const attn_decode_args_t& a, int sms) {
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
    p.block_heads = 8 * head_tiles(p.group);
    p.head_blocks = (int)cdiv(p.group, p.block_heads);
    p.round_mode = a.round_mode;
    p.whole = decode_whole(a, sms);
    p.grid = p.whole ? p.B * p.Hkv * p.head_blocks : sms;
    p.scale = (float)(1.0 / std::sqrt((double)a.d));
    p.scale_log2 = (float)((1.0 / std::sqrt((double)a.d)) * 1.4426950408889634);
}

// what a decoding call reads and writes: pointers, alignment, overlaps; then its workspace, once the size is known
struct DecodeRanges {
    struct Range { uintptr_t at, bytes; } in[5], out[3];
    explicit DecodeRanges(const attn_decode_args_t& a) {
        const uintptr_t cb = (uintptr_t)(a.num_pages * a.page_size * a.Hkv * a.d * 2), qb = (uintptr_t)(a.B * a.H * a.d * 2);
        const uintptr_t wb = (uintptr_t)(a.B * a.Hkv) * (uintptr_t)(a.max_pages * a.page_size) * 4;
        in[0] = {(uintptr_t)a.q, qb};
        in[1] = {(uintptr_t)a.k_cache, cb};
        in[2] = {(uintptr_t)a.v_cache, cb};
        in[3] = {(uintptr_t)a.seqlens_k, (uintptr_t)a.B * 4};
        in[4] = {(uintptr_t)a.block_table, (uintptr_t)(a.B * a.max_pages) * 4};
        out[0] = {(uintptr_t)a.o, qb};
        out[1] = {(uintptr_t)a.lse, a.lse ? (uintptr_t)(a.B * a.H) * 4 : 0};
        out[2] = {(uintptr_t)a.weights, a.weights ? wb : 0};
    }
    // whether a written range meets an input, or one of the first n outputs
    bool clash(const Range& r, int n) const {
        if (!r.bytes) return false;
        for (const Range& x : in)
            if (overlap(r.at, r.at + r.bytes, x.at, x.at + x.bytes)) return true;
        for (int i = 0; i < n; ++i)
            if (out[i].bytes && overlap(r.at, r.at + r.bytes, out[i].at, out[i].at + out[i].bytes)) return true;
        return false;
    }
};

int check_decode_tensors(const attn_decode_args_t& a) {
    if (!a.q || !a.k_cache || !a.v_cache || !a.o || !a.seqlens_k || !a.block_table) return ATTN_ERR_INVALID_ARG;
    if (((uintptr_t)a.q | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache | (uintptr_t)a.o) & 15u) return ATTN_ERR_MISALIGNED;
    if (((uintptr_t)a.lse | (uintptr_t)a.weights | (uintptr_t)a.seqlens_k | (uintptr_t)a.block_table) & 3u)
        return ATTN_ERR_MISALIGNED;
    const DecodeRanges r(a);
    for (int i = 0; i < 3; ++i)
        if (r.clash(r.out[i], i)) return ATTN_ERR_ALIAS;
    return ATTN_OK;
}

int check_decode_workspace(const attn_decode_args_t& a, const void* workspace, size_t bytes, size_t need) {
    if (!need) return ATTN_OK;
    if (!workspace || bytes < need) return ATTN_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15u) return ATTN_ERR_MISALIGNED;
    return DecodeRanges(a).clash({(uintptr_t)workspace, need}, 3) ? ATTN_ERR_ALIAS : ATTN_OK;
}

// common: leading keys that every sequence has of the first one's pages
int launch_decode_call(const attn_decode_args_t& a, int64_t common, int sms, void* workspace, cudaStream_t stream) {
    const DecodeLayout l = decode_layout(a, sms);
    char* ws = reinterpret_cast<char*>(workspace);
    DecodeParams p;
    fill_decode(p, a, sms);
    p.common = (int)common;
    p.part_o = reinterpret_cast<float*>(ws + l.part_o);
    p.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
    p.split = reinterpret_cast<int4*>(ws + l.split);
    p.row_ml = reinterpret_cast<float2*>(ws + l.row_ml);
    p.scores = reinterpret_cast<float*>(ws + l.scores);
    p.score_room = score_room(a);
    const int nh = head_tiles(p.group);
    if (a.d == 128)
        return nh == 1   ? launch_decode<128, 1>(p, stream)
               : nh == 2 ? launch_decode<128, 2>(p, stream)
                         : launch_decode<128, 4>(p, stream);
    return nh == 1   ? launch_decode<64, 1>(p, stream)
           : nh == 2 ? launch_decode<64, 2>(p, stream)
                     : launch_decode<64, 4>(p, stream);
}

int run_decode(const attn_decode_args_t& a, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_decode_shape(a);
    if (st != ATTN_OK) return st;
    if ((st = check_decode_tensors(a)) != ATTN_OK) return st;
    int sms = 0;
    if ((st = device(&sms)) != ATTN_OK) return st;
    if ((st = check_decode_workspace(a, workspace, workspace_bytes, decode_layout(a, sms).bytes)) != ATTN_OK) return st;
    return launch_decode_call(a, 0, sms, workspace, stream);
}

// ------------------------------------------------------------------------------ shared prefix
// Where a batch's tiles of the prefix, and two a row for its own keys and its end, are few, the decoding kernel itself reads the
// prefix's pages for each sequence: one or two kernels instead of three.  A tile costs it the more the more query heads it takes with one, but a
// batch whose rows it does not split pays a CTA's tiles only.  us a call in a graph, 16 to 100 own keys, again / shared:
//   blocks of 8 heads, d = 128: 16 sequences of 600 shared keys, 8 K/V heads (896 tiles) 9.2 / 22.9;  64 of 200 (2,048) 20.2 / 26.0;  16 of 2,000
//   (2,304) 21.8 / 23.3;  2 of 20,000 (2,544) 27.7 / 28.6;  4 of 10,000 (2,592) 25.3 / 23.4;  64 of 600 (3,584) 29.3 / 26.4;  16 of 4,000 (4,352)
//   35.1 / 24.0.  d = 64: 2,304 16.7 / 20.0;  2,592 18.3 / 19.1;  3,584 22.8 / 21.1.
//   16 heads, d = 128: 16 of 2,000, 4 K/V heads (1,152) 20.2 / 22.4;  4 of 5,000, 8 (1,344) 22.3 / 21.0;  4 of 6,000 (1,568) 24.5 / 21.6;  16 of 1,500
//   (1,792) 25.4 / 26.6;  64 of 200 (2,048) 32.0 / 30.2;  16 of 4,000, 4 (2,176) 27.4 / 23.3.  d = 64: 17.2 / 17.0 at 1,344, 20.6 / 18.3 at 2,176.
//   32 heads, d = 128: 2 of 4,000, 8 K/V heads (544) 28.1 / 21.1;  4 of 2,000 (576) 26.5 / 20.1;  4 of 3,000 (832) 30.1 / 21.7;  4 of 8,000, one of 71
//   heads (780) 33.1 / 20.2;  not split: 16 of 600 (896) 18.7 / 29.6, 16 of 1,000 (1,280) 24.1 / 30.9.  d = 64: 21.6 / 16.6 at 544, 16.7 / 23.6 at 1,280.
bool prefix_again(const attn_decode_args_t& a, int64_t prefix_len, int sms) {
    const int64_t nh = head_tiles(a.H / a.Hkv), rows = a.B * a.Hkv * cdiv(a.H / a.Hkv, 8 * nh);
    return a.B == 1 || decode_whole(a, sms) || 2 * rows * (cdiv(prefix_len, kDecTile) + 2) <= (nh == 1 ? 34 : nh == 2 ? 20 : 7) * sms;
}

// How the prefix's kernel divides: row blocks, and a line of steps over the CTAs.
struct PrefixPlan {
    bool single;
    int64_t row_blocks, steps, line, ctas, slots;
};
PrefixPlan prefix_plan(const attn_decode_args_t& a, int64_t prefix_len, int sms) {
    PrefixPlan p;
    const int64_t rows = a.B * (a.H / a.Hkv), tiles = cdiv(prefix_len, kPfTile);
    p.single = rows <= kPfTile;
    p.row_blocks = cdiv(rows, p.single ? kPfTile : 2 * kPfTile);
    p.steps = p.single ? cdiv(tiles, 2) : tiles;
    p.line = a.Hkv * p.row_blocks * (p.steps + kPfEnd);
    p.ctas = a.Hkv * p.row_blocks * p.steps < sms ? a.Hkv * p.row_blocks * p.steps : sms;
    p.slots = (cdiv(p.line, p.ctas) - 1 + p.steps + kPfEnd - 1) / (p.steps + kPfEnd) + 1;      // of a range that begins anywhere
    return p;
}

struct PrefixLayout {
    size_t x_o, x_ml, part_o, part_ml, span, own_o, own_ml, bytes;
};
PrefixLayout prefix_layout(const attn_decode_args_t& a, const PrefixPlan& plan, int sms) {
    const int64_t heads = 8 * head_tiles(a.H / a.Hkv), blocks = cdiv(a.H / a.Hkv, heads);
    const size_t rows = (size_t)(plan.ctas * plan.slots) * 2 * kPfTile, own = (size_t)(2 * sms * (heads == 8 ? kOwnWarps<1> : kOwnWarps<2>) * heads);
    PrefixLayout l;
    l.x_o = 0;
    l.x_ml = align256(rows * (size_t)a.d * 4);
    l.part_o = l.x_ml + align256(rows * 8);
    l.part_ml = l.part_o + align256(own * (size_t)a.d * 4);
    l.span = l.part_ml + align256(own * 8);
    l.own_o = l.span + align256((size_t)(a.B * a.Hkv * blocks) * 8);
    l.own_ml = l.own_o + align256((size_t)(a.B * a.H) * (size_t)a.d * 4);
    l.bytes = l.own_ml + align256((size_t)(a.B * a.H) * 8);
    return l;
}

int check_prefix_shape(const attn_decode_args_t& a, int64_t prefix_len) {
    const int st = check_decode_shape(a);
    if (st != ATTN_OK) return st;
    if (a.weights || prefix_len < 1 || prefix_len > a.max_pages * a.page_size) return ATTN_ERR_INVALID_ARG;
    // strides of a key are 32 bits, places on the lines of both kernels int32; the join has heads in y, a warp each or more
    if (a.Hkv * a.d > kLim) return ATTN_ERR_UNSUPPORTED;
    const int64_t group = a.H / a.Hkv, rows = a.B * a.Hkv * cdiv(group, 8 * head_tiles(group));
    if (cdiv(a.max_pages * a.page_size - prefix_len, kDecKeys) + 1 > (2 * kLim - 1) / rows) return ATTN_ERR_UNSUPPORTED;
    if (cdiv(prefix_len, kPfTile) + kPfEnd > (kLim - 1) / (a.Hkv * cdiv(a.B * group, kPfTile)) || a.H > 65535) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

template <int D, int NH>
int launch_own(const DecodeParams& p, cudaStream_t stream) {
    return launch(attn_decode_kernel<D, NH, false, kOwnKeys>, p.grid, 1, 32 * kOwnWarps<NH>, DecGeo<D>::kSmem, stream, p);
}
template <int D, bool kSingle>
int launch_prefix(const PrefixParams& p, int64_t ctas, cudaStream_t stream) {
    return launch(attn_prefix_kernel<D, kSingle>, ctas, 1, PfGeo<D, kSingle>::kThreads, PfGeo<D, kSingle>::kSmem, stream, p);
}

int run_prefix_decode(const attn_decode_args_t& a, int64_t prefix_len, uint32_t wait_limit_ms, uint32_t test_hooks, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
    int st = check_prefix_shape(a, prefix_len);
    if (st != ATTN_OK) return st;
    if (test_hooks != 0 && test_hooks != ATTN_TEST_WITHHOLD_O_READY) return ATTN_ERR_INVALID_ARG;
    if ((st = check_decode_tensors(a)) != ATTN_OK) return st;
    int sms = 0;
    if ((st = device(&sms)) != ATTN_OK) return st;
    if (prefix_again(a, prefix_len, sms)) {
        if ((st = check_decode_workspace(a, workspace, workspace_bytes, decode_layout(a, sms).bytes)) != ATTN_OK) return st;
        return launch_decode_call(a, prefix_len, sms, workspace, stream);
    }
    const PrefixPlan plan = prefix_plan(a, prefix_len, sms);
    const PrefixLayout l = prefix_layout(a, plan, sms);
    if ((st = check_decode_workspace(a, workspace, workspace_bytes, l.bytes)) != ATTN_OK) return st;
    char* ws = reinterpret_cast<char*>(workspace);
    PrefixJoin j;
    memset(&j, 0, sizeof j);
    fill_decode(j.s, a, sms);
    j.s.first = (int)prefix_len;
    j.s.whole = 0;
    j.s.grid = sms;
    j.s.part_o = reinterpret_cast<float*>(ws + l.part_o);
    j.s.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
    j.s.span = reinterpret_cast<int2*>(ws + l.span);
    j.s.own_o = reinterpret_cast<float*>(ws + l.own_o);
    j.s.own_ml = reinterpret_cast<float2*>(ws + l.own_ml);
    PrefixParams& x = j.x;
    x.q = j.s.q;
    x.k = j.s.k;
    x.v = j.s.v;
    x.pages = j.s.pages;
    x.H = j.s.H;
    x.Hkv = j.s.Hkv;
    x.group = j.s.group;
    x.rows = j.s.B * j.s.group;
    auto divisor = [](int64_t n) {
        const Pages c = make_pages(nullptr, 1, n, 1);
        return Divisor{c.mul, c.shift};
    };
    x.by_group = divisor(x.group);
    x.prefix_len = (int)prefix_len;
    x.row_blocks = (int)plan.row_blocks;
    x.steps = (int)plan.steps;
    x.ctas = (int)plan.ctas;
    x.per = (int)(plan.line / plan.ctas);
    x.more = (int)(plan.line % plan.ctas);
    x.slots = (int)plan.slots;
    x.by_places = divisor(plan.steps + kPfEnd);
    x.by_per = divisor(x.per);
    x.by_more = divisor(x.per + 1);
    x.scale_log2 = j.s.scale_log2;
    x.part_o = reinterpret_cast<float*>(ws + l.x_o);
    x.part_ml = reinterpret_cast<float2*>(ws + l.x_ml);
    x.wait_limit_ns = (wait_limit_ms ? wait_limit_ms : 2000u) * 1000000ull;
    x.test_hooks = (int)test_hooks;
    j.single = plan.single;
    // several warps a row where a row has more parts than a warp has in flight, while the SMs have room (16 warps each):
    // every warp has the same arithmetic to begin with (with 40: 66.3 us for 63.8 of 768 rows with 40 parts, 63.4 for 61.3 of 2,048 with 20)
    const int64_t parts = (cdiv(plan.steps - 1, x.per) + 1) * (plan.single ? 2 : 1);
    j.warps = 1;
    while (j.warps < kPfJoinWarps && parts > 8 * j.warps && a.B * a.H * j.warps <= 16 * sms) j.warps *= 2;
    st = a.d == 128 ? (plan.single ? launch_prefix<128, true>(x, plan.ctas, stream) : launch_prefix<128, false>(x, plan.ctas, stream))
                    : (plan.single ? launch_prefix<64, true>(x, plan.ctas, stream) : launch_prefix<64, false>(x, plan.ctas, stream));
    if (st != ATTN_OK) return st;
    const int nh = head_tiles(j.s.group);
    if (a.d == 128)
        st = nh == 1 ? launch_own<128, 1>(j.s, stream) : nh == 2 ? launch_own<128, 2>(j.s, stream) : launch_own<128, 4>(j.s, stream);
    else
        st = nh == 1 ? launch_own<64, 1>(j.s, stream) : nh == 2 ? launch_own<64, 2>(j.s, stream) : launch_own<64, 4>(j.s, stream);
    if (st != ATTN_OK) return st;
    const int heads = (int)cdiv(a.H * j.warps, 2 * kPfJoinWarps);
    auto* join = a.d == 128 ? (parts <= 4 ? attn_prefix_join_kernel<128, 4> : attn_prefix_join_kernel<128, 8>)
                            : (parts <= 4 ? attn_prefix_join_kernel<64, 4> : attn_prefix_join_kernel<64, 8>);
    return launch(join, a.B, heads, 32 * kPfJoinWarps, 0, stream, j);
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

// ------------------------------------------------------------------------------ norms with positions
View rows_view(const void* p, const attn_norm_rope_args_t& a, int64_t heads, const int64_t* s) {
    return view(p, a.B, a.S, heads, a.d, s[0], s[1], s[2]);
}
bool weight_ok(const void* w, int32_t bf16) { return ((uintptr_t)w & (bf16 ? 1u : 3u)) == 0; }
bool weights_meet(const View& out, const void* w, int64_t d, int32_t bf16) {
    return w && out.span() && overlap(out.at, out.end(), (uintptr_t)w, (uintptr_t)w + (uintptr_t)d * (bf16 ? 2 : 4));
}

// what attn_norm_rope and its gradient check alike: sizes, then pointers and strides
int check_norm_rope_shape(const attn_norm_rope_args_t& a) {
    const int64_t Hkv = a.k ? a.Hkv : 0;
    if (a.B < 1 || a.S < 0 || a.H < 1 || (a.k && Hkv < 1)) return ATTN_ERR_INVALID_ARG;
    if (!(a.eps >= 0.0f) || std::isinf(a.eps) || (a.weight_bf16 != 0 && a.weight_bf16 != 1) || a.reserved != 0)
        return ATTN_ERR_INVALID_ARG;
    const int st = check_pairs(a.pairs, a.num_axes, a.pairing, head_dim(a.d) ? a.d : 128);
    if (st != ATTN_OK) return st;
    if (!head_dim(a.d)) return ATTN_ERR_UNSUPPORTED;
    if (a.B > kLim || a.S > kLim || a.H > kLim || Hkv > kLim || a.B * a.S > kLim || a.H + Hkv > kLim)
        return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}
int check_norm_rope(const attn_norm_rope_args_t& a) {
    const int64_t Hkv = a.k ? a.Hkv : 0;
    if (!a.q || !a.q_out || (a.k && !a.k_out)) return ATTN_ERR_INVALID_ARG;
    if (a.pairs != 0 && (!a.positions || !a.freqs || !a.axes)) return ATTN_ERR_INVALID_ARG;
    const int st = check_norm_rope_shape(a);
    if (st != ATTN_OK) return st;
    const int64_t nq[3] = {a.B, a.S, a.H}, nk[3] = {a.B, a.S, Hkv};
    const int64_t np[2] = {a.num_axes, a.B}, ps[2] = {a.pos_axis_stride, a.pos_batch_stride};
    if (!strides_ok(a.q_stride, nq, 3) || !strides_ok(a.q_out_stride, nq, 3)) return ATTN_ERR_INVALID_ARG;
    if (a.pairs != 0 && !strides_ok(ps, np, 2)) return ATTN_ERR_INVALID_ARG;
    if (a.k && (!strides_ok(a.k_stride, nk, 3) || !strides_ok(a.k_out_stride, nk, 3))) return ATTN_ERR_INVALID_ARG;
    if (((uintptr_t)a.q | (uintptr_t)a.q_out | (uintptr_t)a.k | (a.k ? (uintptr_t)a.k_out : 0)) & 15u)
        return ATTN_ERR_MISALIGNED;
    if (a.pairs != 0 && (((uintptr_t)a.positions | (uintptr_t)a.axes) & 3u || (uintptr_t)a.freqs & 7u))
        return ATTN_ERR_MISALIGNED;
    if (!weight_ok(a.q_weight, a.weight_bf16) || !weight_ok(a.k_weight, a.weight_bf16)) return ATTN_ERR_MISALIGNED;
    if (!strides_aligned(a.q_stride, nq, 3) || !strides_aligned(a.q_out_stride, nq, 3)) return ATTN_ERR_MISALIGNED;
    if (a.k && (!strides_aligned(a.k_stride, nk, 3) || !strides_aligned(a.k_out_stride, nk, 3))) return ATTN_ERR_MISALIGNED;
    const View qo = rows_view(a.q_out, a, a.H, a.q_out_stride);
    const View ko = rows_view(a.k ? a.k_out : nullptr, a, Hkv, a.k_out_stride);
    if (!nested(qo) || (a.k && (!nested(ko) || meet(qo, ko)))) return ATTN_ERR_ALIAS;
    for (const void* w : {a.q_weight, a.k_weight})
        if (weights_meet(qo, w, a.d, a.weight_bf16) || (a.k && weights_meet(ko, w, a.d, a.weight_bf16))) return ATTN_ERR_ALIAS;
    return ATTN_OK;
}

void fill_norm_rope(NormRopeParams& p, const attn_norm_rope_args_t& a) {
    memset(&p, 0, sizeof p);
    p.x[0] = rope_tensor(a.q, a.q_out, a.q_stride, a.q_out_stride, a.H);
    if (a.k) p.x[1] = rope_tensor(a.k, a.k_out, a.k_stride, a.k_out_stride, a.Hkv);
    p.weight[0] = a.q_weight;
    p.weight[1] = a.k_weight;
    p.weight_bf16 = a.weight_bf16;
    p.eps = a.eps;
    p.positions = a.positions;
    p.freqs = a.freqs;
    p.axes = a.axes;
    p.pos_axis = a.pos_axis_stride;
    p.pos_b = a.pos_batch_stride;
    p.S = a.S;
    p.tokens = a.B * a.S;
    p.pairs = a.pairs;
    p.num_axes = a.num_axes;
    p.heads = (int)(a.H + (a.k ? a.Hkv : 0));
}

template <bool kAppend>
int launch_norm_rope(NormRopeParams& p, int64_t d, bool halves, int sms, cudaStream_t stream) {
    // Few tokens have their heads split over blocks, as long as all blocks still run at once: a second wave takes as long as the
    // first.  24 heads of d = 128, us: 600 tokens 5.4 (in more parts and two waves 7.6); 1,200 5.4 (11.1);
    // 2,400 7.1 (12.0); 6,144 tokens of 48 heads, appending, 29.6 in one part and 31.3 in two.
    const int64_t lanes = p.tokens * 32, full = (int64_t)kNormBlocks * kNormThreads * sms, piece = 32 / (d / 16);
    int64_t splits = lanes < full ? full / lanes : 1;
    if (splits > cdiv(p.heads, piece)) splits = cdiv(p.heads, piece);
    p.heads_per_block = (int)(cdiv(cdiv(p.heads, splits), piece) * piece);
    const int64_t most = cdiv(p.tokens, kNormWarps), grid = most < kNormBlocks * sms ? most : kNormBlocks * sms;
    const int gy = (int)cdiv(p.heads, p.heads_per_block);
    if (gy > 65535) return ATTN_ERR_UNSUPPORTED;
    auto* kernel = d == 128 ? (halves ? attn_norm_rope_kernel<128, true, kAppend> : attn_norm_rope_kernel<128, false, kAppend>)
                            : (halves ? attn_norm_rope_kernel<64, true, kAppend> : attn_norm_rope_kernel<64, false, kAppend>);
    return launch(kernel, grid, gy, kNormThreads, 0, stream, p);
}

int run_norm_rope(const attn_norm_rope_args_t& a, cudaStream_t stream) {
    int st = check_norm_rope(a);
    if (st != ATTN_OK) return st;
    const View q = rows_view(a.q, a, a.H, a.q_stride), qo = rows_view(a.q_out, a, a.H, a.q_out_stride);
    if (!same(q, qo) && meet(q, qo)) return ATTN_ERR_ALIAS;
    if (a.k) {
        const View k = rows_view(a.k, a, a.Hkv, a.k_stride), ko = rows_view(a.k_out, a, a.Hkv, a.k_out_stride);
        if ((!same(k, ko) && meet(k, ko)) || meet(qo, k) || meet(ko, q)) return ATTN_ERR_ALIAS;
    }
    if (a.S == 0) return ATTN_OK;
    int sms = 0;
    if ((st = device(&sms)) != ATTN_OK) return st;
    NormRopeParams p;
    fill_norm_rope(p, a);
    return launch_norm_rope<false>(p, a.d, a.pairs && a.pairing == ATTN_ROPE_HALVES, sms, stream);
}

// blocks of the gradient's kernel: as many as fit at once (each leaves 2 * d sums to be added up)
int norm_bwd_blocks(const attn_norm_rope_args_t& a, int sms) {
    const int64_t most = cdiv(a.B * a.S, kNormWarps), all = (int64_t)kNormBwdBlocks * sms;
    return (int)(most < 1 ? 1 : all < most ? all : most);
}
size_t norm_bwd_bytes(const attn_norm_rope_args_t& a, int sms) {
    return 2 * (size_t)norm_bwd_blocks(a, sms) * (size_t)a.d * 4;
}

int run_norm_rope_bwd(const attn_norm_rope_bwd_args_t& g, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    const attn_norm_rope_args_t& a = g.fwd;
    int st = check_norm_rope(a);
    if (st != ATTN_OK) return st;
    if (!g.dq || (g.dk != nullptr) != (a.k != nullptr) || (g.dk_weight && !a.k)) return ATTN_ERR_INVALID_ARG;
    const int64_t Hkv = a.k ? a.Hkv : 0, nq[3] = {a.B, a.S, a.H}, nk[3] = {a.B, a.S, Hkv};
    if (!strides_ok(g.dq_stride, nq, 3) || (a.k && !strides_ok(g.dk_stride, nk, 3))) return ATTN_ERR_INVALID_ARG;
    if (((uintptr_t)g.dq | (uintptr_t)g.dk) & 15u || ((uintptr_t)g.dq_weight | (uintptr_t)g.dk_weight) & 3u)
        return ATTN_ERR_MISALIGNED;
    if (!strides_aligned(g.dq_stride, nq, 3) || (a.k && !strides_aligned(g.dk_stride, nk, 3))) return ATTN_ERR_MISALIGNED;
    // tensors read, and written; what is flat in memory
    const View in[4] = {rows_view(a.q, a, a.H, a.q_stride), rows_view(g.dq, a, a.H, g.dq_stride),
                        rows_view(a.k, a, Hkv, a.k_stride), rows_view(g.dk, a, Hkv, g.dk_stride)};
    const View out[2] = {rows_view(a.q_out, a, a.H, a.q_out_stride), rows_view(a.k ? a.k_out : nullptr, a, Hkv, a.k_out_stride)};
    struct { uintptr_t at, bytes; } flat[3] = {{(uintptr_t)g.dq_weight, g.dq_weight ? (uintptr_t)a.d * 4 : 0},
                                               {(uintptr_t)g.dk_weight, g.dk_weight ? (uintptr_t)a.d * 4 : 0},
                                               {0, 0}};
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < 4; ++i)
            if (!(i == 2 * o + 1 && same(in[i], out[o])) && meet(in[i], out[o])) return ATTN_ERR_ALIAS;
    auto clash = [&](int f) {
        const uintptr_t b = flat[f].at, e = b + flat[f].bytes;
        if (b == e) return false;
        for (const View& v : in)
            if (v.span() && overlap(b, e, v.at, v.end())) return true;
        for (const View& v : out)
            if (v.span() && overlap(b, e, v.at, v.end())) return true;
        for (const void* w : {a.q_weight, a.k_weight})
            if (w && overlap(b, e, (uintptr_t)w, (uintptr_t)w + (uintptr_t)a.d * (a.weight_bf16 ? 2 : 4))) return true;
        for (int o = 0; o < f; ++o)
            if (flat[o].bytes && overlap(b, e, flat[o].at, flat[o].at + flat[o].bytes)) return true;
        return false;
    };
    if (clash(0) || clash(1)) return ATTN_ERR_ALIAS;
    int sms = 0;
    if ((st = device(&sms)) != ATTN_OK) return st;
    const size_t need = norm_bwd_bytes(a, sms);            // (the workspace, once its size is known)
    if (!workspace || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15u) return ATTN_ERR_MISALIGNED;
    flat[2].at = (uintptr_t)workspace;
    flat[2].bytes = need;
    if (clash(2)) return ATTN_ERR_ALIAS;
    NormRopeParams p;
    fill_norm_rope(p, a);
    p.dy[0] = rope_tensor(g.dq, nullptr, g.dq_stride, g.dq_stride, a.H);
    if (a.k) p.dy[1] = rope_tensor(g.dk, nullptr, g.dk_stride, g.dk_stride, Hkv);
    p.part = reinterpret_cast<float*>(workspace);
    p.dw[0] = g.dq_weight;
    p.dw[1] = g.dk_weight;
    p.blocks = a.S > 0 ? norm_bwd_blocks(a, sms) : 0;      // (no tokens: the weights' gradients are sums of nothing)
    if (a.S == 0) p.pairs = 0;
    const bool halves = a.pairs && a.pairing == ATTN_ROPE_HALVES;
    auto* kernel = a.d == 128 ? (halves ? attn_norm_rope_bwd_kernel<128, true> : attn_norm_rope_bwd_kernel<128, false>)
                              : (halves ? attn_norm_rope_bwd_kernel<64, true> : attn_norm_rope_bwd_kernel<64, false>);
    if (a.S > 0 && (st = launch(kernel, p.blocks, 1, kNormThreads, 0, stream, p)) != ATTN_OK) return st;
    if (!p.dw[0] && !p.dw[1]) return ATTN_OK;
    const int64_t grid = (a.k ? 2 : 1) * (a.d / 32);
    return a.d == 128 ? launch(attn_norm_rope_dw_kernel<128>, grid, 1, 32 * kDwRows, 0, stream, p)
                      : launch(attn_norm_rope_dw_kernel<64>, grid, 1, 32 * kDwRows, 0, stream, p);
}

int run_norm_append(const attn_norm_append_args_t& a, cudaStream_t stream) {
    const int64_t H = a.q ? a.H : 0;
    if (!a.k || !a.v || !a.k_cache || !a.v_cache || (a.q && !a.q_out) || !a.slots) return ATTN_ERR_INVALID_ARG;
    if (a.pairs != 0 && (!a.positions || !a.freqs || !a.axes)) return ATTN_ERR_INVALID_ARG;
    int st = check_cache(1, a.Hkv, a.num_pages, a.page_size, 1, a.d);
    if (st != ATTN_OK) return st;
    if (a.total < 0 || (a.q && H < 1) || a.reserved != 0 || a.pos_axis_stride < 0 ||
        a.pos_axis_stride > ((int64_t)1 << 40))
        return ATTN_ERR_INVALID_ARG;
    if (!(a.eps >= 0.0f) || std::isinf(a.eps) || (a.weight_bf16 != 0 && a.weight_bf16 != 1)) return ATTN_ERR_INVALID_ARG;
    if ((st = check_pairs(a.pairs, a.num_axes, a.pairing, a.d)) != ATTN_OK) return st;
    if (a.total > kLim || H > kLim || H + 2 * a.Hkv > kLim) return ATTN_ERR_UNSUPPORTED;
    const int64_t nk[2] = {a.total, a.Hkv}, nq[2] = {a.total, H};
    if (!strides_ok(a.k_stride, nk, 2) || !strides_ok(a.v_stride, nk, 2) || (a.q && !strides_ok(a.q_stride, nq, 2)))
        return ATTN_ERR_INVALID_ARG;
    if (((uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache | (uintptr_t)a.q |
         (a.q ? (uintptr_t)a.q_out : 0)) & 15u)
        return ATTN_ERR_MISALIGNED;
    if ((uintptr_t)a.slots & 7u) return ATTN_ERR_MISALIGNED;
    if (a.pairs && (((uintptr_t)a.positions | (uintptr_t)a.axes) & 3u || (uintptr_t)a.freqs & 7u)) return ATTN_ERR_MISALIGNED;
    if (!weight_ok(a.q_weight, a.weight_bf16) || !weight_ok(a.k_weight, a.weight_bf16)) return ATTN_ERR_MISALIGNED;
    if (!strides_aligned(a.k_stride, nk, 2) || !strides_aligned(a.v_stride, nk, 2) ||
        (a.q && !strides_aligned(a.q_stride, nq, 2)))
        return ATTN_ERR_MISALIGNED;
    const int64_t qs[3] = {0, a.q_stride[0], a.q_stride[1]}, qo[3] = {0, H * a.d, a.d};
    const int64_t ks[3] = {0, a.k_stride[0], a.k_stride[1]}, vs[3] = {0, a.v_stride[0], a.v_stride[1]};
    const int64_t co[3] = {0, a.Hkv * a.d, a.d};
    auto v = [&](const void* p, int64_t rows, int64_t heads, const int64_t* s) {
        return view(p, 1, rows, heads, a.d, 0, s[1], s[2]);
    };
    auto hits = [](const View& x, const View& y) { return x.span() && y.span() && overlap(x.at, x.end(), y.at, y.end()); };
    const int64_t rows = a.num_pages * a.page_size;
    const View in[3] = {v(a.k, a.total, a.Hkv, ks), v(a.v, a.total, a.Hkv, vs), v(a.q, a.total, H, qs)};
    const View kc = v(a.k_cache, rows, a.Hkv, co), vc = v(a.v_cache, rows, a.Hkv, co), out = v(a.q ? a.q_out : nullptr, a.total, H, qo);
    if (hits(kc, vc) || hits(out, kc) || hits(out, vc)) return ATTN_ERR_ALIAS;
    for (const View& x : in)
        if (hits(x, kc) || hits(x, vc) || (!(&x == &in[2] && same(x, out)) && meet(x, out))) return ATTN_ERR_ALIAS;
    for (const void* w : {a.q_weight, a.k_weight})
        for (const View* o : {&kc, &vc, &out})
            if (weights_meet(*o, w, a.d, a.weight_bf16)) return ATTN_ERR_ALIAS;
    if (a.total == 0) return ATTN_OK;
    int sms = 0;
    if ((st = device(&sms)) != ATTN_OK) return st;
    NormRopeParams p;
    memset(&p, 0, sizeof p);
    if (a.q) p.x[0] = rope_tensor(a.q, a.q_out, qs, qo, H);
    p.x[1] = rope_tensor(a.k, a.k_cache, ks, co, a.Hkv);
    p.x[2] = rope_tensor(a.v, a.v_cache, vs, co, a.Hkv);
    p.weight[0] = a.q_weight;
    p.weight[1] = a.k_weight;
    p.weight_bf16 = a.weight_bf16;
    p.eps = a.eps;
    p.positions = a.positions;
    p.freqs = a.freqs;
    p.axes = a.axes;
    p.pos_axis = a.pos_axis_stride;
    p.S = p.tokens = a.total;
    p.pairs = a.pairs;
    p.num_axes = a.num_axes;
    p.heads = (int)(H + 2 * a.Hkv);
    p.slots = a.slots;
    p.rows = rows;
    return launch_norm_rope<true>(p, a.d, a.pairs && a.pairing == ATTN_ROPE_HALVES, sms, stream);
}

// ------------------------------------------------------------------------------ pages and slots
int run_reserve(const attn_reserve_args_t& a, cudaStream_t stream) {
    if (!a.seqlens_k || !a.cu_seqlens_new || !a.block_table || !a.pages_held || !a.held_out || !a.free_pages ||
        !a.free_count || !a.count_out || (a.total > 0 && !a.slots))
        return ATTN_ERR_INVALID_ARG;
    int st = check_cache(a.B, 1, 1, a.page_size, a.max_pages, 128);
    if (st != ATTN_OK) return st;
    if (a.capacity < 1 || a.total < 0) return ATTN_ERR_INVALID_ARG;
    if (a.capacity > kLim || a.total > kLim) return ATTN_ERR_UNSUPPORTED;
    const uintptr_t B = (uintptr_t)a.B;
    const struct { uintptr_t at, bytes; bool written; } all[] = {
        {(uintptr_t)a.seqlens_k, B * 4, false},
        {(uintptr_t)a.cu_seqlens_new, (B + 1) * 4, false},
        {(uintptr_t)a.shared_pages, a.shared_pages ? B * 4 : 0, false},
        {(uintptr_t)a.pages_held, a.pages_held != a.held_out ? B * 4 : 0, false},
        {(uintptr_t)a.free_count, a.free_count != a.count_out ? 4u : 0u, false},
        {(uintptr_t)a.block_table, B * (uintptr_t)a.max_pages * 4, true},
        {(uintptr_t)a.free_pages, (uintptr_t)a.capacity * 4, true},
        {(uintptr_t)a.held_out, B * 4, true},
        {(uintptr_t)a.count_out, 4, true},
        {(uintptr_t)a.positions, a.positions ? (uintptr_t)a.total * 4 : 0, true},
        {(uintptr_t)a.slots, (uintptr_t)a.total * 8, true}};
    for (const auto& x : all) {
        if (x.at & 3u) return ATTN_ERR_MISALIGNED;
        for (const auto& y : all)
            if (&x != &y && (x.written || y.written) && x.bytes && y.bytes && overlap(x.at, x.at + x.bytes, y.at, y.at + y.bytes))
                return ATTN_ERR_ALIAS;
    }
    if ((uintptr_t)a.slots & 7u) return ATTN_ERR_MISALIGNED;
    int sms = 0;
    if ((st = device(&sms)) != ATTN_OK) return st;
    ReserveParams p;
    memset(&p, 0, sizeof p);
    p.seqlens = a.seqlens_k;
    p.cu_new = a.cu_seqlens_new;
    p.table = a.block_table;
    p.held = a.pages_held;
    p.held_out = a.held_out;
    p.shared = a.shared_pages;
    p.free_pages = a.free_pages;
    p.count = a.free_count;
    p.count_out = a.count_out;
    p.slots = a.slots;
    p.positions = a.positions;
    p.pages = make_pages(a.block_table, 1, a.page_size, a.max_pages);
    p.B = (int)a.B;
    p.capacity = (int)a.capacity;
    p.total = a.total;
    // a CTA while every thread has at most one token, else a cluster of them
    const int ctas = a.total > kReserveThreads ? 8 : 1;
    return launch_clusters(attn_reserve_kernel, ctas, ctas, kReserveThreads, 0, stream, p);
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

int attn_norm_rope(const attn_norm_rope_args_t* args, attn_stream_t stream) {
    return args ? run_norm_rope(*args, (cudaStream_t)stream) : ATTN_ERR_INVALID_ARG;
}

size_t attn_norm_rope_bwd_workspace_size(const attn_norm_rope_bwd_args_t* args) {
    int sms = 0;
    if (!args || check_norm_rope_shape(args->fwd) != ATTN_OK || device(&sms) != ATTN_OK) return 0;
    return norm_bwd_bytes(args->fwd, sms);
}

int attn_norm_rope_bwd(const attn_norm_rope_bwd_args_t* args, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
    return args ? run_norm_rope_bwd(*args, workspace, workspace_bytes, (cudaStream_t)stream) : ATTN_ERR_INVALID_ARG;
}

int attn_norm_rope_append(const attn_norm_append_args_t* args, attn_stream_t stream) {
    return args ? run_norm_append(*args, (cudaStream_t)stream) : ATTN_ERR_INVALID_ARG;
}

int attn_paged_reserve(const attn_reserve_args_t* args, attn_stream_t stream) {
    return args ? run_reserve(*args, (cudaStream_t)stream) : ATTN_ERR_INVALID_ARG;
}

size_t attn_paged_prefix_decode_workspace_size(const attn_decode_args_t* args, int64_t prefix_len) {
    int sms = 0;
    if (!args || check_prefix_shape(*args, prefix_len) != ATTN_OK || device(&sms) != ATTN_OK) return 0;
    return prefix_again(*args, prefix_len, sms) ? decode_layout(*args, sms).bytes
                                           : prefix_layout(*args, prefix_plan(*args, prefix_len, sms), sms).bytes;
}

int attn_paged_prefix_decode(const attn_decode_args_t* args, int64_t prefix_len, void* workspace, size_t workspace_bytes,
                             attn_stream_t stream) {
    return attn_paged_prefix_decode_ex(args, prefix_len, 0, 0, workspace, workspace_bytes, stream);
}

int attn_paged_prefix_decode_ex(const attn_decode_args_t* args, int64_t prefix_len, uint32_t wait_limit_ms, uint32_t test_hooks,
                                void* workspace, size_t workspace_bytes, attn_stream_t stream) {
    return args ? run_prefix_decode(*args, prefix_len, wait_limit_ms, test_hooks, workspace, workspace_bytes, (cudaStream_t)stream)
                : ATTN_ERR_INVALID_ARG;
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
