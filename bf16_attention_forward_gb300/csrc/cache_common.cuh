// cache_common.cuh -- what the kernels around the paged K/V cache share: the status word,
// page lookup, and the instruction wrappers that only they use.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/bf16_attn.h"
#include "ptx.cuh"

namespace cache {

__device__ uint32_t g_status[2];   // [0] status code, [1] the check that failed

// first failure wins until the host reads and clears the word
__device__ __forceinline__ void report_invalid(uint32_t site) {
    if (atomicCAS(&g_status[0], 0u, (uint32_t)ATTN_ERR_INVALID_ARG) == 0u) atomicExch(&g_status[1], site);
}

// The paged cache as the kernels see it: key j of sequence b is row
// table[b][j / page_size] * page_size + j % page_size of a [rows][Hkv][d] tensor.
struct Pages {
    const int32_t* table;
    int page_size, max_pages, num_pages;
    uint32_t mul, shift;           // j / page_size = j * mul >> shift for 0 <= j < 2^30
};

// With 2^(L-1) < page_size <= 2^L and mul = ceil(2^(30+L) / page_size) < 2^31 the excess mul * page_size - 2^(30+L) is
// below 2^L, so for j < 2^30 it never carries the quotient to the next integer.
__device__ __forceinline__ int page_of(const Pages& c, int j) {
    return (int)(((unsigned long long)(uint32_t)j * c.mul) >> c.shift);
}

// row of slot j of a sequence whose table row is `t` (j inside the table), -1 for a page that
// the cache does not have
__device__ __forceinline__ int page_row(const Pages& c, const int32_t* t, int j) {
    const int pg = page_of(c, j);
    const int phys = __ldg(t + pg);
    return (unsigned)phys < (unsigned)c.num_pages ? phys * c.page_size + (j - pg * c.page_size) : -1;
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 16 bytes global -> shared under an L2 policy; bytes = 0 writes zeros and reads nothing
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void st_policy(float* p, float x, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.f32 [%0], %1, %2;" ::"l"(p), "f"(x), "l"(policy) : "memory");
}
__device__ __forceinline__ float4 ld_policy(const float4* p, uint64_t policy) {
    float4 v;
    asm volatile("ld.global.L2::cache_hint.v4.f32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p), "l"(policy)
                 : "memory");
    return v;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// transpose of an 8x8 matrix of 16-bit values held by a warp
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// D (16x8 fp32) += A (16x16 bf16, row) * B (16x8 bf16, column)
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// fp32 -> bf16 bits in a rounding mode; every NaN becomes 0x7FC0
__device__ __forceinline__ uint32_t round_bf16(float f, int mode) {
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;
    if (mode == ATTN_ROUND_RTNE) u += 0x7FFFu + ((u >> 16) & 1u);
    else if (mode == ATTN_ROUND_RTNA) u += 0x8000u;
    return u >> 16;
}

}  // namespace cache
