// Row tensors of several element types and strides: host checks shared by
// the entry points that take them, and device loads and stores of 4 values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "o1_common.cuh"

static inline bool o1_dtype_ok(int t) { return t == O1_F32 || t == O1_BF16 || t == O1_F16; }
static inline size_t o1_dtype_bytes(int t) { return t == O1_F32 ? 4 : 2; }

// `rows` rows of `width` bytes, `stride` bytes apart (a plain buffer: one row).
struct O1Span {
    const void *p;
    size_t width, stride;
    int64_t rows;
};

static inline O1Span o1_span(const void *p, size_t bytes) { return {p, bytes, bytes, 1}; }
static inline O1Span o1_row_span(const void *p, int dtype, int64_t heads, int64_t d, int64_t stride, int64_t rows) {
    const size_t e = o1_dtype_bytes(dtype);
    return {p, (size_t)(heads * d) * e, (size_t)stride * e, rows};
}

// Base and stride of a row tensor: 16-byte multiples, rows apart.
static inline bool o1_rows_ok(const O1Span &s) {
    return s.p && (uintptr_t)s.p % 16 == 0 && s.stride % 16 == 0 && s.stride >= s.width &&
           s.stride < ((size_t)1 << 40);
}

// Whether two spans share a byte. Exact for spans apart and for equal
// strides (columns of one buffer); otherwise spans whose extents meet count as
// overlapping.
static inline bool o1_spans_overlap(const O1Span &a, const O1Span &b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || !a.width || !b.width) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    const uintptr_t a1 = a0 + a.stride * (size_t)(a.rows - 1) + a.width;
    const uintptr_t b1 = b0 + b.stride * (size_t)(b.rows - 1) + b.width;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.stride != b.stride || a.rows < 2 || b.rows < 2) return true;
    const size_t s = a.stride, delta = b0 >= a0 ? (b0 - a0) % s : (s - (a0 - b0) % s) % s;
    return !(delta >= a.width && s - delta >= b.width);
}

// ------------------------------------------------------------ device: values

template <typename T>
__device__ __forceinline__ float o1_ld1(const T *p);
template <>
__device__ __forceinline__ float o1_ld1<float>(const float *p) { return *p; }
template <>
__device__ __forceinline__ float o1_ld1<__nv_bfloat16>(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float o1_ld1<__half>(const __half *p) { return __half2float(*p); }

// 4 consecutive values (16 or 8 bytes, aligned to that size)
__device__ __forceinline__ float4 o1_ld4(const float *p) { return *(const float4 *)p; }
__device__ __forceinline__ float4 o1_ld4(const __nv_bfloat16 *p) {
    const uint2 u = *(const uint2 *)p;
    const float2 a = __bfloat1622float2(*(const __nv_bfloat162 *)&u.x);
    const float2 b = __bfloat1622float2(*(const __nv_bfloat162 *)&u.y);
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 o1_ld4(const __half *p) {
    const uint2 u = *(const uint2 *)p;
    const float2 a = __half22float2(*(const __half2 *)&u.x);
    const float2 b = __half22float2(*(const __half2 *)&u.y);
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void o1_st4(float *p, float4 x) { *(float4 *)p = x; }
__device__ __forceinline__ void o1_st4(__nv_bfloat16 *p, float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *(uint2 *)p = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
}
__device__ __forceinline__ void o1_st4(__half *p, float4 x) {
    const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
    *(uint2 *)p = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
}
