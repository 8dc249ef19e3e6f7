// qx_layer.cuh -- what the kernels between the weight products share: 16- and
// 32-bit element types as f32, a token's sequence and position, a key's place
// in the paged cache, and launches under programmatic stream serialisation.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "qx_device.cuh"
#include "qx_internal.h"

namespace qx {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two f32 rounded to a pair of 16-bit values (the first in the low half).
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}

// N consecutive elements (16-byte aligned for N * sizeof(T) >= 16, else 8) as f32.
template <int N, typename T>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 f = reinterpret_cast<const float4*>(p)[i];
            v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
        }
    } else if constexpr (N == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const float2 a = unpack2<T>(u.x), b = unpack2<T>(u.y);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            const uint4 u = reinterpret_cast<const uint4*>(p)[i];
            const float2 a = unpack2<T>(u.x), b = unpack2<T>(u.y), c = unpack2<T>(u.z), d = unpack2<T>(u.w);
            v[8 * i] = a.x, v[8 * i + 1] = a.y, v[8 * i + 2] = b.x, v[8 * i + 3] = b.y;
            v[8 * i + 4] = c.x, v[8 * i + 5] = c.y, v[8 * i + 6] = d.x, v[8 * i + 7] = d.y;
        }
    }
}
template <int N, typename T>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            reinterpret_cast<uint4*>(p)[i] =
                make_uint4(pack2<T>(v[8 * i], v[8 * i + 1]), pack2<T>(v[8 * i + 2], v[8 * i + 3]),
                           pack2<T>(v[8 * i + 4], v[8 * i + 5]), pack2<T>(v[8 * i + 6], v[8 * i + 7]));
    }
}

// The sequence of token t (-1: none) and, through it, the token's position.
// A decode step brings one token a sequence, so sequence t is tried first.
__device__ __forceinline__ int seq_of_token(const KvView& kv, int t) {
    if (t < kv.n_seqs && kv.q_start[t] <= t && t < kv.q_start[t + 1]) return t;
    int lo = 0, hi = kv.n_seqs;  // the last sequence that starts at or before t lies in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (kv.q_start[mid] <= t) lo = mid;
        else hi = mid;
    }
    return (kv.q_start[lo] <= t && t < kv.q_start[lo + 1]) ? lo : -1;
}
__device__ __forceinline__ int64_t position_of(const KvView& kv, int seq, int t) {
    return int64_t(kv.kv_len[seq]) - kv.q_start[seq + 1] + t;
}

// The page that holds key j of a sequence (j >= 0), or -1 (reported) where the
// table has none or a page outside the cache.
__device__ __forceinline__ int page_of(const KvView& kv, int seq, int64_t j) {
    const int64_t i = j >> kv.page_shift;
    int page = -1;
    if (i < kv.table_stride) page = kv.table[int64_t(seq) * kv.table_stride + i];
    if (page < 0 || page >= kv.n_pages) {
        atomicOr(kv.err, kErrRange);
        return -1;
    }
    return page;
}
// Element offset of key j's slot in its page, for head h.
__device__ __forceinline__ int64_t slot_offset(const KvView& kv, int page, int h, int64_t j) {
    return int64_t(page) * kv.page_stride + int64_t(h) * kv.head_stride +
           (j & ((int64_t(1) << kv.page_shift) - 1)) * kv.slot_stride;
}

// A launch that may begin while the stream's preceding kernel drains; every
// kernel launched this way waits for that kernel before its first access to
// memory (pdl_wait_prior_grid), so the order is the plain stream order.
template <typename K, typename P>
inline cudaError_t launch_serial(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, const P& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace qx
