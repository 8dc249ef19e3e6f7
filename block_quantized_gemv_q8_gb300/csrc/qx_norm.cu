// qx_norm.cu -- the norm after a block, its gate and residual scale, the
// residual sum and the norm before the next block, in one pass over the row.
//
//   u = y w_post / sqrt(mean(y^2) + eps);  r' = r + alpha gate u;
//   x = r' w_pre / sqrt(mean(r'^2) + eps)
//
// A CTA owns a row and keeps it in registers between the two sums, so each
// element is read and written once: the call is bound by those bytes, and for
// one row by the two block-wide sums.
#include "qx_layer.cuh"

namespace qx {

namespace {

// Sum over the CTA (up to 32 warps), the same order in every thread and run.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// N consecutive elements with VEC-wide access (VEC 8: 16-byte aligned rows of
// whole vectors; VEC 1: any row).
template <int VEC, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
    if constexpr (VEC == 1) v[0] = to_f32(*p);
    else load_f32<VEC>(p, v);
}
template <int VEC, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) *p = from_f32<T>(v[0]);
    else store_f32<VEC>(p, v);
}

template <typename A, typename R, int VEC, int N>
__global__ void __launch_bounds__(1024) block_norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float part[2][32];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const A* y = static_cast<const A*>(p.y) + row * p.y_stride;
    const R* r = static_cast<const R*>(p.r) + row * p.r_stride;
    const A* gate = static_cast<const A*>(p.gate) + row * p.gate_stride;
    float u[N][VEC], rr[N][VEC];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) u[n][i] = rr[n][i] = 0.0f;
        if (c < p.cols) {
            if (p.y) load_vec<VEC>(y + c, u[n]);
            load_vec<VEC>(r + c, rr[n]);
        }
    }
    float inv = 1.0f;
    if (p.y && p.w_post) {
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s += u[n][i] * u[n][i];
        inv = 1.0f / sqrtf(block_sum(s, part[0]) / float(p.cols) + p.eps);
    }
    if (p.y) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * blockDim.x + threadIdx.x) * VEC;
            if (c >= p.cols) continue;
            float w[VEC], g[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = g[i] = 1.0f;
            if (p.w_post) load_vec<VEC>(p.w_post + c, w);
            if (p.gate) load_vec<VEC>(gate + c, g);
#pragma unroll
            for (int i = 0; i < VEC; ++i) rr[n][i] += p.alpha * (g[i] * (u[n][i] * inv * w[i]));
        }
    }
    if (p.r_out) {
        R* ro = static_cast<R*>(p.r_out) + row * p.r_out_stride;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * blockDim.x + threadIdx.x) * VEC;
            if (c < p.cols) store_vec<VEC>(ro + c, rr[n]);
        }
    }
    if (!p.w_pre) return;
    float s = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += rr[n][i] * rr[n][i];
    const float inv2 = 1.0f / sqrtf(block_sum(s, part[1]) / float(p.cols) + p.eps);
    A* x = static_cast<A*>(p.x) + row * p.x_stride;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * blockDim.x + threadIdx.x) * VEC;
        if (c >= p.cols) continue;
        float w[VEC];
        load_vec<VEC>(p.w_pre + c, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] *= rr[n][i] * inv2;
        store_vec<VEC>(x + c, w);
    }
}

template <typename A, typename R>
cudaError_t launch_types(const NormParams& p, bool vec, cudaStream_t s) {
    // One vector a thread, up to four for rows above 8192 columns; rows that
    // are not whole aligned vectors take single elements, up to 32 a thread.
    const int units = vec ? p.cols / 8 : p.cols;
    const int per = (units + 1023) / 1024;
    const int n = per <= 1 ? 1 : vec ? 4 : per <= 8 ? 8 : 32;
    int threads = (units + n - 1) / n;
    threads = threads < 32 ? 32 : (threads + 31) / 32 * 32;
    const dim3 grid(static_cast<unsigned>(p.rows));
    if (vec) {
        if (n == 1) return launch_serial(block_norm_kernel<A, R, 8, 1>, grid, threads, 0, s, p);
        return launch_serial(block_norm_kernel<A, R, 8, 4>, grid, threads, 0, s, p);
    }
    if (n == 1) return launch_serial(block_norm_kernel<A, R, 1, 1>, grid, threads, 0, s, p);
    if (n == 8) return launch_serial(block_norm_kernel<A, R, 1, 8>, grid, threads, 0, s, p);
    return launch_serial(block_norm_kernel<A, R, 1, 32>, grid, threads, 0, s, p);
}

template <typename A>
cudaError_t launch_act(int res, const NormParams& p, bool vec, cudaStream_t s) {
    switch (res) {
        case QX_F32: return launch_types<A, float>(p, vec, s);
        case QX_F16: return launch_types<A, __half>(p, vec, s);
        default: return launch_types<A, __nv_bfloat16>(p, vec, s);
    }
}

}  // namespace

cudaError_t launch_norm(int dtype, int res_dtype, const NormParams& p, bool vec, cudaStream_t s) {
    switch (dtype) {
        case QX_F32: return launch_act<float>(res_dtype, p, vec, s);
        case QX_F16: return launch_act<__half>(res_dtype, p, vec, s);
        default: return launch_act<__nv_bfloat16>(res_dtype, p, vec, s);
    }
}

}  // namespace qx
