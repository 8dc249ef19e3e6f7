// qx_norm.cu -- the norm after a block, its gate and residual scale, the
// residual sum and the norm before the next block, in one pass over the row.
//
//   u = y w_post / sqrt(mean(y^2) + eps);  r' = r + alpha gate u;
//   x = r' w_pre / sqrt(mean(r'^2) + eps)
//
// A CTA holds a row in registers between the two sums, so each element is read
// and written once: the call is bound by those bytes, and for few rows by the
// latency of the loads and the two block-wide sums.
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

// Many rows: the CTAs stay, each thread keeps its columns' weights, and rows
// come through a ring in shared memory by bulk copies, several ahead of the
// one being normed, so that the loads never wait for a sum.  (With one row a
// CTA the loads of an SM paused at every sum: 8192 x 4096, bf16 with an f32
// residual, took 84.5 us, 4.8 TB/s; with the ring 64.1 us, 6.3 TB/s, 93 % of
// the measured copy rate.  One row of 4096: 3 us.)
constexpr int kRowVecs = 2;  // vectors of eight a thread
template <typename A, typename R>
__global__ void __launch_bounds__(512) block_norm_rows_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float part[2][32];
    __shared__ uint64_t full[8];
    const bool y_row = p.y != nullptr, gate_row = p.gate != nullptr && p.gate_stride != 0;
    const uint32_t y_bytes = y_row ? p.cols * sizeof(A) : 0, r_bytes = p.cols * sizeof(R), g_bytes = gate_row ? p.cols * sizeof(A) : 0;
    const uint32_t stage_bytes = y_bytes + r_bytes + g_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t rows = p.rows, step = gridDim.x;
    int64_t next = blockIdx.x;  // the next row to fetch (thread 0)
    int fetched = 0;
    const auto fetch = [&](int stage) {
        if (next >= rows) return;
        uint8_t* to = smem + stage * stage_bytes;
        mbar_arrive_expect_tx(&full[stage], stage_bytes);
        if (y_row) bulk_g2s(to, static_cast<const A*>(p.y) + next * p.y_stride, y_bytes, &full[stage]);
        bulk_g2s(to + y_bytes, static_cast<const R*>(p.r) + next * p.r_stride, r_bytes, &full[stage]);
        if (gate_row) bulk_g2s(to + y_bytes + r_bytes, static_cast<const A*>(p.gate) + next * p.gate_stride, g_bytes, &full[stage]);
        next += step;
        ++fetched;
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < p.stages; ++i) fetch(i);
    float wa[kRowVecs][8], wb[kRowVecs][8];  // alpha * gate of all rows * w_post, and w_pre
#pragma unroll
    for (int n = 0; n < kRowVecs; ++n) {
        const int c = (n * blockDim.x + threadIdx.x) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) wa[n][i] = p.alpha, wb[n][i] = 0.0f;
        if (c >= p.cols) continue;
        float g[8];
        if (p.w_post) {
            load_f32<8>(p.w_post + c, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) wa[n][i] *= g[i];
        }
        if (p.gate && !gate_row) {
            load_f32<8>(static_cast<const A*>(p.gate) + c, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) wa[n][i] *= g[i];
        }
        if (p.w_pre) load_f32<8>(p.w_pre + c, wb[n]);
    }
    const float inv_cols = 1.0f / float(p.cols);
    int stage = 0, done = 0, turn = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t row = blockIdx.x; row < rows; row += step) {
        // (after a wait that ran out the rest runs through without waiting, for the barriers' sake)
        if (ok) ok = mbar_wait_bounded(&full[stage], phase, 2000000000ull, p.err, kErrTimeoutFull);
        done += ok;
        const uint8_t* at = smem + stage * stage_bytes;
        float u[kRowVecs][8], rr[kRowVecs][8], inv = 1.0f, s = 0.0f;
#pragma unroll
        for (int n = 0; n < kRowVecs; ++n) {
            const int c = (n * blockDim.x + threadIdx.x) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) u[n][i] = rr[n][i] = 0.0f;
            if (c >= p.cols) continue;
            load_f32<8>(reinterpret_cast<const R*>(at + y_bytes) + c, rr[n]);
            if (!y_row) continue;
            load_f32<8>(reinterpret_cast<const A*>(at) + c, u[n]);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += u[n][i] * u[n][i];
            if (gate_row) {
                float g[8];
                load_f32<8>(reinterpret_cast<const A*>(at + y_bytes + r_bytes) + c, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[n][i] *= g[i];
            }
        }
        // the row is in registers once every thread has arrived here: its
        // stage takes the row `stages` further
        // (without a second sum, the first one's buffers alternate)
        if (p.w_post) inv = 1.0f / sqrtf(block_sum(s, part[p.w_pre ? 0 : turn]) * inv_cols + p.eps);
        else __syncthreads();
        turn ^= 1;
        if (threadIdx.x == 0 && ok) fetch(stage);
        if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
        }
        s = 0.0f;
#pragma unroll
        for (int n = 0; n < kRowVecs; ++n) {
            const int c = (n * blockDim.x + threadIdx.x) * 8;
            if (c >= p.cols) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                rr[n][i] += u[n][i] * inv * wa[n][i];
                s += rr[n][i] * rr[n][i];
            }
            if (p.r_out) store_f32<8>(static_cast<R*>(p.r_out) + row * p.r_out_stride + c, rr[n]);
        }
        if (!p.w_pre) continue;
        const float inv2 = 1.0f / sqrtf(block_sum(s, part[1]) * inv_cols + p.eps);
#pragma unroll
        for (int n = 0; n < kRowVecs; ++n) {
            const int c = (n * blockDim.x + threadIdx.x) * 8;
            if (c >= p.cols) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) rr[n][i] *= inv2 * wb[n][i];
            store_f32<8>(static_cast<A*>(p.x) + row * p.x_stride + c, rr[n]);
        }
    }
    // after a wait that ran out: the copies in flight land before the CTA ends
    if (threadIdx.x == 0)
        for (; done < fetched; ++done)
            mbar_wait_bounded(&full[done % p.stages], (done / p.stages) & 1, 2000000000ull, p.err, kErrTimeoutDrain);
}

// The ring kernel's threads, stages and CTAs per SM, or false where it does not
// serve: rows of whole aligned vectors, at most 8192 columns; and not below 1536,
// where a CTA has too few warps to hide a row's sums behind another's (20000 x
// 1024: 44.8 us, a row a CTA 40.8; 3584 x 2048: 15.4 against 16.3).
template <typename A, typename R>
bool rows_geometry(const NormParams& p, int& threads, int& stages, int& per_sm, size_t& smem) {
    if (p.cols > 512 * 8 * kRowVecs || p.cols < 1536) return false;
    const size_t stage = size_t(p.cols) * ((p.y ? sizeof(A) : 0) + sizeof(R) + (p.gate && p.gate_stride ? sizeof(A) : 0));
    threads = (p.cols / 8 + kRowVecs - 1) / kRowVecs;
    threads = (threads + 31) / 32 * 32;
    per_sm = 512 / threads < 16 ? 512 / threads : 16;  // 128 registers a thread
    const size_t room = 224 * 1024 / per_sm - 1536;
    if (3 * stage > room) return false;
    stages = int(room / stage < 8 ? room / stage : 8);
    while (stages > 3 && stages * stage * per_sm > 160 * 1024) --stages;  // more in flight gains nothing
    smem = stages * stage;
    return true;
}

template <typename A, typename R>
cudaError_t launch_rows(NormParams p, int threads, int stages, int per_sm, size_t smem, int sm_count, cudaStream_t s) {
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(block_norm_rows_kernel<A, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    p.stages = stages;
    const int64_t ctas = int64_t(per_sm) * sm_count;
    return launch_serial(block_norm_rows_kernel<A, R>, dim3(unsigned(p.rows < ctas ? p.rows : ctas)), threads, smem, s, p);
}

template <typename A, typename R>
cudaError_t launch_types(const NormParams& p, bool vec, int sm_count, cudaStream_t s) {
    int threads_r, stages, per_sm;
    size_t smem;
    if (vec && rows_geometry<A, R>(p, threads_r, stages, per_sm, smem) && p.rows >= 2 * int64_t(per_sm) * sm_count)
        return launch_rows<A, R>(p, threads_r, stages, per_sm, smem, sm_count, s);
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
cudaError_t launch_act(int res, const NormParams& p, bool vec, int sm_count, cudaStream_t s) {
    switch (res) {
        case QX_F32: return launch_types<A, float>(p, vec, sm_count, s);
        case QX_F16: return launch_types<A, __half>(p, vec, sm_count, s);
        default: return launch_types<A, __nv_bfloat16>(p, vec, sm_count, s);
    }
}

}  // namespace

cudaError_t launch_norm(int dtype, int res_dtype, const NormParams& p, bool vec, int sm_count, cudaStream_t s) {
    switch (dtype) {
        case QX_F32: return launch_act<float>(res_dtype, p, vec, sm_count, s);
        case QX_F16: return launch_act<__half>(res_dtype, p, vec, sm_count, s);
        default: return launch_act<__nv_bfloat16>(res_dtype, p, vec, sm_count, s);
    }
}

}  // namespace qx
