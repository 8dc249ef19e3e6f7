// qx_attn.cu -- attention over the paged cache.
//
// Row (token t, query head h) at position pos: with s_j = scale q . k_j over
// the keys it sees, m the running maximum, l the running sum of exp(s_j - m)
// and o the running sum of exp(s_j - m) v_j, a block of keys with maximum m'
// turns (m, l, o) into (M, l e^(m-M) + sum e^(s_j-M), o e^(m-M) + ...), M =
// max(m, m'); the output is o / l.  Exponents are taken to base 2 with
// scale * log2(e) folded into the scores.
#include "qx_layer.cuh"

namespace qx {

namespace {

constexpr int kRowWarps = 4;
constexpr int kMaxDim = QX_MAX_HEAD_DIM;

// Any head size: one CTA per row, its warps taking blocks of 32 keys in turn
// (a lane scores a key, then owns every 32nd output element), joined at the
// end.
template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps) attn_row_kernel(const __grid_constant__ AttnParams p) {
    __shared__ float q[kMaxDim];
    __shared__ float om[kRowWarps], ol[kRowWarps], oo[kRowWarps][kMaxDim];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int t = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dim = p.kv.head_dim, hk = h / (p.n_q_heads / p.kv.n_heads);
    const int seq = seq_of_token(p.kv, t);
    if (seq < 0) return;
    const int64_t pos = position_of(p.kv, seq, t);
    const T* qr = static_cast<const T*>(p.q) + t * p.q_stride + int64_t(h) * dim;
    for (int d = threadIdx.x; d < dim; d += 32 * kRowWarps) q[d] = to_f32(qr[d]);
    __syncthreads();
    const int64_t lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;  // first key of the window
    const int64_t sinks = p.sinks < lo ? p.sinks : lo;
    float m = -INFINITY, l = 0.0f, o[kMaxDim / 32];
#pragma unroll
    for (int i = 0; i < kMaxDim / 32; ++i) o[i] = 0.0f;
    const int64_t n = pos < 0 ? 0 : sinks + (pos + 1 - lo);  // keys seen: 0 .. sinks - 1, lo .. pos
    for (int64_t b = 32 * warp; b < n; b += 32 * kRowWarps) {
        const int64_t i = b + lane;
        const int64_t j = i < sinks ? i : lo + (i - sinks);
        float s = -INFINITY;
        int64_t off = -1;
        if (i < n) {
            const int page = page_of(p.kv, seq, j);
            if (page >= 0) {
                off = slot_offset(p.kv, page, hk, j);
                const T* k = reinterpret_cast<const T*>(p.kv.k) + off;
                s = 0.0f;
                for (int d = 0; d < dim; d += 8) {
                    float kk[8];
                    load_f32<8>(k + d, kk);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s += q[d + e] * kk[e];
                }
                s *= p.scale_log2;
            }
        }
        float mb = s;
#pragma unroll
        for (int w = 16; w >= 1; w >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, w));
        const float mn = fmaxf(m, mb);
        if (mn == -INFINITY) continue;
        const float a = exp2f(m - mn), pr = exp2f(s - mn);
        l = l * a + pr;
        m = mn;
#pragma unroll
        for (int e = 0; e < kMaxDim / 32; ++e) o[e] *= a;
        for (int g = 0; g < 32; ++g) {
            const float pg = __shfl_sync(0xffffffffu, pr, g);
            const int64_t og = __shfl_sync(0xffffffffu, off, g);
            if (og < 0) continue;
            const T* v = reinterpret_cast<const T*>(p.kv.v) + og;
#pragma unroll
            for (int e = 0; e < kMaxDim / 32; ++e)
                if (lane + 32 * e < dim) o[e] += pg * to_f32(v[lane + 32 * e]);
        }
    }
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    if (lane == 0) om[warp] = m, ol[warp] = l;
#pragma unroll
    for (int e = 0; e < kMaxDim / 32; ++e)
        if (lane + 32 * e < dim) oo[warp][lane + 32 * e] = o[e];
    __syncthreads();
    float M = -INFINITY, L = 0.0f, a[kRowWarps];
    for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, om[w]);
    for (int w = 0; w < kRowWarps; ++w) {
        a[w] = om[w] == -INFINITY ? 0.0f : exp2f(om[w] - M);
        L += a[w] * ol[w];
    }
    const int64_t row = int64_t(t) * p.n_q_heads + h;
    if (p.lse && threadIdx.x == 0) p.lse[row] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    for (int d = threadIdx.x; d < dim; d += 32 * kRowWarps) {
        float v = 0.0f;
        for (int w = 0; w < kRowWarps; ++w) v += a[w] * oo[w][d];
        v = L > 0.0f ? v / L : 0.0f;
        if (p.out_f32) static_cast<float*>(p.out)[row * dim + d] = v;
        else static_cast<T*>(p.out)[row * dim + d] = from_f32<T>(v);
    }
}

template <typename T>
cudaError_t launch_row(const AttnParams& p, cudaStream_t s) {
    return launch_serial(attn_row_kernel<T>, dim3(unsigned(p.n_tokens), unsigned(p.n_q_heads)), 32 * kRowWarps, 0, s, p);
}

}  // namespace

cudaError_t launch_attn(int dtype, const AttnParams& p, int, cudaStream_t s) {
    return dtype == QX_F16 ? launch_row<__half>(p, s) : launch_row<__nv_bfloat16>(p, s);
}

}  // namespace qx
