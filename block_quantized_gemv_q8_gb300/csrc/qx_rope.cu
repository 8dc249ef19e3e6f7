// qx_rope.cu -- keys and values appended to a paged cache, the position
// rotation applied to queries and keys on the way.
//
// A head's pair (a, b) turns by the angle whose cosine and sine the table
// holds for the token's position: a' = a c - b s, b' = b c + a s, in f32, one
// rounding to the cache's type.  The call reads each input element and writes
// each output element once, and is bound by those bytes: a thread takes eight
// elements of a head (four pairs), its input in 16-byte loads that go out before
// the token's sequence, position and page are looked up (61.0 -> 57.4 us).
// Measured: 9043 tokens of 32 + 2 x 8 heads of 128, f32 to bf16 (369 MB), 57.4
// us, 6.4 TB/s, 95 % of the measured copy rate; one token 2 us.
#include "qx_layer.cuh"

namespace qx {

namespace {

constexpr int kRopeThreads = 256;

template <typename S, typename D>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int t = blockIdx.x;
    const int per_head = p.kv.head_dim / 8;
    const int item = blockIdx.y * kRopeThreads + threadIdx.x;
    const int head = item / per_head, c = item - head * per_head;
    const int hkv = p.kv.n_heads;
    if (head >= p.n_q_heads + 2 * hkv) return;
    const int dim = p.kv.head_dim;
    const bool is_q = head < p.n_q_heads, is_v = head >= p.n_q_heads + hkv;
    const int h = is_q ? head : head - p.n_q_heads - (is_v ? hkv : 0);
    const S* src = (is_q   ? static_cast<const S*>(p.q) + t * p.q_stride
                    : is_v ? static_cast<const S*>(p.v) + t * p.v_stride
                           : static_cast<const S*>(p.k) + t * p.k_stride) + int64_t(h) * dim;
    const bool turns = !is_v && c * 8 < p.rot;
    // Half-split pairs: elements 4 c .. 4 c + 3 and their partners half a
    // rotation on; otherwise elements 8 c .. 8 c + 7.
    const bool split = turns && !p.interleaved;
    const int half = p.rot / 2;
    const int e0 = split ? 4 * c : 8 * c, e1 = split ? 4 * c + half : 8 * c + 4;
    float lo[4], hi[4], v[8];
    load_f32<4>(src + e0, lo);  // on their way while the token's place is looked up
    load_f32<4>(src + e1, hi);
    const int seq = seq_of_token(p.kv, t);
    if (seq < 0) return;
    const int64_t pos = position_of(p.kv, seq, t);
    // a position without angles: nothing of the token is written, turned or not
    if (p.rot > 0 && pos >= p.n_pos) {
        atomicOr(p.kv.err, kErrRange);
        return;
    }
    D* dst;
    if (is_q) {
        dst = static_cast<D*>(p.q_out) + (int64_t(t) * p.n_q_heads + head) * dim;
    } else {
        if (pos < 0) return;
        const int page = page_of(p.kv, seq, pos);
        if (page < 0) return;
        dst = reinterpret_cast<D*>(is_v ? p.kv.v : p.kv.k) + slot_offset(p.kv, page, h, pos);
    }
    if (pos < 0) {  // padding: a query row of zeros
#pragma unroll
        for (int i = 0; i < 4; ++i) lo[i] = hi[i] = 0.0f;
    } else if (turns) {
        float cs[4], sn[4];
        load_f32<4>(p.cos + pos * half + 4 * c, cs);
        load_f32<4>(p.sin + pos * half + 4 * c, sn);
        if (split) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = lo[i], b = hi[i];
                lo[i] = a * cs[i] - b * sn[i];
                hi[i] = b * cs[i] + a * sn[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float a = lo[2 * i], b = lo[2 * i + 1];
                lo[2 * i] = a * cs[i] - b * sn[i];
                lo[2 * i + 1] = b * cs[i] + a * sn[i];
                const float d = hi[2 * i], e = hi[2 * i + 1];
                hi[2 * i] = d * cs[i + 2] - e * sn[i + 2];
                hi[2 * i + 1] = e * cs[i + 2] + d * sn[i + 2];
            }
        }
    }
    if (split) {
        store_f32<4>(dst + e0, lo);
        store_f32<4>(dst + e1, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lo[i], v[i + 4] = hi[i];
        store_f32<8>(dst + e0, v);
    }
}

template <typename S>
cudaError_t launch_src(int dst, const RopeParams& p, cudaStream_t s) {
    const int items = (p.n_q_heads + 2 * p.kv.n_heads) * (p.kv.head_dim / 8);
    const dim3 grid(unsigned(p.n_tokens), unsigned((items + kRopeThreads - 1) / kRopeThreads));
    if (dst == QX_F16) return launch_serial(rope_append_kernel<S, __half>, grid, kRopeThreads, 0, s, p);
    return launch_serial(rope_append_kernel<S, __nv_bfloat16>, grid, kRopeThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_rope(int src, int dst, const RopeParams& p, int, cudaStream_t s) {
    switch (src) {
        case QX_F32: return launch_src<float>(dst, p, s);
        case QX_F16: return launch_src<__half>(dst, p, s);
        default: return launch_src<__nv_bfloat16>(dst, p, s);
    }
}

}  // namespace qx
