// qx_layer_api.cu -- the C ABI of the operators between the weight products
// (include/qx.h): argument validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/qx.h"
#include "../../include/qx_debug.h"
#include "qx_internal.h"

namespace qx {
namespace {

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_bytes(int dtype) {
    switch (dtype) {
        case QX_F32: return 4;
        case QX_F16:
        case QX_BF16: return 2;
        default: return 0;
    }
}

// Strides stay far below the point where a token or page offset leaves 63 bits.
constexpr int64_t kMaxStride = int64_t(1) << 38;
bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

qx_status check_kv(const qx_kv* kv, KvView& v) {
    if (!kv || !kv->k || !kv->v || !kv->table || !kv->kv_len || !kv->q_start) return QX_ERR_ARG;
    if (kv->dtype != QX_F16 && kv->dtype != QX_BF16) return QX_ERR_FMT;
    if (kv->n_seqs < 1 || kv->n_heads < 1 || kv->n_heads > 65535 || kv->head_dim < 8 || kv->head_dim % 8 ||
        kv->head_dim > QX_MAX_HEAD_DIM || kv->n_pages < 1 || kv->n_pages > INT32_MAX || kv->table_stride < 1 ||
        kv->table_stride > (int64_t(1) << 31) || kv->page_size < 16 || kv->page_size > 65536 ||
        (kv->page_size & (kv->page_size - 1)))
        return QX_ERR_SHAPE;
    if (!stride_ok(kv->page_stride) || !stride_ok(kv->head_stride) || !stride_ok(kv->slot_stride)) return QX_ERR_SHAPE;
    // (the copy engine's maps take no overlapping or standing dimensions)
    if (kv->slot_stride < kv->head_dim || (kv->n_heads > 1 && kv->head_stride < kv->head_dim) ||
        (kv->n_pages > 1 && kv->page_stride < kv->head_dim))
        return QX_ERR_SHAPE;
    if (!on16(kv->k) || !on16(kv->v) || kv->page_stride % 8 || kv->head_stride % 8 || kv->slot_stride % 8)
        return QX_ERR_ALIGN;
    v.k = static_cast<char*>(kv->k);
    v.v = static_cast<char*>(kv->v);
    v.page_stride = kv->page_stride;
    v.head_stride = kv->head_stride;
    v.slot_stride = kv->slot_stride;
    v.table = kv->table;
    v.table_stride = kv->table_stride;
    v.kv_len = kv->kv_len;
    v.q_start = kv->q_start;
    v.n_seqs = kv->n_seqs;
    v.n_heads = kv->n_heads;
    v.head_dim = kv->head_dim;
    v.page_shift = 0;
    while ((1 << v.page_shift) < kv->page_size) ++v.page_shift;
    v.n_pages = int(kv->n_pages);
    v.err = nullptr;
    return QX_OK;
}

qx_status attention(const qx_kv* kv, const void* q, int64_t n_tokens, int n_q_heads, int64_t q_stride, float scale,
                    int64_t window, int64_t sinks, int64_t shared_len, void* out, qx_dtype out_dtype, float* lse,
                    void* scratch, qx_stream_t s) {
    AttnParams p = {};
    qx_status st = check_kv(kv, p.kv);
    if (st != QX_OK) return st;
    if (n_tokens < 0 || n_tokens > INT32_MAX / 2) return QX_ERR_SHAPE;
    if (n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % kv->n_heads || n_q_heads / kv->n_heads > QX_MAX_GROUP)
        return QX_ERR_SHAPE;
    if (!stride_ok(q_stride) || n_tokens * n_q_heads > INT32_MAX) return QX_ERR_SHAPE;
    if (window < 0 || sinks < 0 || shared_len < 0 || !std::isfinite(scale)) return QX_ERR_ARG;
    if (out_dtype != QX_F32 && out_dtype != kv->dtype) return QX_ERR_FMT;
    if (n_tokens == 0) return QX_OK;
    if (n_tokens > 1 && q_stride < int64_t(n_q_heads) * kv->head_dim) return QX_ERR_SHAPE;
    if (!q || !out || !scratch) return QX_ERR_ARG;
    if (!on16(q) || !on16(out) || q_stride % 8 || (reinterpret_cast<uintptr_t>(scratch) & 255u) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return QX_ERR_ALIGN;
    int sms = 0;
    if ((st = current_device(&sms, &p.kv.err)) != QX_OK) return st;
    p.q = q;
    p.q_stride = q_stride;
    p.out = out;
    p.lse = lse;
    p.n_tokens = int(n_tokens);
    p.n_q_heads = n_q_heads;
    p.out_f32 = out_dtype == QX_F32 ? 1 : 0;
    p.scale_log2 = float(double(scale) * 1.4426950408889634);
    p.window = window;
    p.sinks = sinks;
    p.shared_len = shared_len;
    p.scratch = scratch;
    return report_cuda(launch_attn(kv->dtype, p, sms, reinterpret_cast<cudaStream_t>(s)), "attention launch");
}

}  // namespace
}  // namespace qx

using namespace qx;

extern "C" {

qx_status qx_rope_append(const qx_kv* kv, const qx_qkv* in, const float* cos, const float* sin, int64_t n_pos,
                         int rot, int interleaved, void* q_out, qx_stream_t s) {
    RopeParams p = {};
    qx_status st = check_kv(kv, p.kv);
    if (st != QX_OK) return st;
    if (!in) return QX_ERR_ARG;
    const int eb = elem_bytes(in->dtype);
    if (eb == 0) return QX_ERR_FMT;
    if (in->n_tokens < 0 || in->n_tokens > INT32_MAX / 2 || in->n_q_heads < 0 || in->n_q_heads > 65535) return QX_ERR_SHAPE;
    if (rot < 0 || rot % 8 || rot > kv->head_dim || n_pos < 0 || n_pos > INT32_MAX) return QX_ERR_SHAPE;
    if (!stride_ok(in->q_stride) || !stride_ok(in->k_stride) || !stride_ok(in->v_stride)) return QX_ERR_SHAPE;
    if (in->n_tokens == 0) return QX_OK;
    if (!in->k || !in->v || (in->n_q_heads > 0 && (!in->q || !q_out)) || (rot > 0 && (!cos || !sin))) return QX_ERR_ARG;
    if (!on16(in->q) || !on16(in->k) || !on16(in->v) || !on16(cos) || !on16(sin) || !on16(q_out) || in->q_stride % 8 ||
        in->k_stride % 8 || in->v_stride % 8)
        return QX_ERR_ALIGN;
    int sms = 0;
    if ((st = current_device(&sms, &p.kv.err)) != QX_OK) return st;
    p.q = in->q;
    p.k = in->k;
    p.v = in->v;
    p.q_stride = in->q_stride;
    p.k_stride = in->k_stride;
    p.v_stride = in->v_stride;
    p.cos = cos;
    p.sin = sin;
    p.n_pos = n_pos;
    p.q_out = q_out;
    p.n_tokens = int(in->n_tokens);
    p.n_q_heads = in->n_q_heads;
    p.rot = rot;
    p.interleaved = interleaved ? 1 : 0;
    return report_cuda(launch_rope(in->dtype, kv->dtype, p, sms, reinterpret_cast<cudaStream_t>(s)), "rope launch");
}

qx_status qx_attn_paged(const qx_kv* kv, const void* q, int64_t n_tokens, int n_q_heads, int64_t q_stride,
                        float scale, int64_t window, int64_t sinks, void* out, qx_dtype out_dtype, float* lse,
                        void* scratch, qx_stream_t s) {
    return attention(kv, q, n_tokens, n_q_heads, q_stride, scale, window, sinks, 0, out, out_dtype, lse, scratch, s);
}

qx_status qx_attn_shared(const qx_kv* kv, const void* q, int64_t n_tokens, int n_q_heads, int64_t q_stride,
                         float scale, int64_t shared_len, void* out, qx_dtype out_dtype, float* lse, void* scratch,
                         qx_stream_t s) {
    return attention(kv, q, n_tokens, n_q_heads, q_stride, scale, 0, 0, shared_len, out, out_dtype, lse, scratch, s);
}

size_t qx_attn_scratch_bytes(int64_t n_tokens, int n_q_heads, int n_heads, int head_dim, int n_seqs) {
    if (n_tokens < 0 || n_tokens > INT32_MAX / 2 || n_heads < 1 || n_heads > 65535 || n_q_heads < 1 ||
        n_q_heads > 65535 || n_q_heads % n_heads || n_q_heads / n_heads > QX_MAX_GROUP || head_dim < 8 ||
        head_dim % 8 || head_dim > QX_MAX_HEAD_DIM || n_seqs < 1)
        return 0;
    return attn_scratch_bytes(n_tokens, n_q_heads, n_heads, head_dim, n_seqs);
}

uint64_t qx_stream_capture_id(qx_stream_t s) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(reinterpret_cast<cudaStream_t>(s), &status, &id) != cudaSuccess) {
        cudaGetLastError();  // (the legacy stream may not be asked while another one is captured)
        return 0;
    }
    return status == cudaStreamCaptureStatusActive ? id : 0;
}

qx_status qx_block_norm(const qx_norm_args* a, qx_stream_t s) {
    if (!a) return QX_ERR_ARG;
    const int eb = elem_bytes(a->dtype), rb = elem_bytes(a->res_dtype);
    if (eb == 0 || rb == 0) return QX_ERR_FMT;
    if (a->rows < 0 || a->rows > INT32_MAX || a->cols < 1 || a->cols > QX_MAX_COLS) return QX_ERR_SHAPE;
    if (!stride_ok(a->y_stride) || !stride_ok(a->r_stride) || !stride_ok(a->gate_stride) ||
        !stride_ok(a->r_out_stride) || !stride_ok(a->x_stride))
        return QX_ERR_SHAPE;
    if (a->rows == 0) return QX_OK;
    if (a->rows > 1) {
        // rows written over one another would race, in place over other rows' inputs too
        if ((a->r_out && a->r_out_stride < a->cols) || (a->x && a->x_stride < a->cols)) return QX_ERR_SHAPE;
        if ((a->r_out && a->r_out == a->r && a->r_out_stride != a->r_stride) || (a->x && a->x == a->y && a->x_stride != a->y_stride))
            return QX_ERR_SHAPE;
    }
    if (!a->r) return QX_ERR_ARG;
    if ((a->w_pre != nullptr) != (a->x != nullptr) || (!a->r_out && !a->x)) return QX_ERR_ARG;
    if (!a->y && (a->gate || a->w_post)) return QX_ERR_ARG;
    if (!(a->eps >= 0.0f) || !std::isfinite(a->eps) || !std::isfinite(a->alpha)) return QX_ERR_ARG;
    const auto whole = [](const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(bytes - 1)) == 0; };
    if (!whole(a->y, eb) || !whole(a->r, rb) || !whole(a->gate, eb) || !whole(a->w_post, 4) || !whole(a->w_pre, 4) ||
        !whole(a->r_out, rb) || !whole(a->x, eb))
        return QX_ERR_ALIGN;
    int sms = 0;
    unsigned* err = nullptr;
    const qx_status st = current_device(&sms, &err);
    if (st != QX_OK) return st;
    NormParams p = {};
    p.y = a->y;
    p.r = a->r;
    p.gate = a->gate;
    p.w_post = a->w_post;
    p.w_pre = a->w_pre;
    p.r_out = a->r_out;
    p.x = a->x;
    p.y_stride = a->y_stride;
    p.r_stride = a->r_stride;
    p.gate_stride = a->gate_stride;
    p.r_out_stride = a->r_out_stride;
    p.x_stride = a->x_stride;
    p.rows = a->rows;
    p.cols = int(a->cols);
    p.alpha = a->alpha;
    p.eps = a->eps;
    p.err = err;
    // 16-byte access: whole vectors of eight in every row of every operand.
    const bool vec = a->cols % 8 == 0 && on16(a->y) && on16(a->r) && on16(a->gate) && on16(a->w_post) &&
                     on16(a->w_pre) && on16(a->r_out) && on16(a->x) && a->y_stride % 8 == 0 && a->r_stride % 8 == 0 &&
                     a->gate_stride % 8 == 0 && a->r_out_stride % 8 == 0 && a->x_stride % 8 == 0;
    return report_cuda(launch_norm(a->dtype, a->res_dtype, p, vec, sms, reinterpret_cast<cudaStream_t>(s)), "norm launch");
}

qx_status qx_debug_agree_probe(uint64_t limit_ns, int32_t* got, qx_stream_t s) {
    if (!got || limit_ns < 1000000ull || limit_ns > 100000000ull) return QX_ERR_ARG;
    int sms = 0;
    unsigned* err = nullptr;
    const qx_status st = current_device(&sms, &err);
    if (st != QX_OK) return st;
    return report_cuda(launch_agree_probe(limit_ns, got, err, reinterpret_cast<cudaStream_t>(s)), "probe launch");
}

}  // extern "C"
