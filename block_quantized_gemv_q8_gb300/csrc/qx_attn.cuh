// qx_attn.cuh -- what the attention kernels share (qx_attn.cu, qx_attn_tc.cu).
#pragma once

#include <cuda.h>

#include <cfloat>

#include "qx_layer.cuh"

namespace qx {

template <typename T>
struct IsBf16 {
    static constexpr bool value = false;
};
template <>
struct IsBf16<__nv_bfloat16> {
    static constexpr bool value = true;
};

// The powers of two by which probabilities are raised before they are rounded
// to T, where the running maximum may be BEHIND the row's by so many (their sums
// are raised with them, and o / l stays as it is).  f16 holds up to 2^15 and
// loses bits below 2^-14: so raised, a probability keeps them down to 2^-29 of
// the row's largest (2^-26 with 3 behind).
template <typename T, int BEHIND>
constexpr float kLift = IsBf16<T>::value ? 0.0f : float(15 - BEHIND);

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// A row by a warp, on the plain units: a lane scores a key, then owns every 32nd
// element of the output.  m is the warp's maximum, l the lane's own sum.  The
// maximum begins at a number, so that no difference is inf - inf: fmaxf passes
// over scores that are no numbers, and those have to get into the sums.
template <int NE>
struct RowSums {
    float m = -FLT_MAX, l = 0.0f, o[NE] = {};
};
// 32 more keys of sequence seq, through key head hk: the lane's is j (below 0:
// none, and nothing of it is read); query(d, x) gives eight elements of the query.
// U: how far the loops are unrolled (1 where it is not what the kernel is for).
template <typename T, int U, int NE, typename Query>
__device__ __forceinline__ void row_keys(const AttnParams& p, int seq, int hk, int64_t j, const Query& query, RowSums<NE>& r) {
    const int lane = threadIdx.x & 31, dim = p.kv.head_dim;
    float s = -INFINITY;
    int64_t off = -1;
    if (j >= 0) {
        const int page = page_of(p.kv, seq, j);
        if (page >= 0) {
            off = slot_offset(p.kv, page, hk, j);
            const T* k = reinterpret_cast<const T*>(p.kv.k) + off;
            s = 0.0f;
#pragma unroll U
            for (int d = 0; d < dim; d += 8) {
                float kk[8], qq[8];
                load_f32<8>(k + d, kk);
                query(d, qq);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += qq[e] * kk[e];
            }
            s *= p.scale_log2;
        }
    }
    float mb = s;
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, w));
    const float mn = fmaxf(r.m, mb);
    const float a = exp2f(r.m - mn), pr = exp2f(s - mn);
    r.l = r.l * a + pr;
    r.m = mn;
#pragma unroll
    for (int e = 0; e < NE; ++e) r.o[e] *= a;
    // (loads under a condition, not past a branch: U keys' are in flight)
#pragma unroll U
    for (int g = 0; g < 32; ++g) {
        const float pg = __shfl_sync(0xffffffffu, pr, g);
        const int64_t og = __shfl_sync(0xffffffffu, off, g);
        const T* v = reinterpret_cast<const T*>(p.kv.v) + og;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const float x = og >= 0 && lane + 32 * e < dim ? to_f32(v[lane + 32 * e]) : 0.0f;
            r.o[e] += (og >= 0 ? pg : 0.0f) * x;
        }
    }
}
// The keys that the row at position pos sees of [from, to): 32 from `first` on
// and then every `step`.
template <typename T, int U, int NE, typename Query>
__device__ __forceinline__ void row_sums(const AttnParams& p, int seq, int64_t pos, int hk, int64_t from, int64_t to, int first, int step,
                                         const Query& query, RowSums<NE>& r) {
    int64_t lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;  // first key of the window
    if (lo < from) lo = from;
    const int64_t end = pos + 1 < to ? pos + 1 : to, sinks = p.sinks < lo ? p.sinks : lo;
    const int64_t n = sinks + (end > lo ? end - lo : 0);  // 0 .. sinks - 1, lo .. end - 1
    for (int64_t b = first; pos >= 0 && b < n; b += step) {
        const int64_t i = b + (threadIdx.x & 31);
        row_keys<T, U>(p, seq, hk, i < n ? (i < sinks ? i : lo + (i - sinks)) : -1, query, r);
    }
}

// A tile's values meet all of its rows, and 0 x a value that is infinite or no
// number is no number: a row that does not see that value gets one too.  Where an
// output shows that there is such a value, a warp looks for it among the keys
// that some row does not see, and makes the rows' o / l once more, over the keys
// that each sees alone.
//
// Whether 16 bytes hold an infinity or what is no number (an exponent of ones
// carries into its sign bit).
template <typename T>
__device__ __forceinline__ bool any_odd(uint4 v) {
    constexpr uint32_t kExp = sizeof(T) == 4 ? 0x7f800000u : IsBf16<T>::value ? 0x7f807f80u : 0x7c007c00u;
    constexpr uint32_t kOne = sizeof(T) == 4 ? 0x00800000u : IsBf16<T>::value ? 0x00800080u : 0x04000400u;
    constexpr uint32_t kSign = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
    return (((v.x & kExp) + kOne) | ((v.y & kExp) + kOne) | ((v.z & kExp) + kOne) | ((v.w & kExp) + kOne)) & kSign;
}
// Whether keys [from, to) of sequence seq, key head hk, have such values.
template <typename T, int DIM>
__device__ __forceinline__ bool odd_values(const AttnParams& p, int seq, int hk, int64_t from, int64_t to) {
    bool odd = false;
#pragma unroll 1
    for (int64_t i = from * (DIM / 8) + (threadIdx.x & 31); i < to * (DIM / 8); i += 32) {
        const int64_t j = i / (DIM / 8);
        const int page = page_of(p.kv, seq, j);
        if (page >= 0)
            odd |= any_odd<T>(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.kv.v) + slot_offset(p.kv, page, hk, j) + i % (DIM / 8) * 8));
    }
    return __any_sync(0xffffffffu, odd);
}
// A row's o / l to out (the output's type, or f32) from element `at` on.
template <typename T, int DIM>
__device__ __forceinline__ void write_row_again(RowSums<DIM / 32>& r, void* out, bool f32, int64_t at) {
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) r.l += __shfl_xor_sync(0xffffffffu, r.l, w);
#pragma unroll
    for (int e = 0; e < DIM / 32; ++e) {
        const int64_t to = at + 32 * e + (threadIdx.x & 31);
        const float v = r.l == 0.0f ? 0.0f : r.o[e] / r.l;
        if (f32) static_cast<float*>(out)[to] = v;
        else static_cast<T*>(out)[to] = from_f32<T>(v);
    }
}

// The copy engine's maps of a cache's keys and values as [pages][heads]
// [slots][dim], boxes of min(page, keys) slots x 64 elements, 128-byte swizzle.
bool encode_cache_maps(bool f16, const KvView& kv, int keys, CUtensorMap* k, CUtensorMap* v);

// Parts of every row, from calls that each saw some of its keys: o / l and
// the base-2 log of the sum, [parts][tokens * heads] (at most 32 parts).
struct JoinParams {
    AttnParams a;
    const float* part_o;
    const float* part_lse;
    int parts;
};

int64_t tc_pairs(int64_t n_tokens, int group, int n_seqs, bool prefix);
// The tokens' attention on the tensor cores: over all their keys (from
// shared_len on), or, `prefix`, over keys [0, shared_len) of the first
// sequence.  slots 0: every tile pair in one CTA; else (at least 3) the blocks
// of keys shared out evenly, rows leaving up to `slots` parts.  part_o null:
// written to the output.  counter: two words of scratch, zero between calls.
cudaError_t launch_attn_tc(int dtype, const AttnParams& a, bool prefix, int slots, float* part_o, float* part_lse,
                           unsigned* counter, int sm_count, cudaStream_t s);
cudaError_t launch_attn_join(int dtype, const JoinParams& p, cudaStream_t s);

}  // namespace qx
