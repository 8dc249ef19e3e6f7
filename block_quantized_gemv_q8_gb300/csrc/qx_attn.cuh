// qx_attn.cuh -- what the attention kernels share (qx_attn.cu, qx_attn_tc.cu).
#pragma once

#include <cuda.h>

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
// the row's largest (2^-27 with 2 behind).
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
