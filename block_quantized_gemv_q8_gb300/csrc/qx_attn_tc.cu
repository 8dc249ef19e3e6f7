// qx_attn_tc.cu -- attention of many rows a key head on the fifth-generation
// tensor cores: prefill chunks, and a shared prefix against a whole batch.
//
// A CTA takes 256 rows of one key head -- two tiles of 128, each as many
// tokens as fit with all query heads of the group -- against blocks of 128
// keys.  Per tile and block: S = Q K^T (tcgen05, operands in shared memory, S
// in tensor memory), softmax in registers by the tile's own warpgroup (one
// thread a row), P in the cache's type written over S, and O += P V (P read
// from tensor memory, O kept there).  While one tile's warpgroup works on its
// softmax, the tensor cores work for the other tile.  A key block is fetched
// once for both tiles (TMA, one box a page, 128-byte swizzle; V is the
// MN-major operand as it lies).
//
// O is rescaled by the warp that owns its rows, and only when a row's maximum
// rose by more than kRescale powers of two: until then the old maximum stays
// the base, P at most 2^kRescale, which both 16-bit types and the f32 sums
// hold without loss.  The maximum, the sum of the unrounded exponentials and O
// are f32.
//
// Work per block of 128 keys and tile: 2 x 128 x 128 x head_dim multiply-adds
// against 128 x 128 exponentials: the tensor cores and the softmax warps take
// about the same time, and which of them bounds depends on the head size.
//
// A row's keys may be split over several CTAs (few rows, long context); each
// part then leaves o / l and the base-2 log of its sum, which
// attn_join_kernel joins.  Every wait is bounded and reports through the
// device error word.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>
#include <mutex>

#include "qx_attn.cuh"
#include "qx_layer.cuh"

namespace qx {

namespace {

constexpr int kKeys = 128;             // keys of a block
constexpr int kTileRows = 128;         // rows of a tile; two tiles a CTA
constexpr int kSoftmaxWarps = 8;       // two warpgroups
// A third warpgroup: the MMA issuer, the producer, and two warps that only
// give up registers.  An SM partition holds three of the CTA's warps, so 168
// registers a thread at launch; the softmax warps hold a row of S each.
constexpr int kTcThreads = 32 * (kSoftmaxWarps + 4);
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "registers the CTA was launched with");
constexpr float kRescale = 8.0f;
constexpr unsigned long long kWaitNs = 2000000000ull;

template <int DIM>
struct TcGeom {
    static constexpr int kPanels = DIM / 64;                    // 64 elements (128 bytes) of every row
    static constexpr int kPanelBytes = 128 * 128;               // 128 rows
    static constexpr int kTileBytes = kPanels * kPanelBytes;    // Q of a tile, or a block's K or V
    static constexpr int kSlots = DIM == 128 ? 5 : 10;          // ring of K and V blocks
    static constexpr size_t kSmem = size_t(2 + kSlots) * kTileBytes + 1024 + 256;
};
static_assert(TcGeom<128>::kSmem <= 227 * 1024 && TcGeom<64>::kSmem <= 227 * 1024, "a CTA's shared memory");

struct TcAttnParams {
    CUtensorMap q_map;  // [tokens][heads][dim], boxes of one tile's tokens x the group x 64
    CUtensorMap k_map;  // [pages][heads][slots][dim], boxes of min(page, 128) keys x 64
    CUtensorMap v_map;
    AttnParams a;
    int tile_tokens;    // tokens of a tile: 128 / group
    int splits;         // CTAs that share a tile pair's keys
    int prefix;         // 1: every token against keys [0, shared_len)
    float* part_o;      // parts: [splits][tokens * heads][dim], or null: write the output
    float* part_lse;    // [splits][tokens * heads]
};

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major: rows of 128
// bytes (64 elements), 8-row atoms 1024 bytes apart.  MN-major: 64 elements of
// one key in 128 bytes, atoms of 8 keys 1024 bytes apart along the keys and
// `panel` bytes apart along the head.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t panel) {
    uint64_t d = 0;
    d |= uint64_t((saddr & 0x3FFFF) >> 4);
    d |= uint64_t(panel >> 4) << 16;  // leading byte offset (used by MN-major)
    d |= uint64_t(1024 >> 4) << 32;   // stride byte offset
    d |= uint64_t(1) << 46;           // descriptor version
    d |= uint64_t(2) << 61;           // 128-byte swizzle
    return d;
}
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool b_mn_major) {
    const uint32_t fmt = sizeof(T) == 2 && IsBf16<T>::value ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) |
           (uint32_t(kTileRows >> 4) << 24);
}

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// 32 columns of the warp's 32 rows, no wait.
__device__ __forceinline__ void ld32(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const float* r) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
        "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
        "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}

// What a CTA works on: `tokens` tokens from t0 on (at most two tiles) of
// sequence b, the first at position pos0, and the key blocks that any of its
// rows sees: those of keys [0, sinks), then those of [lo, end).
struct TcWork {
    int b, t0, tokens, pos0, lo, end, sinks, sink_blocks, blocks;
};
__device__ __forceinline__ int key_block(const TcWork& w, int i) {  // first key of the i-th block
    return (i < w.sink_blocks ? i : w.lo / kKeys + (i - w.sink_blocks)) * kKeys;
}
__device__ __forceinline__ void key_range(const TcWork& w, int i, int& lo, int& hi) {  // keys of it that some row sees
    lo = i < w.sink_blocks ? 0 : w.lo;
    hi = i < w.sink_blocks ? w.sinks : w.end;
}

// The tile pair with the given number, counted over all sequences (a sequence
// of n tokens has ceil(n / pair)); false: there is none.  One warp finds it,
// 32 sequences at a time.
__device__ __forceinline__ bool find_pair(const TcAttnParams& p, int number, int lane, TcWork& w) {
    const KvView& kv = p.a.kv;
    const int pair = 2 * p.tile_tokens;
    const int total = kv.q_start[kv.n_seqs] < p.a.n_tokens ? kv.q_start[kv.n_seqs] : p.a.n_tokens;
    if (p.prefix) {
        w.b = 0;
        w.t0 = number * pair;
        w.tokens = total - w.t0 < pair ? total - w.t0 : pair;
        if (w.tokens <= 0) return false;
        w.pos0 = 0;
        w.lo = w.sinks = w.sink_blocks = 0;
        const int64_t most = kv.table_stride << kv.page_shift;
        w.end = int(p.a.shared_len < most ? p.a.shared_len : most);
        w.blocks = (w.end + kKeys - 1) / kKeys;
        return true;
    }
    int base = 0;
    for (int b0 = 0; b0 < kv.n_seqs; b0 += 32) {
        const int b = b0 + lane;
        int n = 0, t0 = 0;
        if (b < kv.n_seqs) {
            t0 = kv.q_start[b];
            n = kv.q_start[b + 1] - t0;
            if (n < 0 || t0 < 0 || t0 + n > p.a.n_tokens) n = 0;
        }
        const int tiles = (n + pair - 1) / pair;
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, number < base + incl);
        if (hit == 0) {
            base += __shfl_sync(0xffffffffu, incl, 31);
            continue;
        }
        const int src = __ffs(hit) - 1;
        const int before = base + __shfl_sync(0xffffffffu, incl - tiles, src);
        n = __shfl_sync(0xffffffffu, n, src);
        t0 = __shfl_sync(0xffffffffu, t0, src);
        const int tile = number - before;
        w.b = b0 + src;
        w.t0 = t0 + tile * pair;
        w.tokens = n - tile * pair < pair ? n - tile * pair : pair;
        const int64_t len = kv.kv_len[w.b], most = kv.table_stride << kv.page_shift;
        if (len > most) atomicOr(kv.err, kErrRange);
        const int64_t pos0 = len - n + tile * pair;
        int64_t end = pos0 + w.tokens;  // one past the last token's position
        if (end > most) end = most;
        if (end < 0) end = 0;
        int64_t lo = p.a.window > 0 && pos0 + 1 > p.a.window ? pos0 + 1 - p.a.window : 0;
        int64_t sinks = p.a.sinks < lo ? p.a.sinks : lo;
        if (p.a.shared_len > 0) sinks = 0, lo = lo > p.a.shared_len ? lo : p.a.shared_len;
        if (sinks > end) sinks = end;
        if (lo > end) lo = end;
        w.pos0 = int(pos0);
        w.end = int(end);
        w.lo = int(lo);
        w.sinks = int(sinks);
        w.sink_blocks = (w.sinks + kKeys - 1) / kKeys;
        w.blocks = w.sink_blocks + (w.end > w.lo ? (w.end + kKeys - 1) / kKeys - w.lo / kKeys : 0);
        return true;
    }
    return false;
}

// Every lane of the warp waits itself, and the outcome is warp-uniform.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned* err, unsigned code) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitNs, err, code));
}

template <typename T, int DIM>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const __grid_constant__ TcAttnParams p) {
    using G = TcGeom<DIM>;
    constexpr int NS = G::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    uint8_t* sq = smem;                        // [2 tiles][panels][128 rows][128 B]
    uint8_t* ring = sq + 2 * G::kTileBytes;    // [NS] blocks: K0, V0, K1, V1, ...
    uint64_t* q_full = reinterpret_cast<uint64_t*>(ring + NS * G::kTileBytes);
    uint64_t* kv_full = q_full + 1;
    uint64_t* kv_empty = kv_full + NS;
    uint64_t* s_full = kv_empty + NS;   // per tile
    uint64_t* p_full = s_full + 2;
    uint64_t* o_full = p_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const KvView& kv = p.a.kv;
    const int hk = blockIdx.x % kv.n_heads;
    TcWork w;
    // the pairs with the most keys (the last of a sequence) first
    const int number = int(gridDim.x / kv.n_heads) - 1 - int(blockIdx.x / kv.n_heads);
    if (!find_pair(p, number, lane, w)) return;
    const int i0 = int(int64_t(w.blocks) * int(blockIdx.y) / p.splits);
    const int i1 = int(int64_t(w.blocks) * (int(blockIdx.y) + 1) / p.splits);
    const int nb = i1 - i0;  // this CTA's blocks
    const int group = p.a.n_q_heads / kv.n_heads;
    const int tiles = w.tokens > p.tile_tokens ? 2 : 1;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
        }
        fence_barrier_init();
    }
    if (warp == kSoftmaxWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem, tO = tmem + 256;  // S (and P) of tile t at 128 t, O at 256 + 128 t

    if (warp >= kSoftmaxWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    if (warp == kSoftmaxWarps + 1) {
        // ---- producer: Q, then K and V of each block
        const int page_keys = (1 << kv.page_shift) < kKeys ? (1 << kv.page_shift) : kKeys;
        const int boxes = kKeys / page_keys;  // of a block (at most 8)
        if (nb > 0 && lane == 0) {
            mbar_arrive_expect_tx(q_full, tiles * G::kPanels * p.tile_tokens * group * 128);
            for (int t = 0; t < tiles; ++t)
                for (int c = 0; c < G::kPanels; ++c)
                    tma_3d(sq + t * G::kTileBytes + c * G::kPanelBytes, &p.q_map, 64 * c, hk * group, w.t0 + t * p.tile_tokens, q_full);
        }
        int issued = 0;
        for (int i = 0; i < 2 * nb; ++i) {
            const int slot = i % NS;
            // lane x of the first `boxes` finds the page of its box
            const int j0 = key_block(w, i0 + (i >> 1));
            int lo, hi;
            key_range(w, i0 + (i >> 1), lo, hi);
            int page = -1;
            if (lane < boxes) {
                const int j = j0 + lane * page_keys;
                if (j + page_keys > lo && j < hi) page = page_of(kv, w.b, j);
            }
            const unsigned live = __ballot_sync(0xffffffffu, page >= 0);
            if (i >= NS && !warp_wait(&kv_empty[slot], ((i / NS) - 1) & 1, kv.err, kErrTimeoutEmpty)) break;
            if (lane == 0) mbar_arrive_expect_tx(&kv_full[slot], __popc(live) * page_keys * 128 * G::kPanels);
            __syncwarp();
            if (page >= 0) {
                const int in_page = (j0 + lane * page_keys) & ((1 << kv.page_shift) - 1);
                uint8_t* dst = ring + slot * G::kTileBytes + lane * page_keys * 128;
                for (int c = 0; c < G::kPanels; ++c)
                    tma_4d(dst + c * G::kPanelBytes, (i & 1) ? &p.v_map : &p.k_map, 64 * c, in_page, hk, page, &kv_full[slot]);
            }
            issued = i + 1;
        }
        // keep the CTA alive until every copy it issued has landed
        if (lane == 0) {
            if (nb > 0) mbar_wait_bounded(q_full, 0, kWaitNs, kv.err, kErrTimeoutDrain);
            for (int i = issued > NS ? issued - NS : 0; i < issued; ++i)
                mbar_wait_bounded(&kv_full[i % NS], (i / NS) & 1, kWaitNs, kv.err, kErrTimeoutDrain);
        }
    } else if (warp == kSoftmaxWarps) {
        // ---- MMA issuer (the whole warp waits; lane 0 issues)
        bool ok = nb > 0 && warp_wait(q_full, 0, kv.err, kErrTimeoutMma);
        const uint32_t qa = smem_addr(sq), ra = smem_addr(ring);
        const auto scores = [&](int t, int i) {  // S of tile t against block i (its K is in ring position 2 i)
            const uint32_t ka = ra + ((2 * i) % NS) * G::kTileBytes;
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < DIM / 16; ++k) {
                    const uint32_t off = (k >> 2) * G::kPanelBytes + (k & 3) * 32;
                    mma_ss(tS + 128 * t, sw128_desc(qa + t * G::kTileBytes + off, 16), sw128_desc(ka + off, 16),
                           idesc<T>(kKeys, false), k > 0 ? 1u : 0u);
                }
                commit(&s_full[t]);
            }
            __syncwarp();
        };
        if (ok) ok = warp_wait(&kv_full[0], 0, kv.err, kErrTimeoutMma);
        if (ok) {
            tc_after();
            for (int t = 0; t < tiles; ++t) scores(t, 0);
            if (lane == 0) commit(&kv_empty[0]);
        }
        for (int i = 0; i < nb && ok; ++i) {
            const int vs = (2 * i + 1) % NS, ks = (2 * i + 2) % NS;
            const uint32_t va = ra + vs * G::kTileBytes;
            if (!(ok = warp_wait(&kv_full[vs], ((2 * i + 1) / NS) & 1, kv.err, kErrTimeoutMma))) break;
            // Values that no row sees are zeroed: whatever the slots hold, 0 x it must be 0.
            int lo, hi;
            key_range(w, i0 + i, lo, hi);
            const int j0 = key_block(w, i0 + i);
            if (j0 < lo || j0 + kKeys > hi) {
                for (int r = lane; r < kKeys; r += 32)
                    if (j0 + r < lo || j0 + r >= hi)
                        for (int c = 0; c < G::kPanels; ++c)
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                *reinterpret_cast<uint4*>(ring + vs * G::kTileBytes + c * G::kPanelBytes + r * 128 + 16 * x) =
                                    make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (i + 1 < nb && !(ok = warp_wait(&kv_full[ks], ((2 * i + 2) / NS) & 1, kv.err, kErrTimeoutMma))) break;
            for (int t = 0; t < tiles; ++t) {
                if (!(ok = warp_wait(&p_full[t], i & 1, kv.err, kErrTimeoutMma))) break;
                tc_after();
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        mma_ts(tO + 128 * t, tS + 128 * t + 8 * k, sw128_desc(va + k * 2048, G::kPanelBytes), idesc<T>(DIM, true),
                               (i | k) > 0 ? 1u : 0u);
                    commit(&o_full[t]);
                }
                __syncwarp();
                if (i + 1 < nb) scores(t, i + 1);
            }
            if (ok && lane == 0) {
                commit(&kv_empty[vs]);
                if (i + 1 < nb) commit(&kv_empty[ks]);
            }
            __syncwarp();
        }
    } else if (warp < kSoftmaxWarps) {
        // ---- softmax: one thread a row
        const int t = warp >> 2;  // tile
        const int r = 32 * (warp & 3) + lane;
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        const uint32_t sa = tS + 128 * t + lanes, oa = tO + 128 * t + lanes;
        const int in_tile = r / group, tok = t * p.tile_tokens + in_tile;
        const bool live = in_tile < p.tile_tokens && tok < w.tokens;
        int pos = -1;
        if (live) {
            if (p.prefix) {
                const int seq = seq_of_token(kv, w.t0 + tok);
                pos = seq < 0 ? -1 : int(position_of(kv, seq, w.t0 + tok));
            } else {
                pos = w.pos0 + tok;
            }
        }
        const int window = p.a.window > 0 && p.a.window < INT32_MAX ? int(p.a.window) : INT32_MAX;
        const int sinks = p.a.sinks < INT32_MAX ? int(p.a.sinks) : INT32_MAX;
        const int wlo = pos >= window ? pos - window + 1 : 0;  // first key of this row's window
        float m = -INFINITY, l = 0.0f;
        bool ok = t < tiles;
        for (int i = 0; i < nb && ok; ++i) {
            if (!(ok = warp_wait(&s_full[t], i & 1, kv.err, kErrTimeoutMma))) break;
            tc_after();
            float s[kKeys];
#pragma unroll
            for (int c = 0; c < 4; ++c) ld32(sa + 32 * c, s + 32 * c);
            wait_ld();
            const int j0 = key_block(w, i0 + i);
            int lo, hi;
            key_range(w, i0 + i, lo, hi);
            const bool sink = i0 + i < w.sink_blocks;
            const int first = sink ? 0 : (wlo > lo ? wlo : lo), last = (pos < hi - 1 ? pos : hi - 1);  // the row sees [first, last]
            if (__any_sync(0xffffffffu, first > j0 || last < j0 + kKeys - 1)) {
                // and, in a window block, sinks that the tile's first row has in its window
                const int a = first - j0, b = last - j0, c0 = lo - j0, c1 = sinks - j0;
#pragma unroll
                for (int x = 0; x < kKeys; ++x)
                    if (!((x >= a || (x >= c0 && x < c1)) && x <= b)) s[x] = -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int x = 4; x < kKeys; ++x) mx[x & 3] = fmaxf(mx[x & 3], s[x]);
            // base-2 scores: the maximum of s scale is scale times the maximum, or the minimum for a negative scale
            float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.a.scale_log2;
            if (p.a.scale_log2 <= 0.0f) {
                // a rare sign: scaled scores instead (masked ones stay at -inf)
                top = -INFINITY;
#pragma unroll
                for (int x = 0; x < kKeys; ++x) {
                    s[x] = s[x] == -INFINITY ? -INFINITY : s[x] * p.a.scale_log2;
                    top = fmaxf(top, s[x]);
                }
            }
            const float f = p.a.scale_log2 <= 0.0f ? 1.0f : p.a.scale_log2;
            if (__any_sync(0xffffffffu, top > m + kRescale || (m == -INFINITY && top > m))) {
                const float mn = fmaxf(m, top);
                const float a = mn == -INFINITY ? 1.0f : exp2_approx(m - mn);
                l *= a;
                m = mn;
                if (i > 0) {
                    if (!(ok = warp_wait(&o_full[t], (i - 1) & 1, kv.err, kErrTimeoutMma))) break;
                    tc_after();
#pragma unroll
                    for (int c = 0; c < DIM / 32; ++c) {
                        float o[32];
                        ld32(oa + 32 * c, o);
                        wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] *= a;
                        st32(oa + 32 * c, o);
                    }
                    wait_st();
                }
            }
            const float base = m == -INFINITY ? 0.0f : m;
            const uint64_t f2 = f32x2_pack(f, f), b2 = f32x2_pack(-base, -base);
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t u[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float2 e = f32x2_unpack(f32x2_fma(f32x2_pack(s[32 * c + 2 * x], s[32 * c + 2 * x + 1]), f2, b2));
                    const float e0 = exp2_approx(e.x), e1 = exp2_approx(e.y);
                    sum[x & 1] = f32x2_add(sum[x & 1], f32x2_pack(e0, e1));
                    u[x] = pack2<T>(e0, e1);
                }
                st16(sa + 16 * c, u);
            }
            const float2 s01 = f32x2_unpack(f32x2_add(sum[0], sum[1]));
            l += s01.x + s01.y;
            wait_st();
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[t]);
        }
        // ---- output
        if (t < tiles && ok && nb > 0) {
            ok = warp_wait(&o_full[t], (nb - 1) & 1, kv.err, kErrTimeoutMma);
            tc_after();
        }
        if (t < tiles && ok) {
            const int64_t row = int64_t(w.t0 + tok) * p.a.n_q_heads + hk * group + r % group;
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            const float lse2 = l > 0.0f ? m + log2f(l) : -INFINITY;
            const int64_t part = int64_t(blockIdx.y) * p.a.n_tokens * p.a.n_q_heads + row;
            if (live) {
                if (p.part_o) p.part_lse[part] = lse2;
                else if (p.a.lse) p.a.lse[row] = lse2 * 0.6931471805599453f;
            }
#pragma unroll
            for (int c = 0; c < DIM / 32; ++c) {
                float o[32];
                if (nb > 0) {
                    ld32(oa + 32 * c, o);
                    wait_ld();
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = l > 0.0f ? o[x] * inv : 0.0f;
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = 0.0f;
                }
                if (!live) continue;
                if (p.part_o) store_f32<32>(p.part_o + part * DIM + 32 * c, o);
                else if (p.a.out_f32) store_f32<32>(static_cast<float*>(p.a.out) + row * DIM + 32 * c, o);
                else store_f32<32>(static_cast<T*>(p.a.out) + row * DIM + 32 * c, o);
            }
        }
    }
    tc_before();
    __syncthreads();
    if (warp == kSoftmaxWarps)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Join the parts of a row: out = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M).
// A warp a row; the parts are few and their sum's order fixed.
template <typename T, int DIM>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ JoinParams p) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    constexpr int V = DIM / 32;
    const int64_t rows = int64_t(p.a.n_tokens) * p.a.n_q_heads;
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    if (seq_of_token(p.a.kv, int(row / p.a.n_q_heads)) < 0) return;
    const float mine = lane < p.parts ? p.part_lse[lane * rows + row] : -INFINITY;
    float M = mine;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float wt = mine == -INFINITY ? 0.0f : exp2_approx(mine - M);
    float L = wt;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float acc[V] = {};
    for (int i = 0; i < p.parts; ++i) {
        const float c = __shfl_sync(0xffffffffu, wt, i);
        const float* src = p.part_o + (i * rows + row) * DIM + V * lane;
        if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            acc[0] += c * v.x, acc[1] += c * v.y, acc[2] += c * v.z, acc[3] += c * v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            acc[0] += c * v.x, acc[1] += c * v.y;
        }
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
    for (int x = 0; x < V; ++x) acc[x] *= inv;
    if (p.a.lse && lane == 0) p.a.lse[row] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    if (p.a.out_f32) {
        float* dst = static_cast<float*>(p.a.out) + row * DIM + V * lane;
        if constexpr (V == 4) *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
    } else {
        T* dst = static_cast<T*>(p.a.out) + row * DIM + V * lane;
        if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(acc[0], acc[1]), pack2<T>(acc[2], acc[3]));
        else *reinterpret_cast<uint32_t*>(dst) = pack2<T>(acc[0], acc[1]);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// A 16-bit tensor, dims[0] contiguous, strides in elements; boxes of box[] in
// 128-byte swizzle.  A dimension of one element may have any stride: it is
// given a valid one.
bool encode(CUtensorMap* m, bool f16, const void* ptr, int rank, const int64_t* dims, const int64_t* strides, const int* box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    cuuint64_t d[5], st[5];
    cuuint32_t b[5], es[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = cuuint64_t(dims[i]);
        b[i] = cuuint32_t(box[i]);
        es[i] = 1;
        if (i > 0) st[i - 1] = cuuint64_t(dims[i] > 1 ? strides[i] * 2 : dims[0] * 2);
    }
    return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank),
               const_cast<void*>(ptr), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DIM>
cudaError_t launch_tc(const AttnParams& a, bool prefix, int splits, float* part_o, float* part_lse, cudaStream_t s) {
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(attn_tc_kernel<T, DIM>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(TcGeom<DIM>::kSmem));
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    TcAttnParams p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    p.prefix = prefix ? 1 : 0;
    p.splits = splits;
    p.part_o = part_o;
    p.part_lse = part_lse;
    const int group = a.n_q_heads / a.kv.n_heads;
    p.tile_tokens = kTileRows / group;
    const int page = 1 << a.kv.page_shift;
    const bool f16 = !IsBf16<T>::value;
    const int64_t kd[4] = {DIM, page, a.kv.n_heads, a.kv.n_pages};
    const int64_t ks[4] = {1, a.kv.slot_stride, a.kv.head_stride, a.kv.page_stride};
    const int kb[4] = {64, page < kKeys ? page : kKeys, 1, 1};
    const int64_t qd[3] = {DIM, a.n_q_heads, a.n_tokens}, qs[3] = {1, DIM, a.q_stride};
    const int qb[3] = {64, group, p.tile_tokens};
    if (!encode(&p.k_map, f16, a.kv.k, 4, kd, ks, kb) || !encode(&p.v_map, f16, a.kv.v, 4, kd, ks, kb) ||
        !encode(&p.q_map, f16, a.q, 3, qd, qs, qb))
        return cudaErrorInvalidValue;
    const int64_t pairs = tc_pairs(a.n_tokens, group, a.kv.n_seqs, prefix);
    return launch_serial(attn_tc_kernel<T, DIM>, dim3(unsigned(pairs * a.kv.n_heads), unsigned(splits)), kTcThreads,
                         TcGeom<DIM>::kSmem, s, p);
}

}  // namespace

// Tile pairs at most: each sequence may end with one that is not full.
int64_t tc_pairs(int64_t n_tokens, int group, int n_seqs, bool prefix) {
    const int pair = 2 * (kTileRows / group);
    return prefix ? (n_tokens + pair - 1) / pair : n_tokens / pair + (n_seqs < n_tokens ? n_seqs : n_tokens);
}

cudaError_t launch_attn_tc(int dtype, const AttnParams& a, bool prefix, int splits, float* part_o, float* part_lse,
                           cudaStream_t s) {
    if (a.kv.head_dim == 128)
        return dtype == QX_F16 ? launch_tc<__half, 128>(a, prefix, splits, part_o, part_lse, s)
                               : launch_tc<__nv_bfloat16, 128>(a, prefix, splits, part_o, part_lse, s);
    return dtype == QX_F16 ? launch_tc<__half, 64>(a, prefix, splits, part_o, part_lse, s)
                           : launch_tc<__nv_bfloat16, 64>(a, prefix, splits, part_o, part_lse, s);
}

cudaError_t launch_attn_join(int dtype, const JoinParams& p, cudaStream_t s) {
    const int64_t rows = int64_t(p.a.n_tokens) * p.a.n_q_heads;
    const dim3 grid(unsigned((rows + 7) / 8));
    if (p.a.kv.head_dim == 128)
        return dtype == QX_F16 ? launch_serial(attn_join_kernel<__half, 128>, grid, 256, 0, s, p)
                               : launch_serial(attn_join_kernel<__nv_bfloat16, 128>, grid, 256, 0, s, p);
    return dtype == QX_F16 ? launch_serial(attn_join_kernel<__half, 64>, grid, 256, 0, s, p)
                           : launch_serial(attn_join_kernel<__nv_bfloat16, 64>, grid, 256, 0, s, p);
}

}  // namespace qx
