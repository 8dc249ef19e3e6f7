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
// the base, P at most 2^kRescale times what it would be, which bf16 and the f32
// sums hold without loss; for f16 P is raised as far as the type goes, and the
// maximum follows sooner.  The maximum, the sum of the unrounded exponentials
// and O are f32.
//
// A block of 128 keys takes the pipe 2048 cycles for both tiles (head size 128)
// and an SM's exponential units 1024; a tile's own chain -- scores 512 cycles,
// their way to the softmax 300, softmax 1300, P V 512, and the handovers -- is
// what bounds a block, at about 2900 cycles.  Measured: 4096 causal tokens, 32
// query heads of 128 over 8, 104 us, 1.32 PFLOP/s of the visible pairs, 68 % of
// the measured bf16 rate; 8191 tokens over a window of 1024 keys and 4 first ones
// 119 us (whole blocks at both ends of the window: 9 blocks where 8 hold visible
// keys); head size 64, 14 query heads over 2, 49.5 us (the same chain for half the
// products).
//
// The CTAs are persistent, one an SM.  Where there are many pairs they take them
// from a counter, those with the most keys first; where there are few (a short
// chunk, a shared prefix, contexts of very different lengths) each takes an
// equal share of the line of all pairs' blocks.  A pair whose keys several CTAs
// share leaves parts (o / l and the base-2 log of its sum) that
// attn_join_kernel joins.  (256 tokens behind 32768 shared keys, 8 key heads, are
// 32 pairs.  With the tails, each pair in four parts, on 128 of the SMs: 199 us; in
// even shares on all of them: 182 us.)  A third warpgroup serves the two: a
// scheduler, a producer that runs ahead with the copies, a warp that issues the
// MMAs, and one that zeroes values that no row sees.  The next pair's first
// scores are computed during this pair's epilogue.
//
// Over a cache in 8 bits (Q8) a fourth warpgroup makes 16 bits of the codes that the
// copies bring, V in f16 and K in the queries' type, and leaves the keys' and values'
// scales for the softmax: a key's multiplies its score, a value's its probability
// before that is rounded to f16.  The maximum then counts the power of two that the
// block's scales stay below.  The conversion's shared-memory traffic stands beside the
// MMAs' and the scalings in a tile's chain: 512 tokens over 16384 keys 176 us (at 188,
// without the conversion 142, without the scalings 158 to 173, without both 116; 16 bits
// 104), 8191 tokens over the window 194, five chunks of prompts at head size 64 96.
//
// Every wait is bounded and reports through the device error word.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>
#include <mutex>
#include <type_traits>

#include "qx_attn.cuh"
#include "qx_attn_codes.cuh"
#include "qx_layer.cuh"

namespace qx {

namespace {

constexpr int kKeys = 128;             // keys of a block
constexpr int kTileRows = 128;         // rows of a tile; two tiles a CTA
constexpr int kSoftmaxWarps = 8;       // two warpgroups
// A third warpgroup: the MMA issuer, the producer, the warp that zeroes, and the
// scheduler.  An SM partition holds three of the CTA's warps, so 168
// registers a thread at launch; the softmax warps hold a row of S each.
constexpr int kTcThreads = 32 * (kSoftmaxWarps + 4);
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "registers the CTA was launched with");
// Over codes a fourth warpgroup makes 16 bits of them.
constexpr int kConverters = 4, kTcThreadsQ8 = kTcThreads + 32 * kConverters;
constexpr int kLaunchRegsQ8 = 128, kSoftmaxRegsQ8 = 184, kOtherRegsQ8 = 72;
static_assert(2 * kSoftmaxRegsQ8 + 2 * kOtherRegsQ8 <= 4 * kLaunchRegsQ8, "registers the CTA was launched with");
// (f16: 3 leaves room to raise P by 2^12.  Causal 4096 tokens, and five chunks of
// prompts at head size 64, in f16: 105.1 and 63.0 us; with 2 107.3 and 64.2, with 4
// 104.4 and 62.6.)
template <typename T>
constexpr int kRescale = IsBf16<T>::value ? 8 : 3;
constexpr int kFixed = 3;              // blocks that a pair's fixed cost (some 5 us) is worth
constexpr int kMinPart = 8;            // blocks of a range at least: a part costs some 5 us beside them
constexpr float kWritten = INFINITY;   // as a row's first base-2 log: the row is in the output already
// (long enough for rows_again() of 32 rows over a million keys, which the other warps wait for)
constexpr unsigned long long kWaitNs = 10000000000ull;

template <int DIM, bool Q8 = false>
struct TcGeom {
    static constexpr int kPanels = DIM / 64;                    // 64 elements (128 bytes) of every row
    static constexpr int kPanelBytes = 128 * 128;               // 128 rows
    static constexpr int kTileBytes = kPanels * kPanelBytes;    // Q of a tile, or a block's K or V
    // ring of K and V blocks.  Over codes it is odd: where a block's K goes, the V of
    // block kScaleSets before it was, so that whoever may write there may also write
    // that block's scales
    static constexpr int kSlots = Q8 ? (DIM == 128 ? 3 : 7) : DIM == 128 ? 4 : 10;
    static constexpr int kCodeBytes = 128 * DIM;                // a block's codes of K or V
    static constexpr int kCodeSlots = !Q8 ? 0 : DIM == 128 ? 3 : 4;
    static constexpr int kScaleSets = Q8 ? (kSlots + 1) / 2 : 0;
    static constexpr int kScaleFloats = 2 * 128 + 8;            // of K and V, the power that each 32 of V's stay below, and the least of theirs
    static constexpr int kOutPass = Q8 ? 64 : 128;              // bytes of a row on its way out at a time
    static constexpr int kAlign = Q8 ? 0 : 1024;                // (the dynamic part begins aligned; there is no room to spare)
    static constexpr size_t kSmem = size_t(2 + kSlots) * kTileBytes + kSoftmaxWarps * 32 * kOutPass + kCodeSlots * kCodeBytes +
                                    kScaleSets * kScaleFloats * 4 + kAlign + 640;
};
static_assert(TcGeom<128>::kSmem <= 227 * 1024 && TcGeom<64>::kSmem <= 227 * 1024, "a CTA's shared memory");
static_assert(TcGeom<128, true>::kSmem <= 227 * 1024 && TcGeom<64, true>::kSmem <= 227 * 1024, "a CTA's shared memory");

struct TcAttnParams {
    CUtensorMap q_map;  // [tokens][heads][dim], boxes of one tile's tokens x the group x 64
    CUtensorMap k_map;  // [pages][heads][slots][dim], boxes of min(page, 128) keys x 64
    CUtensorMap v_map;
    AttnParams a;
    int tile_tokens;    // tokens of a tile: 128 / group
    int slots;          // 0: pairs from a counter; else ranges of blocks, and a row's parts at most
    int prefix;         // 1: every token against keys [0, shared_len)
    int tails;          // 1: the parts of a call whose prefix is taken apart
    float* part_o;      // parts: [slots][tokens * heads][dim], or null: write the output
    float* part_lse;    // [slots][tokens * heads]
    unsigned* counter;  // pairs taken beyond each CTA's first, and CTAs done; zero between calls
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
// One lane of a converged warp.  Around it the warp's code stays uniform, so
// descriptors and tensor-memory addresses live in uniform registers; issued
// from a lane-0 branch every MMA first had its operands moved there (75 to 90
// cycles each, against 64 for the product itself).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// 32 columns of the warp's 32 rows, no wait.
__device__ __forceinline__ void ld32(uint32_t taddr, float* u) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3]), "=f"(u[4]), "=f"(u[5]), "=f"(u[6]), "=f"(u[7]), "=f"(u[8]),
          "=f"(u[9]), "=f"(u[10]), "=f"(u[11]), "=f"(u[12]), "=f"(u[13]), "=f"(u[14]), "=f"(u[15]), "=f"(u[16]),
          "=f"(u[17]), "=f"(u[18]), "=f"(u[19]), "=f"(u[20]), "=f"(u[21]), "=f"(u[22]), "=f"(u[23]), "=f"(u[24]),
          "=f"(u[25]), "=f"(u[26]), "=f"(u[27]), "=f"(u[28]), "=f"(u[29]), "=f"(u[30]), "=f"(u[31])
        : "r"(taddr));
}
__device__ __forceinline__ void ld16(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Bits n .. 31 (all of them for n <= 0, none for n >= 32: the shift clamps).
__device__ __forceinline__ uint32_t bits_from(int n) {
    uint32_t r;
    asm("shl.b32 %0, -1, %1;" : "=r"(r) : "r"(n > 0 ? n : 0));
    return r;
}

// A warp's rows of O (one a lane, in tensor memory at `o`; null rows where
// nothing was summed up) times `inv`, to element `at` of `dst`, through 4 KB
// of shared memory: PASS = 128 bytes of every row at a time, so that eight lanes
// write a row's 128 bytes together.  (Each lane writing its own row made 32
// lines of every store: the epilogue took 8000 cycles, and the MMA issuer's
// barrier accesses stood behind it.)  `left`: told when O has been read.  True:
// an element of the warp's first rows is infinite or no number.
template <int DIM, int PASS, typename T>
__device__ __forceinline__ bool write_rows(T* dst, int64_t at, bool live, uint32_t o, bool some, float inv, uint8_t* stage, int lane,
                                           uint64_t* left) {
    constexpr int E = PASS / int(sizeof(T));  // elements a pass
    constexpr int C = PASS / 16, R = 32 / C;  // lanes that write a row's, and rows that they write at once
    const auto at_place = [](int r, int c) { return r * PASS + ((C == 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4); };
    bool odd = false;
    if (!live) at = -1;
    T* to[32 / R];  // of rows R k + lane / C, this lane's 16 bytes
#pragma unroll
    for (int k = 0; k < 32 / R; ++k) {
        const int64_t a = __shfl_sync(0xffffffffu, at, R * k + lane / C);
        to[k] = a < 0 ? nullptr : dst + a + (lane % C) * (E / C);
    }
#pragma unroll
    for (int x0 = 0; x0 < DIM; x0 += E) {
        float v[E];
#pragma unroll
        for (int x = 0; x < E; ++x) v[x] = 0.0f;
        if (some) {
#pragma unroll
            for (int x = 0; x < E; x += 32) {
                if constexpr (E >= 32) {
                    ld32(o + x0 + x, v + x);
                } else {
                    float(&r)[16] = *reinterpret_cast<float(*)[16]>(v);
                    ld16(o + x0, r);
                }
            }
            wait_ld();
            if (x0 + E >= DIM) {
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(left);
            }
        }
        __syncwarp();  // the pass before is read
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t u[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if constexpr (sizeof(T) == 4) u[x] = __float_as_uint(v[4 * c + x] * inv);
                else u[x] = pack2<T>(v[8 * c + 2 * x] * inv, v[8 * c + 2 * x + 1] * inv);
            }
            *reinterpret_cast<uint4*>(stage + at_place(lane, c)) = make_uint4(u[0], u[1], u[2], u[3]);
        }
        __syncwarp();
        uint4 w[32 / R];
#pragma unroll
        for (int k = 0; k < 32 / R; ++k) w[k] = *reinterpret_cast<const uint4*>(stage + at_place(R * k + lane / C, lane % C));
#pragma unroll
        for (int k = 0; k < 32 / R; ++k)
            if (to[k]) *reinterpret_cast<uint4*>(to[k] + x0) = w[k];
        if (to[0]) odd |= any_odd<T>(w[0]);
    }
    return __any_sync(0xffffffffu, odd);
}

// What a CTA works on: `tokens` tokens from t0 on (at most two tiles) of
// sequence b, the first at position pos0, and the key blocks that any of its
// rows sees: those of keys [0, sinks), then those of [lo, end).  In a kernel
// for JOINT sinks, which lie in page 0 and pages are shorter than a block,
// there is no block for them: page 0 stands in the first block of [lo, end)
// for the page before lo's.
struct TcWork {
    int b, t0, tokens, pos0, lo, end, sinks, sink_blocks, blocks;
    int hk, split, i0, nb;  // key head, part, and its blocks [i0, i0 + nb)
    int parts;              // parts of the pair's rows
    int base;               // JOINT: key at which its blocks begin
};
template <bool JOINT>
__device__ __forceinline__ int key_block(const TcWork& w, int i) {  // first key of the i-th block
    if (JOINT) return w.base + i * kKeys;
    return (i < w.sink_blocks ? i : w.lo / kKeys + (i - w.sink_blocks)) * kKeys;
}
template <bool JOINT>
__device__ __forceinline__ void key_range(const TcWork& w, int i, int& lo, int& hi) {  // keys of it that some row sees
    lo = !JOINT && i < w.sink_blocks ? 0 : w.lo;
    hi = !JOINT && i < w.sink_blocks ? w.sinks : w.end;
}

// Sequence b as the tensor cores' pairs of tiles see it: its first token, its
// tokens (none where q_start is no ascending list of this call's tokens) and
// its keys.  A prefix is one pseudo-sequence of all tokens.
struct TcSeq {
    int t0, tokens, len;
};
__device__ __forceinline__ TcSeq tc_seq(const TcAttnParams& p, int b) {
    const KvView& kv = p.a.kv;
    TcSeq q;
    if (p.prefix) {
        q.t0 = q.len = 0;
        q.tokens = kv.q_start[kv.n_seqs] < p.a.n_tokens ? kv.q_start[kv.n_seqs] : p.a.n_tokens;
        return q;
    }
    q.t0 = kv.q_start[b];
    q.tokens = kv.q_start[b + 1] - q.t0;
    q.len = kv.kv_len[b];
    if (q.tokens < 0 || q.t0 < 0 || q.t0 + q.tokens > p.a.n_tokens) q.tokens = 0;
    return q;
}
__device__ __forceinline__ int tc_seqs(const TcAttnParams& p) { return p.prefix ? 1 : p.a.kv.n_seqs; }

// Pair `tile` of that sequence.
template <bool JOINT>
__device__ __forceinline__ void pair_work(const TcAttnParams& p, int b, const TcSeq& q, int tile, TcWork& w) {
    const KvView& kv = p.a.kv;
    const int pair = 2 * p.tile_tokens;
    const int64_t most = kv.table_stride << kv.page_shift;
    w.b = b;
    w.t0 = q.t0 + tile * pair;
    w.tokens = q.tokens - tile * pair < pair ? q.tokens - tile * pair : pair;
    if (p.prefix) {
        w.pos0 = w.lo = w.sinks = w.sink_blocks = 0;
        w.end = int(p.a.shared_len < most ? p.a.shared_len : most);
        w.blocks = (w.end + kKeys - 1) / kKeys;
        return;
    }
    if (q.len > most) atomicOr(kv.err, kErrRange);
    const int64_t pos0 = int64_t(q.len) - q.tokens + tile * pair;
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
    if (JOINT) {
        const int page = 1 << kv.page_shift;
        w.base = w.lo >= page ? (w.lo & ~(page - 1)) - page : 0;
        w.sink_blocks = 0;
        w.blocks = w.end > w.lo ? (w.end - w.base + kKeys - 1) / kKeys : 0;
    }
}

// The tile pair with the given number, counted over all sequences (a sequence
// of n tokens has ceil(n / pair)); false: there is none.  One warp finds it,
// 32 sequences at a time.
template <bool JOINT>
__device__ __forceinline__ bool find_pair(const TcAttnParams& p, int number, int lane, TcWork& w) {
    const int pair = 2 * p.tile_tokens, seqs = tc_seqs(p);
    int base = 0;
    for (int b0 = 0; b0 < seqs; b0 += 32) {
        const int b = b0 + lane;
        TcSeq q = {0, 0, 0};
        if (b < seqs) q = tc_seq(p, b);
        const int tiles = (q.tokens + pair - 1) / pair;
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
        q.t0 = __shfl_sync(0xffffffffu, q.t0, src);
        q.tokens = __shfl_sync(0xffffffffu, q.tokens, src);
        q.len = __shfl_sync(0xffffffffu, q.len, src);
        pair_work<JOINT>(p, b0 + src, q, number - before, w);
        return true;
    }
    return false;
}

// Ranges: the blocks of all pairs and key heads form one line, in the order of
// sequences, pairs and heads (a pair without blocks counts for one, so that its
// rows are written), and each CTA takes `share` of them, whatever the pairs'
// lengths.  Before its blocks every pair has kFixed places for its fixed cost:
// without them the CTA whose range held the first pairs of a prompt, of a block
// or two each, took twice as long as the others.  Places of one head of a
// sequence, and the most blocks that a pair has:
template <bool JOINT>
__device__ __forceinline__ int seq_blocks(const TcAttnParams& p, int b, const TcSeq& q, int lane, int& most) {
    const int pair = 2 * p.tile_tokens, tiles = (q.tokens + pair - 1) / pair;
    int sum = 0;
    for (int i = lane; i < tiles; i += 32) {
        TcWork w;
        pair_work<JOINT>(p, b, q, i, w);
        const int n = w.blocks > 0 ? w.blocks : 1;
        sum += kFixed + n;
        most = most > n ? most : n;
    }
    return __reduce_add_sync(0xffffffffu, sum);
}
struct Range {
    int64_t begin;  // of the pair (and head) in work, on the line
    int64_t share, left;
    int b, tile, tiles, i;  // the sequence, its pair, how many it has, and the pair's next place
    TcSeq q;
    TcWork w;
};
// The next pair that has tokens, from (b, tile) on; false: the line ends.
template <bool JOINT>
__device__ __forceinline__ bool range_pair(const TcAttnParams& p, Range& r) {
    const int pair = 2 * p.tile_tokens, seqs = tc_seqs(p);
    while (r.tile >= r.tiles) {
        if (++r.b >= seqs) return false;
        r.q = tc_seq(p, r.b);
        r.tile = 0;
        r.tiles = (r.q.tokens + pair - 1) / pair;
    }
    pair_work<JOINT>(p, r.b, r.q, r.tile, r.w);
    return true;
}
// This CTA's range.
template <bool JOINT>
__device__ __forceinline__ void open_range(const TcAttnParams& p, int lane, Range& r) {
    const int seqs = tc_seqs(p), heads = p.a.kv.n_heads;
    int64_t U = 0;
    int most = 1;
    for (int b = 0; b < seqs; ++b) U += int64_t(seq_blocks<JOINT>(p, b, tc_seq(p, b), lane, most)) * heads;
    most = __reduce_max_sync(0xffffffffu, most);
    // a pair of n blocks lies in at most n / share + 2 ranges: its slots hold them
    r.share = (U + gridDim.x - 1) / gridDim.x;
    const int64_t least = (most + p.slots - 3) / (p.slots - 2);
    if (r.share < least) r.share = least;
    if (r.share < kMinPart) r.share = kMinPart;
    const int64_t from = int64_t(blockIdx.x) * r.share;
    r.left = U - from < r.share ? U - from : r.share;
    if (r.left <= 0) return;
    r.begin = 0;
    for (r.b = 0;; ++r.b) {
        r.q = tc_seq(p, r.b);
        const int64_t n = int64_t(seq_blocks<JOINT>(p, r.b, r.q, lane, most)) * heads;
        if (from < r.begin + n) break;
        r.begin += n;
    }
    r.tiles = (r.q.tokens + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
    for (r.tile = 0;; ++r.tile) {
        pair_work<JOINT>(p, r.b, r.q, r.tile, r.w);
        const int64_t n = int64_t(kFixed + (r.w.blocks > 0 ? r.w.blocks : 1)) * heads;
        if (from < r.begin + n) break;
        r.begin += n;
    }
    const int units = kFixed + (r.w.blocks > 0 ? r.w.blocks : 1);
    r.w.hk = int((from - r.begin) / units);
    r.begin += int64_t(r.w.hk) * units;
    r.i = int(from - r.begin);
}
// The next piece of it that has blocks (or is a pair without any).
template <bool JOINT>
__device__ __forceinline__ bool take_range(const TcAttnParams& p, Range& r, TcWork& w) {
    while (r.left > 0) {
        const int units = kFixed + (r.w.blocks > 0 ? r.w.blocks : 1);
        const int n = units - r.i < r.left ? units - r.i : int(r.left);
        const int from = r.i > kFixed ? r.i - kFixed : 0, to = r.i + n - kFixed;
        w = r.w;
        w.i0 = from;
        w.nb = w.blocks > 0 ? to - from : 0;
        const int64_t first = (r.begin + kFixed) / r.share;
        w.split = int(blockIdx.x - first);
        w.parts = int((r.begin + units - 1) / r.share - first) + 1;
        r.left -= n;
        r.i += n;
        if (r.i == units && r.left > 0) {
            r.begin += units;
            r.i = 0;
            if (++r.w.hk == p.a.kv.n_heads) {
                ++r.tile;
                const bool some = range_pair<JOINT>(p, r);
                r.w.hk = 0;
                if (!some) r.left = 0;
            }
        }
        if (to > from) return true;
    }
    return false;
}

template <bool JOINT>
__device__ __forceinline__ bool block_has_unseen(const TcWork& w, int i) {
    int lo, hi;
    key_range<JOINT>(w, i, lo, hi);
    const int j0 = key_block<JOINT>(w, i);
    return j0 < lo || j0 + kKeys > hi;
}
// A row of the pair over its blocks in w once more, by one warp and over the keys
// that the row sees alone.
template <typename T, int DIM, bool JOINT>
__device__ __forceinline__ void blocks_again(const TcAttnParams& p, const TcWork& w, int t, int h, int pos, RowSums<DIM / 32>& sums) {
    const T* q = static_cast<const T*>(p.a.q) + int64_t(t) * p.a.q_stride + int64_t(h) * DIM;
    for (int i = w.i0; i < w.i0 + w.nb; ++i) {
        int lo, hi;
        key_range<JOINT>(w, i, lo, hi);
        for (int k = threadIdx.x & 31; k < kKeys; k += 32) {
            int j = key_block<JOINT>(w, i) + k;
            bool sees = j >= lo && j < hi;
            if (JOINT && i == 0 && k < w.sinks) j = k, sees = true;
            sees = sees && j <= pos && (p.a.window == 0 || j > pos - p.a.window || j < p.a.sinks);
            if (__any_sync(0xffffffffu, sees))
                row_keys<T, 8>(p.a, w.b, w.hk, sees ? j : -1, [&](int d, float (&x)[8]) { load_f32<8>(q + d, x); }, sums);
        }
    }
}
// The warp's rows `sound` (a lane each: token tok of the pair, at position pos,
// head h, o / l from row `at` on) once more, where some of them do not see a
// value that is infinite or no number: a later key's, or one of the first row's
// window before their own.  (A call, not in line: the code of the rows' way out
// stays as short as it was.  Causal 4096 tokens 104.5 us, in line 106.3 to 107,
// without it 103.7.  Where it has work it takes its time: 7 us for 32 keys of a
// row, 57 ms for 2000 tokens over 8192 keys whose last value is no number.)
template <typename T, int DIM, bool JOINT>
__device__ __noinline__ void rows_again(const TcAttnParams& p, const TcWork& w, unsigned sound, int low, int pos, int tok, int h, int64_t at,
                                        bool to_part) {
    __syncwarp();  // (the rows were written by other lanes)
    low = __reduce_min_sync(0xffffffffu, low);
    const int high = __reduce_max_sync(0xffffffffu, pos);
    const int64_t from = p.a.sinks > w.lo ? p.a.sinks : w.lo, to = p.a.window > 0 ? high + 1 - p.a.window : 0;
    if (!odd_values<T, DIM>(p.a, w.b, w.hk, low + 1 > w.lo ? low + 1 : w.lo, w.end) && !odd_values<T, DIM>(p.a, w.b, w.hk, from, to)) return;
    for (unsigned again = sound; again != 0; again &= again - 1) {
        const int src = __ffs(again) - 1;
        RowSums<DIM / 32> sums;
        blocks_again<T, DIM, JOINT>(p, w, w.t0 + __shfl_sync(0xffffffffu, tok, src), __shfl_sync(0xffffffffu, h, src), __shfl_sync(0xffffffffu, pos, src), sums);
        write_row_again<T, DIM>(sums, to_part ? p.part_o : p.a.out, to_part || p.a.out_f32, __shfl_sync(0xffffffffu, at, src) * DIM);
    }
}
__device__ __forceinline__ int count_pairs(const TcAttnParams& p, int lane) {
    const int pair = 2 * p.tile_tokens, seqs = tc_seqs(p);
    int sum = 0;
    for (int b = lane; b < seqs; b += 32) sum += (tc_seq(p, b).tokens + pair - 1) / pair;
    return __reduce_add_sync(0xffffffffu, sum);
}

// A place in the ring and the parity of its current use.
struct RingPos {
    int slot = 0;
    uint32_t phase = 0;
    template <int NS>
    __device__ __forceinline__ void next() {
        if (++slot == NS) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// Every lane of the warp waits itself, and the outcome is warp-uniform.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned* err, unsigned code) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitNs, err, code));
}

// The converters' part of the kernel below (four warps, 128 keys).
template <typename T, int DIM, bool JOINT>
__device__ __forceinline__ void convert_blocks(const TcAttnParams& p, TcWork* work, uint64_t* w_full, uint64_t* w_empty, uint8_t* ring,
                                               const uint8_t* codes, float* scales, uint64_t* code_full, uint64_t* code_empty,
                                               uint64_t* kv_empty, uint64_t* clean, uint64_t* scale_full) {
    using G = TcGeom<DIM, true>;
    constexpr int NS = G::kSlots, NC = G::kCodeSlots;
    const KvView& kv = p.a.kv;
    const int lane = threadIdx.x & 31, part = (threadIdx.x >> 5) & 3, key = 32 * part + lane;
    RingPos from, to;
    bool filled = false;  // the ring, once
    int set = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
        if (!(ok = warp_wait(&w_full[n & 1], (n >> 1) & 1, kv.err, kErrTimeoutFull))) break;
        const TcWork& w = work[n & 1];  // (read where it is needed: registers are short here)
        if (w.tokens == 0) break;
        const int begin = w.i0, end = begin + w.nb;
        // this lane's key of block i, or -1: no row sees it; its page; and where its scales lie
        const auto key_of = [&](int i) -> int {
            int lo, hi;
            key_range<JOINT>(w, i, lo, hi);
            const int j = key_block<JOINT>(w, i) + key;
            if (i >= end) return -1;
            if (JOINT && i == 0 && key < w.sinks) return key;
            return j >= lo && j < hi ? j : -1;
        };
        const auto page_at = [&](int i) -> int {
            const int j = key_of(i);
            const int64_t at = j >> kv.page_shift;
            return j >= 0 && at < kv.table_stride ? kv.table[int64_t(w.b) * kv.table_stride + at] : -1;
        };
        float dk = 0.0f, dv = 0.0f;
        const auto fetch = [&](int i, int page) {  // (what is out of range the producer reports)
            dk = dv = 0.0f;
            if (page < 0 || page >= kv.n_pages) return;
            const int64_t at = scale_offset(kv, page, w.hk, key_of(i));
            dk = kv.k_scale[at];
            dv = kv.v_scale[at];
        };
        int page = page_at(begin);
        fetch(begin, page);
        page = page_at(begin + 1);
        for (int i = begin; i < end && ok; ++i) {
#pragma unroll 1
            for (int v = 0; v < 2; ++v) {
                if (filled && !(ok = warp_wait(&kv_empty[to.slot], to.phase ^ 1, kv.err, kErrTimeoutEmpty))) break;
                if (v == 0) {
                    // A scale that is no number makes no numbers of the scores, of the rows
                    // that see it; the product of probability and scale is every row's.
                    const bool sound = fabsf(dk) < INFINITY && fabsf(dv) < INFINITY;
                    float* const sc = scales + set * G::kScaleFloats;
                    const float d = sound ? dv : 0.0f;
                    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(d)));
                    sc[key] = sound ? dk * inner_scale(p.a.scale_log2) : __uint_as_float(0x7fffffffu);
                    sc[kKeys + key] = d;
                    const int least = __reduce_min_sync(0xffffffffu, key_of(i) < 0 ? 128 : int(scale_power(fabsf(d))));
                    if (lane == 0) sc[2 * kKeys + part] = scale_power(__uint_as_float(most)), sc[2 * kKeys + 4 + part] = float(least);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&scale_full[set]);
                    if (++set == G::kScaleSets) set = 0;
                    fetch(i + 1, page);
                    page = page_at(i + 2);
                }
                if (!(ok = warp_wait(&code_full[from.slot], from.phase, kv.err, kErrTimeoutFull))) break;
                const uint8_t* const src = codes + from.slot * G::kCodeBytes + key * DIM;
                uint8_t* const dst = ring + to.slot * G::kTileBytes + key * 128;
                // (a short loop: the softmax's code needs the instruction caches)
#pragma unroll 1
                for (int c0 = 0; c0 < DIM / 16; c0 += 4) {
                    uint32_t x[4][4], y[4][8];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 u = *reinterpret_cast<const uint4*>(src + ((DIM == 128 ? (c0 + c) ^ (key & 7) : c ^ ((key >> 1) & 3)) << 4));
                        x[c][0] = u.x, x[c][1] = u.y, x[c][2] = u.z, x[c][3] = u.w;
                    }
                    if (IsBf16<T>::value && v == 0) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            y[k / 4][2 * (k % 4)] = code_pair_bf16<0, 1>(x[k / 4][k % 4]);
                            y[k / 4][2 * (k % 4) + 1] = code_pair_bf16<2, 3>(x[k / 4][k % 4]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const uint32_t u = x[k / 4][k % 4] ^ 0x80808080u;
                            y[k / 4][2 * (k % 4)] = code_pair<0, 1>(u);
                            y[k / 4][2 * (k % 4) + 1] = code_pair<2, 3>(u);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint8_t* const panel = dst + (c0 >> 2) * G::kPanelBytes;
                        *reinterpret_cast<uint4*>(panel + (((2 * c) ^ (key & 7)) << 4)) = make_uint4(y[c][0], y[c][1], y[c][2], y[c][3]);
                        *reinterpret_cast<uint4*>(panel + (((2 * c + 1) ^ (key & 7)) << 4)) = make_uint4(y[c][4], y[c][5], y[c][6], y[c][7]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&clean[to.slot]);
                    mbar_arrive(&code_empty[from.slot]);
                }
                to.template next<NS>();
                if (to.slot == 0) filled = true;
                from.template next<NC>();
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_empty[n & 1]);
    }
}

template <typename T, int DIM, bool JOINT, bool Q8>
__global__ void __launch_bounds__(Q8 ? kTcThreadsQ8 : kTcThreads, 1) attn_tc_kernel(const __grid_constant__ TcAttnParams p) {
    using G = TcGeom<DIM, Q8>;
    using P = std::conditional_t<Q8, __half, T>;  // the probabilities' type, and the values'
    constexpr int NS = G::kSlots, NC = G::kCodeSlots;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (Q8 ? 0 : (1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    uint8_t* sq = smem;                        // [2 tiles][panels][128 rows][128 B]
    uint8_t* ring = sq + 2 * G::kTileBytes;    // [NS] blocks: K0, V0, K1, V1, ... of pair after pair
    uint8_t* outs = ring + NS * G::kTileBytes;  // for each softmax warp's rows on their way out
    uint8_t* codes = outs + kSoftmaxWarps * 32 * G::kOutPass;  // Q8: [NC] blocks of codes, 128 or 64 bytes a key in as wide a swizzle
    float* scales = reinterpret_cast<float*>(codes + NC * G::kCodeBytes);  // Q8: [kScaleSets][kScaleFloats]
    uint64_t* q_full = reinterpret_cast<uint64_t*>(scales + G::kScaleSets * G::kScaleFloats);
    uint64_t* q_empty = q_full + 1;
    uint64_t* kv_full = q_empty + 1;  // (Q8: of `codes`, as is code_empty)
    uint64_t* code_empty = kv_full + (Q8 ? NC : NS);
    uint64_t* scale_full = code_empty + NC;
    uint64_t* kv_empty = scale_full + G::kScaleSets;
    uint64_t* clean = kv_empty + NS;  // there, and what no row sees of its values is zeroed
    uint64_t* s_full = clean + NS;    // per tile
    uint64_t* p_full = s_full + 2;      // per tile and half of the block's keys
    uint64_t* o_full = p_full + 4;
    uint64_t* o_empty = o_full + 2;
    uint64_t* w_full = o_empty + 2;     // per entry of `work`
    uint64_t* w_empty = w_full + 2;
    uint64_t* w_taken = w_empty + 2;    // a pair's copies are nearly all on their way
    TcWork* work = reinterpret_cast<TcWork*>(w_taken + 1);  // [2]: pairs in hand; tokens 0: no more
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(work + 2);
    static_assert((2 + 3 * NS + 2 * NC + G::kScaleSets + 2 + 4 + 2 + 2 + 2 + 2 + 1) * 8 + 2 * sizeof(TcWork) + 4 <= 640, "barriers and work entries");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KvView& kv = p.a.kv;
    const int group = p.a.n_q_heads / kv.n_heads;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(w_taken, 1);
        for (int i = 0; i < NS; ++i) {
            if (!Q8) mbar_init(&kv_full[i], 1);
            mbar_init(&clean[i], Q8 ? kConverters : 1);
            mbar_init(&kv_empty[i], Q8 ? 1 : 2);  // the MMAs that read it, and the warp that zeroes
        }
        for (int i = 0; i < NC; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&code_empty[i], kConverters);
        }
        for (int i = 0; i < G::kScaleSets; ++i) mbar_init(&scale_full[i], kConverters);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], 4);
            mbar_init(&w_full[i], 1);
            mbar_init(&w_empty[i], kSoftmaxWarps + (Q8 ? 2 + kConverters : 3));
        }
        fence_barrier_init();
        prefetch_map(&p.q_map);
        prefetch_map(&p.k_map);
        prefetch_map(&p.v_map);
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
    pdl_wait_prior_grid();
    pdl_launch_dependents();

    if (warp >= kSoftmaxWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Q8 ? kOtherRegsQ8 : kOtherRegs));
        if (Q8 && warp >= kSoftmaxWarps + 4) {
            // ---- converters: a lane a key.  Codes to 16 bits, in the MMAs' layout (eight
            // lanes' 16 bytes, of eight keys, lie in different banks on both sides), and
            // the block's scales for the softmax.  Their pages are looked up two blocks
            // ahead and they are fetched one block ahead.
            if constexpr (Q8) convert_blocks<T, DIM, JOINT>(p, work, w_full, w_empty, ring, codes, scales, kv_full, code_empty, kv_empty, clean, scale_full);
        } else if (warp == kSoftmaxWarps + 1) {
            // ---- producer: of each pair Q, then K and V of its blocks
            const int page_keys = (1 << kv.page_shift) < kKeys ? (1 << kv.page_shift) : kKeys;
            const int boxes = kKeys / page_keys;  // of a block (at most 8)
            RingPos at;
            int64_t issued = 0;
            bool ok = true;
            int quse = 0;
            for (int n = 0; ok; ++n) {
                if (!(ok = warp_wait(&w_full[n & 1], (n >> 1) & 1, kv.err, kErrTimeoutFull))) break;
                const TcWork w = work[n & 1];
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&w_empty[n & 1]);
                    if (w.nb == 0) mbar_arrive(w_taken);
                }
                if (w.tokens == 0) break;
                if (w.nb == 0) continue;
                const int tiles = w.tokens > p.tile_tokens ? 2 : 1;
                if (quse > 0 && !(ok = warp_wait(q_empty, (quse - 1) & 1, kv.err, kErrTimeoutEmpty))) break;
                ++quse;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, tiles * G::kPanels * p.tile_tokens * group * 128);
                    for (int t = 0; t < tiles; ++t)
                        for (int c = 0; c < G::kPanels; ++c)
                            tma_load_3d(sq + t * G::kTileBytes + c * G::kPanelBytes, &p.q_map, 64 * c, w.hk * group,
                                        w.t0 + t * p.tile_tokens, q_full);
                }
                __syncwarp();
                // lane x of the first `boxes` finds the page of its box of the block, one block ahead
                const auto page_of_box = [&](int i) -> int {
                    int lo, hi;
                    key_range<JOINT>(w, i, lo, hi);
                    if (JOINT && (i | lane) == 0) return page_of(kv, w.b, 0);
                    const int j = key_block<JOINT>(w, i) + lane * page_keys;
                    return lane < boxes && j + page_keys > lo && j < hi ? page_of(kv, w.b, j) : -1;
                };
                int next_page = page_of_box(w.i0);
                for (int i = w.i0; i < w.i0 + w.nb && ok; ++i) {
                    const int page = next_page;
                    if (i + 1 < w.i0 + w.nb) next_page = page_of_box(i + 1);
                    const unsigned live = __ballot_sync(0xffffffffu, page >= 0);
                    const int in_page = (key_block<JOINT>(w, i) + lane * page_keys) & ((1 << kv.page_shift) - 1);
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        if constexpr (Q8) {
                            if (issued >= NC && !(ok = warp_wait(&code_empty[at.slot], at.phase ^ 1, kv.err, kErrTimeoutEmpty))) break;
                            if (lane == 0) mbar_arrive_expect_tx(&kv_full[at.slot], __popc(live) * page_keys * DIM);
                            __syncwarp();
                            if (page >= 0)
                                tma_load_4d(codes + at.slot * G::kCodeBytes + lane * page_keys * DIM, v ? &p.v_map : &p.k_map, 0, in_page, w.hk, page,
                                            &kv_full[at.slot]);
                            ++issued;
                            at.template next<NC>();
                            continue;
                        }
                        if (issued >= NS && !(ok = warp_wait(&kv_empty[at.slot], at.phase ^ 1, kv.err, kErrTimeoutEmpty))) break;
                        if (lane == 0) mbar_arrive_expect_tx(&kv_full[at.slot], __popc(live) * page_keys * 128 * G::kPanels);
                        __syncwarp();
                        if (page >= 0) {
                            uint8_t* dst = ring + at.slot * G::kTileBytes + lane * page_keys * 128;
                            for (int c = 0; c < G::kPanels; ++c)
                                tma_load_4d(dst + c * G::kPanelBytes, v ? &p.v_map : &p.k_map, 64 * c, in_page, w.hk, page,
                                       &kv_full[at.slot]);
                        }
                        ++issued;
                        at.template next<NS>();
                    }
                    if (lane == 0 && i == w.i0 + (w.nb > 1 ? w.nb - 2 : 0)) mbar_arrive(w_taken);  // (one block is left)
                }
            }
            // keep the CTA alive until every copy it issued has landed
            if (lane == 0) {
                if (quse > 0) mbar_wait_bounded(q_full, (quse - 1) & 1, kWaitNs, kv.err, kErrTimeoutDrain);
                constexpr int N = Q8 ? NC : NS;
                for (int64_t i = issued > N ? issued - N : 0; i < issued; ++i)
                    mbar_wait_bounded(&kv_full[i % N], (i / N) & 1, kWaitNs, kv.err, kErrTimeoutDrain);
            }
        } else if (warp == kSoftmaxWarps + 3) {
            // ---- scheduler.  Pairs from the counter are taken when the one
            // before is nearly all on its way, not earlier: a CTA with a long pair in
            // work would sit on another.
            const int pairs = p.slots == 0 ? count_pairs(p, lane) : 0;
            Range r;
            if (p.slots > 0) open_range<JOINT>(p, lane, r);
            for (int n = 0;; ++n) {
                if (n >= 2 && !warp_wait(&w_empty[n & 1], ((n >> 1) - 1) & 1, kv.err, kErrTimeoutEmpty)) break;
                TcWork w;
                bool more;
                if (p.slots > 0) {
                    more = take_range<JOINT>(p, r, w);
                } else {
                    int item = int(blockIdx.x);
                    if (n > 0) {
                        if (!warp_wait(w_taken, (n - 1) & 1, kv.err, kErrTimeoutEmpty)) break;
                        if (lane == 0) item = int(gridDim.x + atomicAdd(p.counter, 1u));
                        item = __shfl_sync(0xffffffffu, item, 0);
                    }
                    // the pairs with the most keys (the last of a sequence) first
                    const int number = item / kv.n_heads;
                    more = number < pairs && find_pair<JOINT>(p, pairs - 1 - number, lane, w);
                    w.hk = item - number * kv.n_heads;
                    w.split = w.i0 = 0;
                    w.parts = 1;
                    w.nb = w.blocks;
                }
                if (!more) w.tokens = w.nb = 0;
                if (lane == 0) {
                    work[n & 1] = w;
                    mbar_arrive(&w_full[n & 1]);
                }
                __syncwarp();
                if (!more) break;
            }
        } else if (warp == kSoftmaxWarps) {
            // ---- MMA issuer
            const uint32_t base = uniform(smem_addr(sq)), tm = uniform(tmem);
            const uint64_t q_desc = sw128_desc(base, 16), k_desc = sw128_desc(base + 2 * G::kTileBytes, 16),
                           v_desc = sw128_desc(base + 2 * G::kTileBytes, G::kPanelBytes);
            RingPos at;
            uint32_t blocks[2] = {0, 0}, quse = 0;  // blocks of each tile, and pairs so far
            bool ok = true;
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = warp_wait(bar, parity & 1, kv.err, kErrTimeoutMma);
                return ok;
            };
            const auto wait2 = [&](uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) {
                const bool first = mbar_try_wait(a, pa), second = mbar_try_wait(b, pb);
                if (__all_sync(0xffffffffu, first && second)) return true;
                return wait(a, pa) && wait(b, pb);
            };
            const auto scores = [&](int t, int slot, uint64_t* frees, uint64_t* frees_too) {
                const uint64_t q = q_desc + t * (G::kTileBytes >> 4), k = k_desc + slot * (G::kTileBytes >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < DIM / 16; ++x) {
                        const uint64_t off = ((x >> 2) * G::kPanelBytes + (x & 3) * 32) >> 4;
                        mma_ss(tm + 128 * t, q + off, k + off, idesc<T>(kKeys, false), x > 0 ? 1u : 0u);
                    }
                    commit(&s_full[t]);
                    if (frees) commit(frees);
                    if (frees_too) commit(frees_too);
                }
                __syncwarp();
            };
            const auto release = [&](uint64_t* bar, uint64_t* too) {
                if (elect_one()) {
                    commit(bar);
                    if (too) commit(too);
                }
                __syncwarp();
            };
            for (int n = 0; ok; ++n) {
                if (!wait(&w_full[n & 1], n >> 1)) break;
                const TcWork w = work[n & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&w_empty[n & 1]);
                const int tokens = int(uniform(uint32_t(w.tokens))), nb = int(uniform(uint32_t(w.nb)));
                if (tokens == 0) break;
                if (nb == 0) continue;
                const int tiles = tokens > p.tile_tokens ? 2 : 1;
                if (!wait(q_full, quse)) break;
                if (!wait(&clean[at.slot], at.phase)) break;
                tc_after();
                for (int t = 0; t < tiles; ++t) scores(t, at.slot, nullptr, nullptr);
                release(&kv_empty[at.slot], nb == 1 ? q_empty : nullptr);
                at.template next<NS>();
                RingPos v = at, k = at;  // the values of this block, the keys of the next
                k.template next<NS>();
                // (Over codes the ring holds three: V of a block is waited for before its
                // product and K before its scores, not one ahead.)
                if (!Q8 && (!wait(&clean[v.slot], v.phase) || (nb > 1 && !wait(&clean[k.slot], k.phase)))) break;
                for (int i = 0; i < nb && ok; ++i) {
                    const bool last = i + 1 == nb;
                    const uint64_t vd = v_desc + v.slot * (G::kTileBytes >> 4);
                    const int v_slot = v.slot, k_slot = k.slot;
                    const uint32_t k_phase = k.phase;
                    if (Q8 && !wait(&clean[v_slot], v.phase)) break;
                    for (int t = 0; t < tiles && ok; ++t) {
                        // the pair before has left O
                        if (i == 0 && quse > 0 && !wait(&o_empty[t], quse - 1)) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!wait(&p_full[2 * t + h], blocks[t])) break;
                            tc_after();
                            if (elect_one()) {
#pragma unroll
                                for (int x = 4 * h; x < 4 * h + 4; ++x)
                                    mma_ts(tm + 256 + 128 * t, tm + 128 * t + 8 * x, vd + x * (2048 >> 4), idesc<P>(DIM, true),
                                           (i | x) > 0 ? 1u : 0u);
                                if (h == 1) {
                                    commit(&o_full[t]);
                                    if (t + 1 == tiles) commit(&kv_empty[v_slot]);
                                }
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                        ++blocks[t];
                        if (last) continue;
                        // while the pipe works: the next block's values and the keys after them
                        if (t + 1 == tiles) {
                            v = k;
                            v.template next<NS>();
                            k = v;
                            k.template next<NS>();
                            if (!Q8 && (i + 2 < nb ? !wait2(&clean[v.slot], v.phase, &clean[k.slot], k.phase) : !wait(&clean[v.slot], v.phase))) break;
                        }
                        if (Q8 && t == 0) {
                            if (!wait(&clean[k_slot], k_phase)) break;
                            tc_after();
                        }
                        scores(t, k_slot, t + 1 == tiles ? &kv_empty[k_slot] : nullptr, t + 1 == tiles && i + 2 == nb ? q_empty : nullptr);
                    }
                }
                at = k;  // past the last block's values
                ++quse;
            }
        } else if (!Q8 && warp == kSoftmaxWarps + 2) {
            // ---- values that no row sees are zeroed: whatever the slots hold, 0 x it must be 0
            RingPos at;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                if (!(ok = warp_wait(&w_full[n & 1], (n >> 1) & 1, kv.err, kErrTimeoutFull))) break;
                const TcWork w = work[n & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&w_empty[n & 1]);
                if (w.tokens == 0) break;
                for (int i = w.i0; i < w.i0 + w.nb && ok; ++i) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        if (!(ok = warp_wait(&kv_full[at.slot], at.phase, kv.err, kErrTimeoutFull))) break;
                        if (v && block_has_unseen<JOINT>(w, i)) {
                            int lo, hi;
                            key_range<JOINT>(w, i, lo, hi);
                            const int j0 = key_block<JOINT>(w, i), firsts = JOINT && i == 0 ? w.sinks : 0;
                            // (eight lanes a row of 128 bytes: no bank conflicts)
                            for (int r = lane >> 3; r < kKeys; r += 4)
                                if ((j0 + r < lo || j0 + r >= hi) && (!JOINT || r >= firsts))
#pragma unroll
                                    for (int c = 0; c < G::kPanels; ++c)
                                        *reinterpret_cast<uint4*>(ring + at.slot * G::kTileBytes + c * G::kPanelBytes + r * 128 + 16 * (lane & 7)) =
                                            make_uint4(0u, 0u, 0u, 0u);
                            fence_proxy_async_smem();
                        }
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&clean[at.slot]);
                            mbar_arrive(&kv_empty[at.slot]);
                        }
                        at.template next<NS>();
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Q8 ? kSoftmaxRegsQ8 : kSoftmaxRegs));
        // ---- softmax: one thread a row
        const int t = warp >> 2;  // tile
        const int r = 32 * (warp & 3) + lane;
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        const uint32_t sa = tS + 128 * t + lanes, oa = tO + 128 * t + lanes;
        const int in_tile = r / group, head = r - in_tile * group, tok = t * p.tile_tokens + in_tile;
        const int window = p.a.window > 0 && p.a.window < INT32_MAX ? int(p.a.window) : INT32_MAX;
        const int sinks = p.a.sinks < INT32_MAX ? int(p.a.sinks) : INT32_MAX;
        const float f = Q8 ? outer_scale(p.a.scale_log2) : p.a.scale_log2;  // positive: the split kernel takes the others
        uint32_t blocks = 0;             // of this tile so far
        uint32_t set = 0, set_phase = 0; // Q8: of the CTA's, whichever tiles they were for
        bool ok = true;
        for (int n = 0; ok; ++n) {
            if (!(ok = warp_wait(&w_full[n & 1], (n >> 1) & 1, kv.err, kErrTimeoutMma))) break;
            // (the entry is read where it is needed: registers are short here)
            const TcWork& w = work[n & 1];
            if (w.tokens == 0) break;
            const int tiles = w.tokens > p.tile_tokens ? 2 : 1;
            if (t >= tiles) {  // no rows for this warpgroup
                const bool some = w.nb > 0;
                if constexpr (Q8) {
                    const uint32_t on = set + w.nb;
                    set_phase ^= on / G::kScaleSets & 1;
                    set = on % G::kScaleSets;
                }
                __syncwarp();
                if (lane == 0) {
                    if (some) mbar_arrive(&o_empty[t]);
                    mbar_arrive(&w_empty[n & 1]);
                }
                continue;
            }
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
            const int wlo = pos >= window ? pos - window + 1 : 0;  // first key of this row's window
            // (A thread without a row has whatever shared memory held as its scores:
            // with this maximum it never asks for a rescale, which would move its
            // warp's rows to other bases, and their outputs to other roundings.)
            float m = live ? -INFINITY : INFINITY, l = 0.0f;
            float s[kKeys];
            const int nb = w.nb;
            for (int i = 0; i < nb; ++i) {
                const float* const sc = scales + set * G::kScaleFloats;
                if (!(ok = warp_wait(&s_full[t], blocks & 1, kv.err, kErrTimeoutMma))) break;
                if constexpr (Q8) {
                    // (Behind the scores, which the converters' keys were awaited for: the set
                    // has been filled, and is not filled again before this block's values
                    // have been multiplied, so its barrier is in the phase that is asked for.
                    // Before them it may be two uses behind, where this warpgroup had no rows
                    // for a while, and of the same parity.  Asked there, 512 tokens over 16384
                    // keys took 9 us more, and 8191 tokens over the window 2 us less.)
                    if (!(ok = warp_wait(&scale_full[set], set_phase, kv.err, kErrTimeoutMma))) break;
                    if (++set == G::kScaleSets) set = 0, set_phase ^= 1;
                }
                tc_after();
#pragma unroll
                for (int c = 0; c < 4; ++c) ld32(sa + 32 * c, s + 32 * c);
                const int j0 = key_block<JOINT>(w, w.i0 + i);
                int lo, hi;
                key_range<JOINT>(w, w.i0 + i, lo, hi);
                // the row sees [first, last] (a thread without a row: whatever does not make its warp mask)
                const int first = !live || (!JOINT && w.i0 + i < w.sink_blocks) ? 0 : (wlo > lo ? wlo : lo);
                const int last = !live ? INT32_MAX - 1 : pos < hi - 1 ? pos : hi - 1;
                wait_ld();
                float power = 0.0f;  // Q8: that the scales of the values which the row sees stay below
                if constexpr (Q8) {
#pragma unroll
                    for (int x = 0; x < kKeys; x += 4) {
                        const float4 d = *reinterpret_cast<const float4*>(sc + x);
                        const float2 a = f32x2_unpack(f32x2_mul(f32x2_pack(s[x], s[x + 1]), f32x2_pack(d.x, d.y)));
                        const float2 b = f32x2_unpack(f32x2_mul(f32x2_pack(s[x + 2], s[x + 3]), f32x2_pack(d.z, d.w)));
                        s[x] = a.x, s[x + 1] = a.y, s[x + 2] = b.x, s[x + 3] = b.y;
                    }
                    const float4 d = *reinterpret_cast<const float4*>(sc + 2 * kKeys);
                    power = fmaxf(fmaxf(d.x, d.y), fmaxf(d.z, d.w));
                }
                if (__any_sync(0xffffffffu, first > j0 || last < j0 + kKeys - 1)) {
                    // and, in a window block, sinks that the pair's first row has in its window (joint
                    // sinks: all of them in the first block, whose first keys they are)
                    const int a = first - j0, b = last - j0;
                    const int c0 = JOINT ? 0 : lo - j0, c1 = !JOINT ? sinks - j0 : w.i0 + i == 0 ? sinks : 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t see = (bits_from(a - 32 * k) | (bits_from(c0 - 32 * k) & ~bits_from(c1 - 32 * k))) &
                                             ~bits_from(b + 1 - 32 * k);
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (!(see & (1u << x))) s[32 * k + x] = -INFINITY;
                    }
                    if constexpr (Q8) {
                        // The block's power may be that of a key which the row does not see.
                        // Where all are within kPowers of one another, that costs the row
                        // no more than those of the powers its products have to spare.
                        // (Looking through the row's own in every such block: 8191 tokens
                        // over a window of 1024, of whose nine blocks three are such, 214
                        // us, so 195.)
                        constexpr float kPowers = 4.0f;
                        const float4 e = *reinterpret_cast<const float4*>(sc + 2 * kKeys + 4);
                        if (power - fminf(fminf(e.x, e.y), fminf(e.z, e.w)) > kPowers) {
                            float most = 0.0f;
#pragma unroll
                            for (int x = 0; x < kKeys; ++x)
                                if (s[x] != -INFINITY) most = fmaxf(most, fabsf(sc[kKeys + x]));
                            power = scale_power(most);
                        }
                    }
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int x = 4; x < kKeys; x += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y) mx[y] = x + 4 < kKeys ? max3(mx[y], s[x + y], s[x + 4 + y]) : fmaxf(mx[y], s[x + y]);
                float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * f;
                if constexpr (Q8) top += power;
                if (__any_sync(0xffffffffu, top > m + float(kRescale<P>))) {
                    const float mn = fmaxf(m, top);
                    float a;
                    if constexpr (Q8) {
                        const float h = mn == -INFINITY ? 1.0f : exp2_approx(0.5f * (m - mn));
                        a = h * h;
                        l = twice(l, h);
                    } else {
                        a = mn == -INFINITY ? 1.0f : exp2_approx(m - mn);
                        l *= a;
                    }
                    m = mn;
                    if (i > 0) {
                        if (!(ok = warp_wait(&o_full[t], (blocks - 1) & 1, kv.err, kErrTimeoutMma))) break;
                        tc_after();
#pragma unroll
                        for (int c = 0; c < DIM / 16; ++c) {
                            float o[16];
                            ld16(oa + 16 * c, o);
                            wait_ld();
                            uint32_t u[16];
#pragma unroll
                            for (int x = 0; x < 16; ++x) u[x] = __float_as_uint(o[x] * a);
                            st16(oa + 16 * c, u);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.0f : m - kLift<P, kRescale<P>>;
                const uint64_t f2 = f32x2_pack(f, f), b2 = f32x2_pack(-base, -base);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t u[16];
                    float4 d4;
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const float2 e = f32x2_unpack(f32x2_fma(f32x2_pack(s[32 * c + 2 * x], s[32 * c + 2 * x + 1]), f2, b2));
                        const float e0 = exp2_approx(e.x), e1 = exp2_approx(e.y);
                        sum[x & 1] = f32x2_add(sum[x & 1], f32x2_pack(e0, e1));
                        if constexpr (Q8) {
                            if (x % 2 == 0) d4 = *reinterpret_cast<const float4*>(sc + kKeys + 32 * c + 2 * x);
                            const float2 d = x % 2 == 0 ? make_float2(d4.x, d4.y) : make_float2(d4.z, d4.w);
                            const float2 w = f32x2_unpack(f32x2_mul(f32x2_pack(e0, e1), f32x2_pack(d.x, d.y)));
                            u[x] = pack2<P>(w.x, w.y);
                        } else {
                            u[x] = pack2<T>(e0, e1);
                        }
                    }
                    st16(sa + 16 * c, u);
                    if (c & 1) {  // half of the keys: the tensor cores may begin
                        wait_st();
                        tc_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_full[2 * t + (c >> 1)]);
                    }
                }
                const float2 s01 = f32x2_unpack(f32x2_add(sum[0], sum[1]));
                l += s01.x + s01.y;
                ++blocks;
            }
            if (!ok) break;
            // ---- output
            if (nb > 0) {
                if (!(ok = warp_wait(&o_full[t], (blocks - 1) & 1, kv.err, kErrTimeoutMma))) break;
                tc_after();
            }
            // a row whose keys were all here goes to the output, others to their part
            const int split = w.split;
            const bool to_part = p.part_o && (p.prefix || p.tails || w.parts > 1);
            const int64_t row = int64_t(w.t0 + tok) * p.a.n_q_heads + w.hk * group + head;
            const int64_t part = int64_t(split) * p.a.n_tokens * p.a.n_q_heads + row;
            const float lse2 = l == 0.0f ? -INFINITY : m - kLift<P, kRescale<P>> + log2f(l);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (live && p.part_o) {
                p.part_lse[part] = to_part ? lse2 : kWritten;
                if (to_part && split == w.parts - 1)  // the row has no further parts
                    for (int e = w.parts; e < p.slots; ++e) p.part_lse[part + (e - split) * int64_t(p.a.n_tokens) * p.a.n_q_heads] = -INFINITY;
            }
            {
                if (live && !to_part && p.a.lse) p.a.lse[row] = lse2 * 0.6931471805599453f;
                uint8_t* stage = outs + warp * 32 * G::kOutPass;
                // A value that is infinite or no number shows in all rows, so the first ones tell.
                bool odd;
                if (to_part) odd = write_rows<DIM, G::kOutPass>(p.part_o, part * DIM, live, oa, nb > 0, inv, stage, lane, &o_empty[t]);
                else if (p.a.out_f32) odd = write_rows<DIM, G::kOutPass>(static_cast<float*>(p.a.out), row * DIM, live, oa, nb > 0, inv, stage, lane, &o_empty[t]);
                else odd = write_rows<DIM, G::kOutPass>(static_cast<T*>(p.a.out), row * DIM, live, oa, nb > 0, inv, stage, lane, &o_empty[t]);
                // (where the sum of a row's probabilities is no number, no element of it is one)
                const unsigned sound = __ballot_sync(0xffffffffu, live && l == l);
                if constexpr (!Q8) if (odd)
                    rows_again<T, DIM, JOINT>(p, w, sound, live ? pos : INT32_MAX, pos, tok, head + w.hk * group, to_part ? part : row, to_part);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_empty[n & 1]);
        }
    }
    tc_before();
    __syncthreads();
    __syncwarp();
    if (warp == kSoftmaxWarps)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    if (threadIdx.x == 0) {
        // the last CTA leaves the counters at zero for the next call
        __threadfence();
        if (atomicAdd(p.counter + 1, 1u) == gridDim.x - 1) p.counter[0] = p.counter[1] = 0;
    }
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
    const float mine = lane < p.parts ? p.part_lse[lane * rows + row] : -INFINITY;
    if (int(row / p.a.n_q_heads) >= p.a.kv.q_start[p.a.kv.n_seqs]) return;  // a token of no sequence
    if (__shfl_sync(0xffffffffu, mine, 0) == kWritten) return;
    float M = mine;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float wt = mine == -INFINITY ? 0.0f : exp2_approx(mine - M);
    float L = wt;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float acc[V] = {};
    // the parts that say something, four loads in flight
    for (unsigned left = __ballot_sync(0xffffffffu, wt != 0.0f); left != 0;) {
        float v[4][V], c[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int i = left ? __ffs(left) - 1 : 0;
            c[y] = __shfl_sync(0xffffffffu, wt, i);
            if (!left) c[y] = 0.0f;
#pragma unroll
            for (int x = 0; x < V; ++x) v[y][x] = 0.0f;
            const float* src = p.part_o + (i * rows + row) * DIM + V * lane;
            if (left) {
                if constexpr (V == 4) {
                    const float4 f = *reinterpret_cast<const float4*>(src);
                    v[y][0] = f.x, v[y][1] = f.y, v[y][2] = f.z, v[y][3] = f.w;
                } else {
                    const float2 f = *reinterpret_cast<const float2*>(src);
                    v[y][0] = f.x, v[y][1] = f.y;
                }
            }
            left &= left - 1;
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int x = 0; x < V; ++x) acc[x] += c[y] * v[y][x];
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int x = 0; x < V; ++x) acc[x] *= inv;
    if (p.a.lse && lane == 0) p.a.lse[row] = L != 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
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

// A tensor of `bytes` an element, dims[0] contiguous, strides in elements; boxes
// of box[], whose rows are 128 bytes, or 64, in a swizzle as wide.  A dimension of
// one element may have any stride: it is given a valid one.
bool encode(CUtensorMap* m, CUtensorMapDataType type, int bytes, const void* ptr, int rank, const int64_t* dims, const int64_t* strides,
            const int* box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    cuuint64_t d[5], st[5];
    cuuint32_t b[5], es[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = cuuint64_t(dims[i]);
        b[i] = cuuint32_t(box[i]);
        es[i] = 1;
        if (i > 0) st[i - 1] = cuuint64_t(dims[i] > 1 ? strides[i] * bytes : dims[0] * bytes);
    }
    return enc(m, type, cuuint32_t(rank), const_cast<void*>(ptr), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               box[0] * bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode(CUtensorMap* m, bool f16, const void* ptr, int rank, const int64_t* dims, const int64_t* strides, const int* box) {
    return encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, rank, dims, strides, box);
}

template <typename T, int DIM, bool Q8 = false>
cudaError_t launch_tc(const AttnParams& a, bool prefix, int slots, float* part_o, float* part_lse, unsigned* counter,
                      int sm_count, cudaStream_t s) {
    // Sinks in page 0, of several pages to a block: no block of their own.  (8191
    // tokens, window 1024 + 4, pages of 64: 119 us, against 125 with one; a kernel of
    // its own, since the same choice at run time made the other calls 1 to 3 % slower.)
    const int page = 1 << a.kv.page_shift;
    const bool joint = !prefix && a.window > 0 && a.sinks > 0 && a.sinks <= page && page < kKeys && a.shared_len == 0;
    const auto kernel = joint ? attn_tc_kernel<T, DIM, true, Q8> : attn_tc_kernel<T, DIM, false, Q8>;
    static bool ready[64][2] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev][joint]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(TcGeom<DIM, Q8>::kSmem));
        if (e != cudaSuccess) return e;
        ready[dev][joint] = true;
    }
    TcAttnParams p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    p.prefix = prefix ? 1 : 0;
    p.tails = !prefix && a.shared_len > 0 ? 1 : 0;
    p.slots = slots;
    p.part_o = part_o;
    p.part_lse = part_lse;
    p.counter = counter;
    const int group = a.n_q_heads / a.kv.n_heads;
    p.tile_tokens = kTileRows / group;
    const bool f16 = !IsBf16<T>::value;
    const int64_t qd[3] = {DIM, a.n_q_heads, a.n_tokens}, qs[3] = {1, DIM, a.q_stride};
    const int qb[3] = {64, group, p.tile_tokens};
    if (!(Q8 ? encode_code_maps(a.kv, kKeys, &p.k_map, &p.v_map) : encode_cache_maps(f16, a.kv, kKeys, &p.k_map, &p.v_map)) ||
        !encode(&p.q_map, f16, a.q, 3, qd, qs, qb))
        return cudaErrorInvalidValue;
    const int64_t items = tc_pairs(a.n_tokens, group, a.kv.n_seqs, prefix) * a.kv.n_heads;
    return launch_serial(kernel, dim3(unsigned(slots == 0 && items < sm_count ? items : sm_count)), Q8 ? kTcThreadsQ8 : kTcThreads,
                         TcGeom<DIM, Q8>::kSmem, s, p);
}

}  // namespace

bool encode_cache_maps(bool f16, const KvView& kv, int keys, CUtensorMap* k, CUtensorMap* v) {
    const int page = 1 << kv.page_shift;
    const int64_t dims[4] = {kv.head_dim, page, kv.n_heads, kv.n_pages};
    const int64_t strides[4] = {1, kv.slot_stride, kv.head_stride, kv.page_stride};
    const int box[4] = {64, page < keys ? page : keys, 1, 1};
    return encode(k, f16, kv.k, 4, dims, strides, box) && encode(v, f16, kv.v, 4, dims, strides, box);
}

bool encode_code_maps(const KvView& kv, int keys, CUtensorMap* k, CUtensorMap* v) {
    const int page = 1 << kv.page_shift;
    const int64_t dims[4] = {kv.head_dim, page, kv.n_heads, kv.n_pages};
    const int64_t strides[4] = {1, kv.slot_stride, kv.head_stride, kv.page_stride};
    const int box[4] = {kv.head_dim, page < keys ? page : keys, 1, 1};
    return encode(k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kv.k, 4, dims, strides, box) &&
           encode(v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kv.v, 4, dims, strides, box);
}

// Tile pairs at most: each sequence may end with one that is not full.
int64_t tc_pairs(int64_t n_tokens, int group, int n_seqs, bool prefix) {
    const int pair = 2 * (kTileRows / group);
    return prefix || n_seqs == 1 ? (n_tokens + pair - 1) / pair : n_tokens / pair + (n_seqs < n_tokens ? n_seqs : n_tokens);
}

cudaError_t launch_attn_tc(int dtype, const AttnParams& a, bool prefix, int slots, float* part_o, float* part_lse,
                           unsigned* counter, int sm_count, cudaStream_t s) {
    if (a.kv.head_dim == 128)
        return dtype == QX_F16 ? launch_tc<__half, 128>(a, prefix, slots, part_o, part_lse, counter, sm_count, s)
                               : launch_tc<__nv_bfloat16, 128>(a, prefix, slots, part_o, part_lse, counter, sm_count, s);
    return dtype == QX_F16 ? launch_tc<__half, 64>(a, prefix, slots, part_o, part_lse, counter, sm_count, s)
                           : launch_tc<__nv_bfloat16, 64>(a, prefix, slots, part_o, part_lse, counter, sm_count, s);
}

cudaError_t launch_attn_tc_q8(int dtype, const AttnParams& a, int slots, float* part_o, float* part_lse, unsigned* counter, int sm_count,
                              cudaStream_t s) {
    if (a.kv.head_dim == 128)
        return dtype == QX_F16 ? launch_tc<__half, 128, true>(a, false, slots, part_o, part_lse, counter, sm_count, s)
                               : launch_tc<__nv_bfloat16, 128, true>(a, false, slots, part_o, part_lse, counter, sm_count, s);
    return dtype == QX_F16 ? launch_tc<__half, 64, true>(a, false, slots, part_o, part_lse, counter, sm_count, s)
                           : launch_tc<__nv_bfloat16, 64, true>(a, false, slots, part_o, part_lse, counter, sm_count, s);
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
