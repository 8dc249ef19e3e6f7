// qx_attn.cu -- attention over the paged cache.
//
// Row (token t, query head h) at position pos: with s_j = scale q . k_j over
// the keys it sees, m the running maximum, l the running sum of exp(s_j - m)
// and o the running sum of exp(s_j - m) v_j, a block of keys with maximum m'
// turns (m, l, o) into (M, l e^(m-M) + sum e^(s_j-M), o e^(m-M) + ...), M =
// max(m, m'); the output is o / l.  Exponents are taken to base 2 with
// scale * log2(e) folded into the scores.
#include "qx_attn.cuh"
#include "qx_layer.cuh"

namespace qx {

namespace {

constexpr int kRowWarps = 4;
constexpr int kMaxDim = QX_MAX_HEAD_DIM;

// Any head size: one CTA per row, its warps taking blocks of 32 keys in turn
// (a lane scores a key, then owns every 32nd output element), joined at the
// end.  It serves the head sizes that the kernels below do not (all but 64 and
// 128), keeps the probabilities in f32, and reads a key once for every row: 8
// tokens over 2000 keys, 32 query heads of 80 over 8, take it 299 us (with the
// values' loads past a branch 400), where the split kernel takes 20.5 at head size
// 128.
template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps, 8) attn_row_kernel(const __grid_constant__ AttnParams p) {
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
    RowSums<kMaxDim / 32> r;
    row_sums<T, 4>(p, seq, pos, hk, 0, INT64_MAX, 32 * warp, 32 * kRowWarps,
                [&](int d, float (&x)[8]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = q[d + e];
                },
                r);
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) r.l += __shfl_xor_sync(0xffffffffu, r.l, w);
    if (lane == 0) om[warp] = r.m, ol[warp] = r.l;
#pragma unroll
    for (int e = 0; e < kMaxDim / 32; ++e)
        if (lane + 32 * e < dim) oo[warp][lane + 32 * e] = r.o[e];
    __syncthreads();
    float M = -FLT_MAX, L = 0.0f, a[kRowWarps];
    for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, om[w]);
    for (int w = 0; w < kRowWarps; ++w) {
        a[w] = exp2f(om[w] - M);
        L += a[w] * ol[w];
    }
    const int64_t row = int64_t(t) * p.n_q_heads + h;
    if (p.lse && threadIdx.x == 0) p.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    for (int d = threadIdx.x; d < dim; d += 32 * kRowWarps) {
        float v = 0.0f;
        for (int w = 0; w < kRowWarps; ++w) v += a[w] * oo[w][d];
        v = L == 0.0f ? 0.0f : v / L;
        if (p.out_f32) static_cast<float*>(p.out)[row * dim + d] = v;
        else static_cast<T*>(p.out)[row * dim + d] = from_f32<T>(v);
    }
}

// ---------------------------------------------------------------------------
// Few rows a sequence: the keys split over the whole GPU
// ---------------------------------------------------------------------------
//
// Decode reads each visible key and value once and multiplies them with the
// few rows of their group, so it is bound by those bytes.  The rows of one
// sequence and key head (its tokens times the group's query heads), sixteen at
// a time, are a tile; a tile's visible keys are cut into units of 64.  All
// units of all tiles form one line that the workers (CTAs, two per SM) share
// out evenly, whatever the lengths of the sequences: worker w takes units
// [w U / N, (w + 1) U / N).  A tile inside one worker's share is written by
// it; a tile that several share is joined by the last of them to arrive, from
// the others' (m, l, o) in the order of the workers, so the result does not
// depend on who is last.
//
// In a CTA a producer warp walks the line and fetches the units by TMA (one
// box a page, 128-byte swizzle, so that ldmatrix meets no bank conflict) into
// a ring of 96 KB, 64 KB of it ahead of the products; each of four warps takes
// 16 of a unit's keys with an online softmax of its own and meets the others
// only where the tile ends.  Products: mma.sync m16n8k16, whose 16 rows the
// group fills at most partly; the tensor pipe is not what bounds this kernel.
//
// Measured: 64 tokens over windows of 4096 keys (8 key heads of 128, bf16, 0.94
// GB) 149 us, 6.3 TB/s, 93 % of the measured copy rate; 256 over up to 1000 keys
// 97 us (81 %: a tile has eight units, and its join and its queries' way cost
// about two); one over 131072 keys 91 us (87 %); one over 1023 keys 7.7 us, of
// which 2 us are spent finding the worker's place and 3 us joining.

constexpr int kUnit = 64;                // keys of a unit
constexpr uint64_t kSplitWaitNs = 10000000000ull;  // (four_again() over millions of keys may be waited for)
constexpr int kSplitWarps = 4;
// A second warpgroup for the producer (its other three warps only give up
// registers): 128 registers a thread at launch, of which the consumers, who hold
// a tile's queries and output, take most.
constexpr int kSplitThreads = 2 * 32 * kSplitWarps;
constexpr int kConsumerRegs = 176, kProducerRegs = 80;
static_assert(kConsumerRegs + kProducerRegs <= 2 * 128, "registers the CTA was launched with");
constexpr int kRows = 16;                // rows of a tile
constexpr int kRingBytes = 96 * 1024;    // of one CTA; two CTAs fit on an SM

template <int DIM>
struct SplitGeom {
    static constexpr int kPanels = DIM / 64;                  // 64 elements (128 bytes) of every key
    static constexpr int kPanelBytes = kUnit * 128;
    static constexpr int kHalfStage = kPanels * kPanelBytes;  // a unit's keys; its values follow
    static constexpr int kStages = kRingBytes / (2 * kHalfStage);
    static constexpr int kJoin = (kSplitWarps * 8 * (DIM + 2)) * 4;  // joining buffer: 8 rows of each warp, then their m and l
    static constexpr int kMisc = 640;     // barriers, what is known of each unit, the worker's place on the line
    static constexpr size_t kSmem = kRingBytes + kJoin + kMisc;
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
};

// Scratch: arrival counters (one a worker, and 64 words for the tensor-core
// kernel's; zero between calls), then two partial tiles a worker: o [16][DIM], then m and l of the 16 rows.
constexpr int kMaxWorkers = 512;
constexpr size_t kCounterBytes = QX_ATTN_COUNTER_BYTES;
static_assert(kCounterBytes == (kMaxWorkers + 64) * 4, "the counters");
template <int DIM>
__host__ __device__ constexpr int partial_floats() { return kRows * DIM + 2 * kRows; }

__device__ __forceinline__ void ldmatrix4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// What a sequence brings: its tokens, and the keys that any of them sees --
// the first `sinks` (only where the window of the first token begins later)
// and [lo, end) -- as units of 64: those of the sinks, then those from the
// unit of lo on.  At least one unit, so that rows that see nothing are written.
struct SeqWork {
    int t0, tokens;        // first token, tokens
    int row_tiles;         // tiles of 16 rows for each key head
    int sink_units, units; // of one tile
    int pos0;              // position of the first token
    int lo, end, sinks;
};
constexpr int kMostKeys = INT32_MAX - 4 * kUnit;  // of a sequence: key numbers stay in 32 bits
__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, int b, int group, bool report) {
    SeqWork w;
    if (b == p.kv.n_seqs) {  // every token against the shared prefix (their positions are looked up)
        const int total = p.kv.q_start[b];
        const int64_t room = p.kv.table_stride << p.kv.page_shift, most = room < kMostKeys ? room : kMostKeys;
        w.t0 = w.pos0 = w.lo = w.sinks = w.sink_units = 0;
        w.tokens = total < p.n_tokens ? total : p.n_tokens;
        w.end = int(p.shared_len < most ? p.shared_len : most);
        w.units = (w.end + kUnit - 1) / kUnit;
        w.row_tiles = (w.tokens * group + kRows - 1) / kRows;
        return w;
    }
    w.t0 = p.kv.q_start[b];
    w.tokens = p.kv.q_start[b + 1] - w.t0;
    const int kv = p.kv.kv_len[b];
    if (w.tokens < 0 || w.t0 < 0 || w.t0 + w.tokens > p.n_tokens) w.tokens = 0;  // not an ascending list of this call's tokens
    w.pos0 = kv - w.tokens;
    const int64_t room = p.kv.table_stride << p.kv.page_shift;
    const int most = room < kMostKeys ? int(room) : kMostKeys;
    if (kv > most && report) atomicOr(p.kv.err, kErrRange);
    w.end = kv < 0 ? 0 : kv < most ? kv : most;
    const int window = p.window < INT32_MAX ? int(p.window) : 0;
    const int shared = p.shared_len < INT32_MAX ? int(p.shared_len) : INT32_MAX;
    w.lo = window > 0 && w.pos0 >= window ? w.pos0 - window + 1 : 0;
    if (w.lo < shared) w.lo = shared;
    if (w.lo > w.end) w.lo = w.end;
    w.sinks = shared > 0 ? 0 : p.sinks < w.lo ? int(p.sinks) : w.lo;
    w.sink_units = (w.sinks + kUnit - 1) / kUnit;
    w.units = w.sink_units + (w.end > w.lo ? (w.end + kUnit - 1) / kUnit - w.lo / kUnit : 0);
    if (w.units < 1) w.units = 1;
    w.row_tiles = (w.tokens * group + kRows - 1) / kRows;
    return w;
}

// A place on the line of units: tile (sequence b, row tile rt, key head hk),
// whose units are [begin, begin + w.units) of the line.
struct Cursor {
    int64_t begin;
    int b, rt, hk;
    SeqWork w;
};
__device__ __forceinline__ void next_tile(const AttnParams& p, Cursor& c, int group, int seqs) {
    c.begin += c.w.units;
    if (++c.hk < p.kv.n_heads) return;
    c.hk = 0;
    if (++c.rt < c.w.row_tiles) return;
    c.rt = 0;
    do {
        if (++c.b >= seqs) return;
        c.w = seq_work(p, c.b, group, false);
    } while (c.w.row_tiles == 0);
}
// The first key of unit u of a tile, and the keys [lo, hi) of it that any row sees.
__device__ __forceinline__ int unit_keys(const SeqWork& w, int u, int& lo, int& hi) {
    const bool sink = u < w.sink_units;
    lo = sink ? 0 : w.lo;
    hi = sink ? w.sinks : w.end;
    return (sink ? u : w.lo / kUnit + (u - w.sink_units)) * kUnit;
}

// What the consumers are told of a unit, beside its keys and values in the
// ring: its first key and the keys [lo, hi) that any row sees; the tile's
// rows; and the workers that share the tile.
struct UnitInfo {
    int j0, lo, hi;
    int flags;           // kSink, kOpens, kCloses (for this worker), kPrefix
    int t0, r0, rows;    // the sequence's first token, the tile's first row and the rows from it on
    int hk, pos0;
    int wf, parts, part; // first worker, workers after it, and the part of the scratch that the first one writes
};
constexpr int kSink = 1, kOpens = 2, kCloses = 4, kPrefix = 8;

struct SplitParams {
    CUtensorMap k_map;  // [pages][heads][slots][dim], boxes of min(page, 64) keys x 64
    CUtensorMap v_map;
    AttnParams a;
    float* part_o;    // not null: the rows are a part to be joined (o / l, base-2 log of the sum)
    float* part_lse;
    int beside;       // 1: launched beside the kernel before it, which belongs to the same call
    int prefix;       // 1: the shared prefix, too: its tiles end the line, and give part 0, the tails part 1
};

// Quotients of non-negative numbers, in 32 bits where they fit (nearly always).
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return int64_t(uint32_t(a) / uint32_t(b));
    return a / b;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kSplitWarps) : "memory"); }
// The same, and whether every consumer came with `ok`: the answer is the same
// for all, so they go on together or leave together.  (`ok` is warp-uniform.)
__device__ __forceinline__ bool consumers_agree(bool ok) {
    uint32_t all;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, 1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(all)
        : "r"(ok ? 1u : 0u), "n"(32 * kSplitWarps)
        : "memory");
    return all != 0;
}

// The consumers' barrier, and whether any thread came with `flag`.
__device__ __forceinline__ bool consumers_any(bool flag) {
    uint32_t any;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred q, 1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(any)
        : "r"(flag ? 1u : 0u), "n"(32 * kSplitWarps)
        : "memory");
    return any != 0;
}

// Four elements of row r of a tile (its sum o, not divided yet).  True, where
// `look`: one of them is infinite or no number though the sum of the row's
// probabilities is neither.
template <typename T, int DIM>
__device__ __forceinline__ bool write_four(const SplitParams& pp, const UnitInfo& tile, int r, int d, float M, float L, float4 v, bool look) {
    const AttnParams& p = pp.a;
    const int group = p.n_q_heads / p.kv.n_heads, rr = tile.r0 + r;
    const int64_t row = int64_t(tile.t0 + rr / group) * p.n_q_heads + tile.hk * group + rr % group;
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
    const bool odd = look && !(0.0f * (v.x + v.y + v.z + v.w) == 0.0f) && L == L;
    if (pp.part_o) {
        const int64_t at = row + (pp.prefix && !(tile.flags & kPrefix) ? int64_t(p.n_tokens) * p.n_q_heads : 0);
        *reinterpret_cast<float4*>(pp.part_o + at * DIM + d) = v;
        if (d == 0) pp.part_lse[at] = L == 0.0f ? -INFINITY : M + log2f(L);
        return odd;
    }
    if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * DIM + d) = v;
    else *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * DIM + d) = make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
    if (p.lse && d == 0) p.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    return odd;
}
// Such a row once more, by one warp.
template <typename T, int DIM>
__device__ __forceinline__ void four_again(const SplitParams& pp, const UnitInfo& tile, int r) {
    const AttnParams& p = pp.a;
    const int group = p.n_q_heads / p.kv.n_heads, rr = tile.r0 + r;
    const int t = tile.t0 + rr / group, h = tile.hk * group + rr % group, seq = seq_of_token(p.kv, t);
    if (seq < 0) return;
    const bool prefix = tile.flags & kPrefix;
    // the keys that were fetched and it does not see: later ones, and those of the first token's window before its own
    const int64_t pos = position_of(p.kv, seq, t), room = p.kv.table_stride << p.kv.page_shift;
    const int64_t end = prefix ? p.shared_len : p.kv.kv_len[seq], later = pos + 1 > 0 ? pos + 1 : 0;
    const int64_t first = p.window > 0 ? position_of(p.kv, seq, p.kv.q_start[seq]) + 1 - p.window : 0;
    if (!odd_values<T, DIM>(p, prefix ? 0 : seq, tile.hk, later > p.shared_len || prefix ? later : p.shared_len, end < room ? end : room) &&
        !(p.window > 0 && odd_values<T, DIM>(p, seq, tile.hk, first > p.sinks ? first : p.sinks, pos + 1 - p.window)))
        return;
    const T* q = static_cast<const T*>(p.q) + int64_t(t) * p.q_stride + int64_t(h) * DIM;
    RowSums<DIM / 32> sums;
    row_sums<T, 4>(p, prefix ? 0 : seq, pos, tile.hk, prefix ? 0 : p.shared_len, prefix ? p.shared_len : INT64_MAX, 0, 32,
                [&](int d, float (&x)[8]) { load_f32<8>(q + d, x); }, sums);
    const int64_t row = int64_t(t) * p.n_q_heads + h;
    if (pp.part_o) {
        const int64_t at = row + (pp.prefix && !prefix ? int64_t(p.n_tokens) * p.n_q_heads : 0);
        write_row_again<T, DIM>(sums, pp.part_o, true, at * DIM);
    } else {
        write_row_again<T, DIM>(sums, p.out, p.out_f32, row * DIM);
    }
}

// (M, L) and (m, l) become one maximum and one sum.  Sums over scores that are
// no numbers have a maximum of -inf, and stay what they are.
__device__ __forceinline__ void join_sums(float& M, float& L, float m, float l) {
    const float mn = fmaxf(M, m), base = mn == -INFINITY ? 0.0f : mn;
    L = L * exp2_approx(M - base) + l * exp2_approx(m - base);
    M = mn;
}

// The parts of a tile that several workers shared, joined by the consumers of
// the last of them to arrive.  The rows of which write_four says so, as bits.
template <typename T, int DIM>
__device__ __forceinline__ uint32_t join_parts(const SplitParams& pp, const UnitInfo& tile, float* buf, bool look) {
    float* partials = reinterpret_cast<float*>(static_cast<uint8_t*>(pp.a.scratch) + kCounterBytes);
    float* buf_ml = buf + kSplitWarps * 8 * DIM;
    const int live = tile.rows < kRows ? tile.rows : kRows, parts = tile.parts + 1;
    const float* const begin = partials + int64_t(tile.part) * partial_floats<DIM>();
    const float* const rest = partials + int64_t(2 * (tile.wf + 1)) * partial_floats<DIM>();
    constexpr int64_t kStep = 2 * partial_floats<DIM>();
    const auto src = [&](int i) -> const float* { return i == 0 ? begin : rest + (i - 1) * kStep; };
    // eight threads a row find its maximum and sum, and leave each part's
    // weight in the buffer
    float* weight = buf;  // [16][parts], where that fits
    const bool fits = kRows * parts <= kSplitWarps * 8 * DIM;
    const int r8 = threadIdx.x >> 3, i8 = threadIdx.x & 7;
    float M = -INFINITY, L = 0.0f;
    if (r8 < live) {
#pragma unroll 4
        for (int i = i8; i < parts; i += 8) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(src(i) + kRows * DIM + 2 * r8));
            join_sums(M, L, ml.x, ml.y);
            if (fits) weight[r8 * parts + i] = ml.x;
        }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, M, o), ol = __shfl_xor_sync(0xffffffffu, L, o);
        join_sums(M, L, om, ol);
    }
    if (r8 < live) {
        if (fits)
            for (int i = i8; i < parts; i += 8) {
                const float m = weight[r8 * parts + i];
                weight[r8 * parts + i] = m == -INFINITY ? 0.0f : exp2_approx(m - M);
            }
        if (i8 == 0) *reinterpret_cast<float2*>(buf_ml + 2 * r8) = make_float2(M, L);
    }
    consumers_sync();
    uint32_t odd = 0;
    for (int x = threadIdx.x; x < live * (DIM / 4); x += 32 * kSplitWarps) {
        const int r = x / (DIM / 4), d = x % (DIM / 4) * 4;
        const float2 ml = *reinterpret_cast<const float2*>(buf_ml + 2 * r);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // eight parts' loads in flight at a time
        for (int w0 = 0; w0 < parts; w0 += 8) {
            float4 v[8];
#pragma unroll
            for (int y = 0; y < 8; ++y)
                v[y] = __ldcg(reinterpret_cast<const float4*>(src(w0 + y < parts ? w0 + y : parts - 1) + r * DIM + d));
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                if (w0 + y >= parts) break;
                float c;
                if (fits) {
                    c = weight[r * parts + w0 + y];
                } else {
                    const float m = __ldcg(src(w0 + y) + kRows * DIM + 2 * r);
                    c = m == -INFINITY ? 0.0f : exp2_approx(m - ml.x);
                }
                acc.x += c * v[y].x, acc.y += c * v[y].y, acc.z += c * v[y].z, acc.w += c * v[y].w;
            }
        }
        if (write_four<T, DIM>(pp, tile, r, d, ml.x, ml.y, acc, look)) odd |= 1u << r;
    }
    return odd;
}

template <typename T, int DIM>
__global__ void __launch_bounds__(kSplitThreads, 2) attn_split_kernel(const __grid_constant__ SplitParams pp) {
    using G = SplitGeom<DIM>;
    constexpr int KS = DIM / 16;  // 16-wide steps along a head
    constexpr int NS = G::kStages;
    const AttnParams& p = pp.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* buf = reinterpret_cast<float*>(smem + kRingBytes);  // [4 warps][8 rows][DIM], then m and l of each
    float* buf_ml = buf + kSplitWarps * 8 * DIM;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRingBytes + G::kJoin);
    uint64_t* empty = full + NS;
    int64_t* scan = reinterpret_cast<int64_t*>(empty + NS);  // [8]
    Cursor* start = reinterpret_cast<Cursor*>(scan + 2 * kSplitWarps);
    UnitInfo* info = reinterpret_cast<UnitInfo*>(start + 1);  // [NS]
    int* last_flag = reinterpret_cast<int*>(info + NS);
    static_assert((2 * NS + 2 * kSplitWarps) * 8 + sizeof(Cursor) + NS * sizeof(UnitInfo) + 4 <= G::kMisc,
                  "barriers, units and the worker's place");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 2);  // the copies, and the description
            mbar_init(&empty[i], kSplitWarps);
        }
        fence_barrier_init();
        prefetch_map(&pp.k_map);
        prefetch_map(&pp.v_map);
    }
    // Beside a kernel that works on the same call's prefix: that one has
    // waited for the work before it, and this one reads nothing of its.
    if (!pp.beside) pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int group = p.n_q_heads / p.kv.n_heads;
    const int B = p.kv.n_seqs + pp.prefix;

    // ---- the line's length, and where this worker's share begins
    int64_t mine = 0;
    const int per = (B + kSplitThreads - 1) / kSplitThreads, b0 = threadIdx.x * per;
    SeqWork own;  // of the thread's last sequence (its only one, for up to 256 sequences)
    for (int b = b0; b < b0 + per && b < B; ++b) {
        own = seq_work(p, b, group, blockIdx.x == 0);
        mine += int64_t(own.row_tiles) * p.kv.n_heads * own.units;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t U = 0, before = 0;
#pragma unroll
    for (int w = 0; w < 2 * kSplitWarps; ++w) {
        if (w < warp) before += scan[w];
        U += scan[w];
    }
    // (two units each at least: one token over 1023 keys took 8.5 us with one)
    const int64_t pairs = (U + 1) / 2, N = gridDim.x < pairs ? gridDim.x : pairs;
    if (blockIdx.x >= N) {
        if (pp.beside) pdl_wait_prior_grid();
        return;
    }
    // the first `extra` workers have one unit more than the others
    const int64_t share = quot(U, N), extra = U - share * N;
    const auto begin_of = [&](int64_t w) { return w * share + (w < extra ? w : extra); };
    const auto worker_of = [&](int64_t u) {
        return u < extra * (share + 1) ? quot(u, share + 1) : extra + quot(u - extra * (share + 1), share);
    };
    const int64_t first = begin_of(blockIdx.x), last = begin_of(blockIdx.x + 1);  // this worker's units
    int64_t at = before + incl - mine;
    if (first >= at && first < at + mine) {
        for (int b = b0; b < b0 + per && b < B; ++b) {
            if (per > 1) own = seq_work(p, b, group, false);
            const int64_t n = int64_t(own.row_tiles) * p.kv.n_heads * own.units;
            if (first < at + n) {
                const int64_t tile = quot(first - at, own.units);
                start->b = b;
                start->w = own;
                start->begin = at + tile * own.units;
                start->rt = int(quot(tile, p.kv.n_heads));
                start->hk = int(tile - int64_t(start->rt) * p.kv.n_heads);
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    int64_t left = last - first;  // units to go
    const auto describe = [&](const Cursor& c, int u, UnitInfo& x) {
        x.j0 = unit_keys(c.w, u, x.lo, x.hi);
        const int64_t begin = c.begin, end = c.begin + c.w.units, here = begin + u;
        x.flags = (u < c.w.sink_units ? kSink : 0) | (here == first || u == 0 ? kOpens : 0) | (here + 1 == last || here + 1 == end ? kCloses : 0) |
                  (c.b == p.kv.n_seqs ? kPrefix : 0);
        x.t0 = c.w.t0;
        x.r0 = kRows * c.rt;
        x.rows = c.w.tokens * group - x.r0;
        x.hk = c.hk;
        x.pos0 = c.w.pos0;
        // only a worker's first and last tile may be shared; its part of a
        // tile lies in its first slot, or in its second where another tile's
        // end came first
        const int64_t wf = begin < first ? worker_of(begin) : blockIdx.x, wl = end > last ? worker_of(end - 1) : blockIdx.x;
        x.wf = int(wf);
        x.parts = int(wl - wf);
        x.part = 2 * int(wf) + (begin_of(wf) < begin ? 1 : 0);
    };

    if (warp >= kSplitWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        if (warp > kSplitWarps) {
            if (pp.beside) pdl_wait_prior_grid();
            return;
        }
        // ---- producer: a lane for each page of a unit
        Cursor cur = *start;
        int ui = int(first - cur.begin);  // unit of the tile
        const int page_keys = (1 << p.kv.page_shift) < kUnit ? (1 << p.kv.page_shift) : kUnit;
        const int in_page_mask = (1 << p.kv.page_shift) - 1;
        const int boxes = kUnit / page_keys;  // at most 4
        // the lane's page of unit ui, or -1 where no row sees any of its keys
        const auto page_for = [&](int u) -> int {
            int lo, hi;
            const int j = unit_keys(cur.w, u, lo, hi) + lane * page_keys;
            return lane < boxes && j + page_keys > lo && j < hi ? page_of(p.kv, cur.b < p.kv.n_seqs ? cur.b : 0, j) : -1;
        };
        int page = page_for(ui);
        int slot = 0;
        uint32_t phase = 1;  // the ring is empty at first: the wait for the phase before the first returns
        bool ok = true;
        int used = 0;
        for (; left > 0; --left) {
            int lo, hi;
            const int j0 = unit_keys(cur.w, ui, lo, hi);
            const int in_page = (j0 + lane * page_keys) & in_page_mask;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[slot], phase, kSplitWaitNs, p.kv.err, kErrTimeoutEmpty));
            if (!ok) break;
            const unsigned live = __ballot_sync(0xffffffffu, page >= 0);
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], __popc(live) * page_keys * 128 * G::kPanels * 2);
            __syncwarp();
            if (page >= 0) {
                uint8_t* dst = smem + slot * 2 * G::kHalfStage + lane * page_keys * 128;
#pragma unroll
                for (int c = 0; c < G::kPanels; ++c) {
                    tma_load_4d(dst + c * G::kPanelBytes, &pp.k_map, 64 * c, in_page, cur.hk, page, &full[slot]);
                    tma_load_4d(dst + G::kHalfStage + c * G::kPanelBytes, &pp.v_map, 64 * c, in_page, cur.hk, page, &full[slot]);
                }
            }
            if (lane == 0) {  // while they are on their way
                UnitInfo x;
                describe(cur, ui, x);
                info[slot] = x;
                mbar_arrive(&full[slot]);
            }
            __syncwarp();
            if (left > 1) {  // the next unit's pages are looked up while its room is awaited
                if (++ui == cur.w.units) {
                    next_tile(p, cur, group, B);
                    ui = 0;
                }
                page = page_for(ui);
            }
            if (used < NS) ++used;
            if (++slot == NS) {
                slot = 0;
                phase ^= 1;
            }
        }
        // keep the CTA alive until every copy it issued has landed
        if (lane == 0) {
            for (int i = 0; i < used; ++i) {  // the last `used` slots, most recent first
                if (--slot < 0) {
                    slot = NS - 1;
                    phase ^= 1;
                }
                mbar_wait_bounded(&full[slot], phase ^ 1, kSplitWaitNs, p.kv.err, kErrTimeoutDrain);
            }
        }
        if (pp.beside) pdl_wait_prior_grid();
        return;
    }

    // ---- consumers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
    uint32_t qf[KS][4];
    float o[DIM / 8][4], m[2], l[2];
    int rpos[2];             // positions of this lane's two rows (-1: none)
    int pos_first, pos_last; // of the tile's rows
    // A tile's rows: 16 rt + lane / 4 and eight further.
    const auto open_tile = [&](const UnitInfo& x) {
        const int live_rows = x.rows < kRows ? x.rows : kRows;
        int low = INT32_MAX, high = -1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (lane >> 2) + 8 * i;
            const bool live = r < live_rows;
            const int tok = (x.r0 + (live ? r : 0)) / group, g = x.r0 + (live ? r : 0) - tok * group;
            int pos = x.pos0 + tok;
            if (x.flags & kPrefix) {
                const int seq = live ? seq_of_token(p.kv, tok) : -1;
                pos = seq < 0 ? -1 : int(position_of(p.kv, seq, tok));
            }
            rpos[i] = live && pos >= 0 ? pos : -1;
            if (live) low = low < rpos[i] ? low : rpos[i], high = high > rpos[i] ? high : rpos[i];
            const T* q = static_cast<const T*>(p.q) + int64_t(x.t0 + tok) * p.q_stride + int64_t(x.hk * group + g) * DIM + 2 * (lane & 3);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][i] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * k) : 0u;
                qf[k][i + 2] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8) : 0u;
            }
        }
        pos_first = __reduce_min_sync(0xffffffffu, low);
        pos_last = __reduce_max_sync(0xffffffffu, high);
    };
    {
        UnitInfo x;
        x.t0 = start->w.t0, x.pos0 = start->w.pos0, x.hk = start->hk;
        x.r0 = kRows * start->rt, x.rows = start->w.tokens * group - x.r0;
        x.flags = start->b == p.kv.n_seqs ? kPrefix : 0;
        open_tile(x);
    }
    float* partials = reinterpret_cast<float*>(static_cast<uint8_t*>(p.scratch) + kCounterBytes);
    unsigned* counters = static_cast<unsigned*>(p.scratch);
    const int window = p.window > 0 && p.window < INT32_MAX ? int(p.window) : INT32_MAX;
    const int sinks = p.sinks < INT32_MAX ? int(p.sinks) : INT32_MAX;
    // This lane's part of the ldmatrix addresses, relative to a stage: keys
    // 16 warp + (0-7 and 8-15 by d 0-7 and 8-15 of a step), and values 16 warp
    // + (0-15 by d 0-7 and 8-15).
    const uint32_t ring = smem_addr(smem);
    const int kr = 16 * warp + (lane & 7) + ((lane >> 4) << 3), kh = (lane >> 3) & 1;
    const int vr = 16 * warp + (lane & 15), vh = lane >> 4;
    const uint32_t k_row = ring + kr * 128, v_row = ring + G::kHalfStage + vr * 128;
    int slot = 0;
    uint32_t phase = 0;
    // A wait that runs out ends the consumers, but not at the same time: each
    // warp waits by itself, and copies may land between two warps' limits.  So
    // the first barrier of a tile's end asks whether all four are there, and a
    // warp that gave up comes to it once more (it is the next barrier of the
    // others, whatever tile they are at: every worker's line ends with a tile's
    // end).  All four leave there; none is left at a barrier.
    bool ok = true, together = true;
    const auto arrived = [&]() {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[slot], phase, kSplitWaitNs, p.kv.err, kErrTimeoutFull));
    };
    arrived();
    for (; left > 0 && ok; --left) {
        const int flags = info[slot].flags, lo = info[slot].lo, hi = info[slot].hi;
        const int j0 = info[slot].j0 + 16 * warp;  // this warp's sixteen keys
        if (flags & kOpens) {
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.0f;
#pragma unroll
            for (int d = 0; d < DIM / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.0f;
        }
        if (j0 + 16 > lo && j0 < hi) {
            const uint32_t off = slot * 2 * G::kHalfStage;
            float s[2][4] = {};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t b[4];
                ldmatrix4(k_row + off + (k >> 2) * G::kPanelBytes + (((2 * (k & 3) + kh) ^ (kr & 7)) << 4), b);
                mma16816<T>(s[0], qf[k], b[0], b[1]);
                mma16816<T>(s[1], qf[k], b[2], b[3]);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] *= p.scale_log2;
            const bool sink_unit = flags & kSink;
            if (j0 < lo || j0 + 16 > hi || j0 + 15 > pos_first || (!sink_unit && pos_last - window >= j0)) {
                // some row does not see some of them.  This lane's keys,
                // relative to the first: 2 (lane % 4) + {0, 1, 8, 9}.
                const int a = lo - j0, b = hi - j0, c = sinks - j0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int end = rpos[i] - j0 + 1 < b ? rpos[i] - j0 + 1 : b;
                    const int low = rpos[i] >= window ? rpos[i] - window + 1 : 0;  // of the row's window
                    const int from = sink_unit || low - j0 < a ? a : low - j0;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = 8 * n + 2 * (lane & 3) + e;
                            if (!(j < end && (j >= from || (j >= a && j < c)))) s[n][2 * i + e] = -INFINITY;
                        }
                }
                // Values that no row sees are zeroed: whatever the slots hold, 0 x it must be 0.
                if (j0 < lo || j0 + 16 > hi) {
                    if (vr - 16 * warp < a || vr - 16 * warp >= b) {
#pragma unroll
                        for (int c2 = 0; c2 < G::kPanels; ++c2)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                *reinterpret_cast<uint4*>(smem + slot * 2 * G::kHalfStage + G::kHalfStage + c2 * G::kPanelBytes + vr * 128 +
                                                          64 * vh + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();  // before the slot's next copy
                    __syncwarp();
                }
            }
            float mx[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[i] = fmaxf(m[i], fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1])));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            }
            // the maximum moves less and less often: o is rescaled only when it does
            if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
                float a[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    a[i] = mx[i] == -INFINITY ? 1.0f : exp2_approx(m[i] - mx[i]);
                    l[i] *= a[i];
                    m[i] = mx[i];
                }
#pragma unroll
                for (int d = 0; d < DIM / 8; ++d) {
                    o[d][0] *= a[0], o[d][1] *= a[0];
                    o[d][2] *= a[1], o[d][3] *= a[1];
                }
            }
            const float base[2] = {m[0] == -INFINITY ? 0.0f : m[0] - kLift<T, 0>, m[1] == -INFINITY ? 0.0f : m[1] - kLift<T, 0>};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = exp2_approx(s[n][e] - base[e >> 1]);
                    l[e >> 1] += s[n][e];
                }
            const uint32_t pf[4] = {pack2<T>(s[0][0], s[0][1]), pack2<T>(s[0][2], s[0][3]), pack2<T>(s[1][0], s[1][1]),
                                    pack2<T>(s[1][2], s[1][3])};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t b[4];
                ldmatrix4_t(v_row + off + (k >> 2) * G::kPanelBytes + (((2 * (k & 3) + vh) ^ (vr & 7)) << 4), b);
                mma16816<T>(o[2 * k], pf, b[0], b[1]);
                mma16816<T>(o[2 * k + 1], pf, b[2], b[3]);
            }
        }
        const UnitInfo* const x = &info[slot];
        UnitInfo done;
        if (flags & kCloses) done = *x;
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (++slot == NS) {
            slot = 0;
            phase ^= 1;
        }
        if (left > 1) arrived();
        if (!(flags & kCloses)) continue;
        // ---- the tile ends here (for this worker).  The next one's queries
        // are on their way while its warps are joined, eight rows at a time:
        // every warp leaves its (m, l, o), and every thread then joins some
        // elements.
        if (left > 1 && ok) open_tile(info[slot]);
        const int rows = done.rows;  // (16 at most count)
        const auto part_at = [&](int i) -> float* { return partials + int64_t(i) * partial_floats<DIM>(); };
        const bool look = done.r0 + rows != group;  // (a sequence's only token sees all that was fetched)
        uint32_t odd = 0;                           // rows that write_four found odd
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (8 * i >= rows) break;
            const int live = rows - 8 * i < 8 ? rows - 8 * i : 8;
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (i > 0) consumers_sync();  // the first eight are read
            if ((lane >> 2) < live) {
                // (groups of eight elements permuted by the row, for the banks)
                float* row = buf + (8 * warp + (lane >> 2)) * DIM + 2 * (lane & 3);
#pragma unroll
                for (int d = 0; d < DIM / 8; ++d)
                    *reinterpret_cast<float2*>(row + 8 * (d ^ (lane >> 2))) = make_float2(o[d][2 * i], o[d][2 * i + 1]);
                if ((lane & 3) == 0) *reinterpret_cast<float2*>(buf_ml + 2 * (8 * warp + (lane >> 2))) = make_float2(m[i] - kLift<T, 0>, l[i]);
            }
            if (i > 0) consumers_sync();
            else if (!(together = consumers_agree(ok))) break;
            for (int x = threadIdx.x; x < live * (DIM / 4); x += 32 * kSplitWarps) {
                const int r = x / (DIM / 4), d = x % (DIM / 4) * 4;
                float2 ml[kSplitWarps];
                float M = -INFINITY, L = 0.0f;
#pragma unroll
                for (int w = 0; w < kSplitWarps; ++w) {
                    ml[w] = *reinterpret_cast<const float2*>(buf_ml + 2 * (8 * w + r));
                    M = fmaxf(M, ml[w].x);
                }
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kSplitWarps; ++w) {
                    const float a = ml[w].x == -INFINITY ? 0.0f : exp2_approx(ml[w].x - M);
                    const float4 v = *reinterpret_cast<const float4*>(buf + (8 * w + r) * DIM + (d ^ (8 * r)));
                    L += a * ml[w].y;
                    acc.x += a * v.x, acc.y += a * v.y, acc.z += a * v.z, acc.w += a * v.w;
                }
                if (done.parts == 0) {
                    if (write_four<T, DIM>(pp, done, 8 * i + r, d, M, L, acc, look)) odd |= 1u << (8 * i + r);
                } else {
                    float* to = part_at(int(blockIdx.x) == done.wf ? done.part : 2 * int(blockIdx.x));
                    *reinterpret_cast<float4*>(to + (8 * i + r) * DIM + d) = acc;
                    if (d == 0) *reinterpret_cast<float2*>(to + kRows * DIM + 2 * (8 * i + r)) = make_float2(M, L);
                }
            }
        }
        if (!together) break;
        if (done.parts > 0) {
            // ---- this worker's part is written; the last to arrive joins all
            consumers_sync();
            if (threadIdx.x == 0) {
                __threadfence();  // for all, behind the barrier
                const unsigned n = atomicAdd(&counters[done.wf], 1u);
                *last_flag = n == unsigned(done.parts);
                if (*last_flag) {
                    counters[done.wf] = 0;  // for the next call
                    __threadfence();
                }
            }
            consumers_sync();
            if (*last_flag) odd = join_parts<T, DIM>(pp, done, buf, look);
        }
        if (!look) {
            consumers_sync();  // the buffer is read
        } else if (consumers_any(odd != 0)) {
            unsigned* const mask = reinterpret_cast<unsigned*>(buf);
            if (threadIdx.x == 0) *mask = 0;
            consumers_sync();
            if (odd) atomicOr(mask, odd);
            consumers_sync();
            for (int r = warp; r < kRows; r += kSplitWarps)
                if (*mask & (1u << r)) four_again<T, DIM>(pp, done, r);
            consumers_sync();
        }
    }
    if (!ok && together) consumers_agree(false);
    if (pp.beside) pdl_wait_prior_grid();  // complete only after that kernel, too
}

// Four consumers of which the first gives up on a unit after `limit_ns`, before
// it arrives (half a limit later), and the others do not: who went on past the
// barrier, by warp (test hook).
__global__ void __launch_bounds__(32 * (kSplitWarps + 1)) agree_probe_kernel(uint64_t limit_ns, int* got, unsigned* err) {
    __shared__ __align__(8) uint64_t full;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&full, 1);
        fence_barrier_init();
    }
    __syncthreads();
    if (warp == kSplitWarps) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < limit_ns + limit_ns / 2) {}
        if (lane == 0) mbar_arrive(&full);
        return;
    }
    const uint64_t limit = warp == 0 ? limit_ns : 100 * limit_ns;
    const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full, 0, limit, err, kErrTimeoutProbe));
    const bool together = consumers_agree(ok);
    if (lane == 0) got[warp] = (ok ? 1 : 0) | (together ? 2 : 0);
}

template <typename T, int DIM>
cudaError_t launch_split(SplitParams& p, int sm_count, cudaStream_t s) {
    if (!encode_cache_maps(!IsBf16<T>::value, p.a.kv, kUnit, &p.k_map, &p.v_map)) return cudaErrorInvalidValue;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(attn_split_kernel<T, DIM>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SplitGeom<DIM>::kSmem));
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    const int workers = 2 * sm_count < kMaxWorkers ? 2 * sm_count : kMaxWorkers;
    return launch_serial(attn_split_kernel<T, DIM>, dim3(unsigned(workers)), kSplitThreads, SplitGeom<DIM>::kSmem, s, p);
}

cudaError_t launch_split_any(int dtype, const AttnParams& a, float* part_o, float* part_lse, bool beside, bool prefix,
                             int sm_count, cudaStream_t s) {
    SplitParams p;
    p.a = a;
    p.part_o = part_o;
    p.part_lse = part_lse;
    p.beside = beside ? 1 : 0;
    p.prefix = prefix ? 1 : 0;
    const bool f16 = dtype == QX_F16;
    if (a.kv.head_dim == 128)
        return f16 ? launch_split<__half, 128>(p, sm_count, s) : launch_split<__nv_bfloat16, 128>(p, sm_count, s);
    return f16 ? launch_split<__half, 64>(p, sm_count, s) : launch_split<__nv_bfloat16, 64>(p, sm_count, s);
}

template <typename T>
cudaError_t launch_row(const AttnParams& p, cudaStream_t s) {
    return launch_serial(attn_row_kernel<T>, dim3(unsigned(p.n_tokens), unsigned(p.n_q_heads)), 32 * kRowWarps, 0, s, p);
}

constexpr size_t kSplitScratch = kCounterBytes + size_t(kMaxWorkers) * 2 * partial_floats<128>() * 4;
// Rows of parts that the scratch holds for a call of `rows` rows: every row
// split kMaxSplits ways, but no more than kPartRows rows in all (calls of that
// many rows fill the GPU without splitting their keys), or two parts of a call
// whose shared prefix is taken apart.
constexpr int kPrefixUnits = 10, kShortPrefix = 4096;
constexpr int kMaxSplits = 31;  // parts of one launch: with the tails' part a row has at most 32
constexpr int64_t kPartRows = 262144, kMaxSharedRows = 131072;
int64_t part_rows(int64_t rows) {
    int64_t n = rows < kPartRows / kMaxSplits ? rows * kMaxSplits : kPartRows;
    const int64_t two = 2 * (rows < kMaxSharedRows ? rows : kMaxSharedRows);
    if (n < two) n = two;
    return (n + 63) / 64 * 64;  // 256-byte multiples
}

// Parts of a row at most where the tensor-core kernel shares the key blocks of
// all pairs out evenly, or 0: every pair in one CTA.  Even shares are for calls
// of few pairs (fewer than kEvenPairs an SM, times the key heads): with more,
// the counter balances them, and parts cost their f32 bytes and a launch.  The
// scheduler of every CTA reads every sequence, so there are to be few of them.
constexpr int kEvenPairs = 3, kEvenSeqs = 32;
int slots_for(int64_t pairs, int64_t blocks, int seqs, int64_t rows, int64_t spare_rows, int sm_count) {
    if (pairs >= int64_t(kEvenPairs) * sm_count || seqs > kEvenSeqs || blocks < 12) return 0;
    int64_t n = blocks + 1 < kMaxSplits ? blocks + 1 : kMaxSplits;
    if (n * rows > spare_rows) n = spare_rows / rows;
    return n < 5 ? 0 : int(n);  // (with fewer the shares have to grow to fit a long pair's parts in)
}

}  // namespace

cudaError_t launch_agree_probe(uint64_t limit_ns, int* got, unsigned* err, cudaStream_t s) {
    agree_probe_kernel<<<1, 32 * (kSplitWarps + 1), 0, s>>>(limit_ns, got, err);
    return cudaGetLastError();
}

size_t attn_scratch_bytes(int64_t n_tokens, int n_q_heads, int, int head_dim, int) {
    // calls of up to this head size: only those of 64 and 128 leave parts
    const int dim = head_dim < 64 ? 0 : head_dim < 128 ? 64 : 128;
    return kSplitScratch + (dim > 0 ? size_t(part_rows(n_tokens * n_q_heads)) * (dim + 1) * 4 : 0);
}

cudaError_t launch_attn(int dtype, const AttnParams& params, int sm_count, cudaStream_t s) {
    AttnParams p = params;
    const int dim = p.kv.head_dim;
    if (dim != 64 && dim != 128) {
        p.shared_len = 0;  // every sequence's table leads to the prefix, too
        return dtype == QX_F16 ? launch_row<__half>(p, s) : launch_row<__nv_bfloat16>(p, s);
    }
    const int group = p.n_q_heads / p.kv.n_heads;
    const int64_t rows = int64_t(p.n_tokens) * p.n_q_heads;
    float* part_lse = reinterpret_cast<float*>(static_cast<char*>(p.scratch) + kSplitScratch);
    float* part_o = part_lse + part_rows(rows);
    // a scale that is not positive is an oddity that only the split kernel serves
    unsigned* counter = static_cast<unsigned*>(p.scratch) + kMaxWorkers;
    if (rows > kMaxSharedRows || p.n_tokens < 2 || p.scale_log2 <= 0.0f) p.shared_len = 0;
    // Rows of a key head a sequence, on average: the split kernel reads a
    // sequence's keys once for every 16 of them, the tensor cores' once for
    // 256, but only they need whole tiles to be efficient.
    const bool many = int64_t(p.n_tokens) * group >= 64 * int64_t(p.kv.n_seqs) && p.scale_log2 > 0.0f;
    JoinParams j;
    j.a = p;
    j.part_o = part_o;
    j.part_lse = part_lse;
    j.parts = 0;
    cudaError_t e;
    const int64_t spare = part_rows(rows);
    if (p.shared_len > 0) {
        // A short prefix for few rows: the split kernel takes it with the
        // tails, though it reads it once for every 16 rows.  (16 sequences
        // behind 2000 keys: 23 us, against 32 with a launch of its own; 64
        // behind 2000 or 16 behind 8000: 49 and 41 against 46 and 37; 4 behind
        // 8000, whose tiles many workers share: 36 against 28.)
        const int64_t units = (int64_t(p.n_tokens) * group + kRows - 1) / kRows * p.kv.n_heads * ((p.shared_len + kUnit - 1) / kUnit);
        if (!many && p.shared_len <= kShortPrefix && units <= int64_t(kPrefixUnits) * 2 * sm_count) {
            j.parts = 2;
            e = launch_split_any(dtype, p, part_o, part_lse, false, true, sm_count, s);
            return e != cudaSuccess ? e : launch_attn_join(dtype, j, s);
        }
        // the prefix, the tails beside it, and both joined
        const int slots = slots_for(0, (p.shared_len + 127) / 128, 1, rows, spare - rows, sm_count);
        if ((e = launch_attn_tc(dtype, p, true, slots, part_o, part_lse, counter, sm_count, s)) != cudaSuccess) return e;
        j.parts = slots > 0 ? slots : 1;
        float* o = part_o + j.parts * rows * dim;
        float* l = part_lse + j.parts * rows;
        ++j.parts;
        e = many ? launch_attn_tc(dtype, p, false, 0, o, l, counter, sm_count, s) : launch_split_any(dtype, p, o, l, true, false, sm_count, s);
        return e != cudaSuccess ? e : launch_attn_join(dtype, j, s);
    }
    if (!many) return launch_split_any(dtype, p, nullptr, nullptr, false, false, sm_count, s);
    int64_t keys = p.kv.table_stride << p.kv.page_shift;
    if (p.window > 0 && p.window + p.sinks + 256 < keys) keys = p.window + p.sinks + 256;
    const int64_t pairs = tc_pairs(p.n_tokens, group, p.kv.n_seqs, false) * p.kv.n_heads;
    const int slots = slots_for(pairs, (keys + 127) / 128, p.kv.n_seqs, rows, spare, sm_count);
    if (slots == 0) return launch_attn_tc(dtype, p, false, 0, nullptr, nullptr, counter, sm_count, s);
    if ((e = launch_attn_tc(dtype, p, false, slots, part_o, part_lse, counter, sm_count, s)) != cudaSuccess) return e;
    j.parts = slots;
    return launch_attn_join(dtype, j, s);
}

}  // namespace qx
