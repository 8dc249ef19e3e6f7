// qx_attn_line.cuh -- what the attention kernels of few rows a sequence share
// (qx_attn.cu, qx_attn_q8.cu): the line of units that their workers cut up, what
// a unit's consumers are told of it, and the join of a tile's parts.
//
// The rows of one sequence and key head (its tokens times the group's query
// heads), ROWS at a time, are a tile; a tile's visible keys are cut into units.
#pragma once

#include "qx_attn.cuh"
#include "qx_layer.cuh"

namespace qx {

constexpr int kUnit = 64;                // keys of a unit
constexpr uint64_t kSplitWaitNs = 10000000000ull;  // (four_again() over millions of keys may be waited for)
constexpr int kSplitWarps = 4;
// A second warpgroup for the producers (in 16 bits one warp, and the other three
// only give up registers; over codes all four work): 128 registers a thread at
// launch, of which the consumers, who hold a tile's queries and output, take most.
constexpr int kSplitThreads = 2 * 32 * kSplitWarps;
constexpr int kConsumerRegs = 176, kProducerRegs = 80;
static_assert(kConsumerRegs + kProducerRegs <= 2 * 128, "registers the CTA was launched with");
constexpr int kRows = 16;                // rows of a tile, in 16 bits
// Scratch: arrival counters (one a worker, and 64 words for the tensor-core
// kernel's; zero between calls), then two partial tiles a worker: o [rows][DIM], then m and l of the rows.
constexpr int kMaxWorkers = 512;
constexpr size_t kCounterBytes = QX_ATTN_COUNTER_BYTES;
static_assert(kCounterBytes == (kMaxWorkers + 64) * 4, "the counters");
template <int DIM, int ROWS = kRows>
__host__ __device__ constexpr int partial_floats() { return ROWS * DIM + 2 * ROWS; }

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
    int row_tiles;         // tiles of ROWS rows for each key head
    int sink_units, units; // of one tile
    int pos0;              // position of the first token
    int lo, end, sinks;
};
constexpr int kMostKeys = INT32_MAX - 4 * kUnit;  // of a sequence: key numbers stay in 32 bits
template <int ROWS>
__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, int b, int group, bool report) {
    SeqWork w;
    if (b == p.kv.n_seqs) {  // every token against the shared prefix (their positions are looked up)
        const int total = p.kv.q_start[b];
        const int64_t room = p.kv.table_stride << p.kv.page_shift, most = room < kMostKeys ? room : kMostKeys;
        w.t0 = w.pos0 = w.lo = w.sinks = w.sink_units = 0;
        w.tokens = total < p.n_tokens ? total : p.n_tokens;
        w.end = int(p.shared_len < most ? p.shared_len : most);
        w.units = (w.end + kUnit - 1) / kUnit;
        w.row_tiles = (w.tokens * group + ROWS - 1) / ROWS;
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
    w.row_tiles = (w.tokens * group + ROWS - 1) / ROWS;
    return w;
}

// A place on the line of units: tile (sequence b, row tile rt, key head hk),
// whose units are [begin, begin + w.units) of the line.
struct Cursor {
    int64_t begin;
    int b, rt, hk;
    SeqWork w;
};
template <int ROWS>
__device__ __forceinline__ void next_tile(const AttnParams& p, Cursor& c, int group, int seqs) {
    c.begin += c.w.units;
    if (++c.hk < p.kv.n_heads) return;
    c.hk = 0;
    if (++c.rt < c.w.row_tiles) return;
    c.rt = 0;
    do {
        if (++c.b >= seqs) return;
        c.w = seq_work<ROWS>(p, c.b, group, false);
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

// A worker's share of the line: units [first, last).
struct Line {
    int64_t share, extra;  // the first `extra` workers have one unit more than the others
    int64_t first, last;
    __device__ __forceinline__ int64_t begin_of(int64_t w) const { return w * share + (w < extra ? w : extra); }
    __device__ __forceinline__ int64_t worker_of(int64_t u) const {
        return u < extra * (share + 1) ? quot(u, share + 1) : extra + quot(u - extra * (share + 1), share);
    }
    // What the consumers are told of the tile at c, and of its unit u.
    template <int ROWS>
    __device__ __forceinline__ void describe_tile(const AttnParams& p, const Cursor& c, int group, UnitInfo& x) const {
        x.t0 = c.w.t0;
        x.r0 = ROWS * c.rt;
        x.rows = c.w.tokens * group - x.r0;
        x.hk = c.hk;
        x.pos0 = c.w.pos0;
        // only a worker's first and last tile may be shared; its part of a
        // tile lies in its first slot, or in its second where another tile's
        // end came first
        const int64_t begin = c.begin, end = c.begin + c.w.units;
        const int64_t wf = begin < first ? worker_of(begin) : blockIdx.x, wl = end > last ? worker_of(end - 1) : blockIdx.x;
        x.wf = int(wf);
        x.parts = int(wl - wf);
        x.part = 2 * int(wf) + (begin_of(wf) < begin ? 1 : 0);
    }
    __device__ __forceinline__ void describe_unit(const AttnParams& p, const Cursor& c, int u, UnitInfo& x) const {
        x.j0 = unit_keys(c.w, u, x.lo, x.hi);
        const int64_t end = c.begin + c.w.units, here = c.begin + u;
        x.flags = (u < c.w.sink_units ? kSink : 0) | (here == first || u == 0 ? kOpens : 0) | (here + 1 == last || here + 1 == end ? kCloses : 0) |
                  (c.b == p.kv.n_seqs ? kPrefix : 0);
    }
    template <int ROWS>
    __device__ __forceinline__ void describe(const AttnParams& p, const Cursor& c, int u, int group, UnitInfo& x) const {
        describe_unit(p, c, u, x);
        describe_tile<ROWS>(p, c, group, x);
    }
};
// The line's length, and where this worker's share of it begins (for the whole
// CTA, to `start`; scan: a word a warp).  B: sequences.  LEAST: units of a worker at
// least, where there are so many.  False: it has none.
template <int ROWS, int LEAST = 2>
__device__ __forceinline__ bool open_line(const AttnParams& p, int B, int group, int64_t* scan, Cursor* start, Line& line) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t mine = 0;
    const int per = (B + kSplitThreads - 1) / kSplitThreads, b0 = threadIdx.x * per;
    SeqWork own;  // of the thread's last sequence (its only one, for up to 256 sequences)
    for (int b = b0; b < b0 + per && b < B; ++b) {
        own = seq_work<ROWS>(p, b, group, blockIdx.x == 0);
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
    const int64_t most = (U + LEAST - 1) / LEAST, N = gridDim.x < most ? gridDim.x : most;
    if (blockIdx.x >= N) return false;
    line.share = quot(U, N);
    line.extra = U - line.share * N;
    const int64_t first = line.first = line.begin_of(blockIdx.x);
    line.last = line.begin_of(blockIdx.x + 1);
    int64_t at = before + incl - mine;
    if (first >= at && first < at + mine) {
        for (int b = b0; b < b0 + per && b < B; ++b) {
            if (per > 1) own = seq_work<ROWS>(p, b, group, false);
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
    return true;
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
// (M, L) and (m, l) become one maximum and one sum.  Sums over scores that are
// no numbers have a maximum of -inf, and stay what they are.  FAR: the maxima
// count more than the scores, so a lower one's sum may weigh as much.
template <bool FAR>
__device__ __forceinline__ void join_sums(float& M, float& L, float m, float l) {
    const float mn = fmaxf(M, m), base = mn == -INFINITY ? 0.0f : mn;
    if constexpr (FAR) L = twice(L, exp2_approx(0.5f * (M - base))) + twice(l, exp2_approx(0.5f * (m - base)));
    else L = L * exp2_approx(M - base) + l * exp2_approx(m - base);
    M = mn;
}

// The parts of a tile that several workers shared, joined by the consumers of
// the last of them to arrive.  The rows of which write_four says so, as bits.
template <typename T, int DIM, int ROWS = kRows, bool FAR = false>
__device__ __forceinline__ uint32_t join_parts(const SplitParams& pp, const UnitInfo& tile, float* buf, bool look) {
    float* partials = reinterpret_cast<float*>(static_cast<uint8_t*>(pp.a.scratch) + kCounterBytes);
    float* buf_ml = buf + kSplitWarps * 8 * DIM;
    const int live = tile.rows < ROWS ? tile.rows : ROWS, parts = tile.parts + 1;
    const float* const begin = partials + int64_t(tile.part) * partial_floats<DIM, ROWS>();
    const float* const rest = partials + int64_t(2 * (tile.wf + 1)) * partial_floats<DIM, ROWS>();
    constexpr int64_t kStep = 2 * partial_floats<DIM, ROWS>();
    const auto src = [&](int i) -> const float* { return i == 0 ? begin : rest + (i - 1) * kStep; };
    // eight threads a row find its maximum and sum, and leave each part's
    // weight in the buffer
    float* weight = buf;  // [ROWS][parts], where that fits
    const bool fits = ROWS * parts <= kSplitWarps * 8 * DIM;
    const int i8 = threadIdx.x & 7;
#pragma unroll
    for (int r0 = 0; r0 < ROWS; r0 += 4 * kSplitWarps) {
        const int r8 = r0 + (threadIdx.x >> 3);
        float M = -INFINITY, L = 0.0f;
        if (r8 < live) {
#pragma unroll 4
            for (int i = i8; i < parts; i += 8) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(src(i) + ROWS * DIM + 2 * r8));
                join_sums<FAR>(M, L, ml.x, ml.y);
                if (fits) weight[r8 * parts + i] = ml.x;
            }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, M, o), ol = __shfl_xor_sync(0xffffffffu, L, o);
            join_sums<FAR>(M, L, om, ol);
        }
        if (r8 < live) {
            if (fits)
                for (int i = i8; i < parts; i += 8) {
                    const float m = weight[r8 * parts + i];
                    weight[r8 * parts + i] = m == -INFINITY ? 0.0f : exp2_approx(m - M);
                }
            if (i8 == 0) *reinterpret_cast<float2*>(buf_ml + 2 * r8) = make_float2(M, L);
        }
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
                    const float m = __ldcg(src(w0 + y) + ROWS * DIM + 2 * r);
                    c = m == -INFINITY ? 0.0f : exp2_approx(m - ml.x);
                }
                acc.x += c * v[y].x, acc.y += c * v[y].y, acc.z += c * v[y].z, acc.w += c * v[y].w;
            }
        }
        if (write_four<T, DIM>(pp, tile, r, d, ml.x, ml.y, acc, look)) odd |= 1u << r;
    }
    return odd;
}

}  // namespace qx
