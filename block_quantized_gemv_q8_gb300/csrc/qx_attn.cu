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
// In a CTA each of four warps takes 16 of a unit's keys with an online
// softmax of its own: it copies its keys and values to its own ring in shared
// memory (cp.async, whole 16-byte chunks, chunk c of row r at c ^ (r % 8) so
// that ldmatrix meets no bank conflict) and needs no other warp until the
// tile ends.  Products: mma.sync m16n8k16, whose 16 rows the group fills at
// most partly; the tensor pipe is not what bounds this kernel.

constexpr int kUnit = 64;                // keys of a unit
constexpr int kSplitWarps = 4;
constexpr int kSplitThreads = 32 * kSplitWarps;
constexpr int kRows = 16;                // rows of a tile
constexpr int kRingBytes = 96 * 1024;    // of one CTA; two CTAs fit on an SM

template <int DIM>
struct SplitGeom {
    static constexpr int kRowBytes = 2 * DIM;
    static constexpr int kStageBytes = 2 * 16 * kRowBytes;  // one warp's keys and values
    static constexpr int kStages = kRingBytes / (kSplitWarps * kStageBytes);
    static constexpr int kPad = DIM + 4;  // floats of a row in the joining buffer: 8 rows of each warp, then their m and l
    static constexpr int kJoin = (kSplitWarps * 8 * (kPad + 2)) * 4;
    static constexpr size_t kSmem = kRingBytes + kJoin;
    static_assert(2 * (kSmem + 1200) <= 228 * 1024, "two CTAs an SM");
};

// Scratch: arrival counters (one a worker, and 64 words for the tensor-core
// kernel's; zero between calls), then two partial tiles a worker: o [16][DIM], then m and l of the 16 rows.
constexpr int kMaxWorkers = 512;
constexpr size_t kCounterBytes = (kMaxWorkers + 64) * 4;
template <int DIM>
__host__ __device__ constexpr int partial_floats() { return kRows * DIM + 2 * kRows; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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
    int64_t pos0;          // position of the first token
    int64_t lo, end, sinks;
};
__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, int b, int group, bool report) {
    SeqWork w;
    w.t0 = p.kv.q_start[b];
    w.tokens = p.kv.q_start[b + 1] - w.t0;
    if (w.tokens < 0 || w.t0 < 0 || w.t0 + w.tokens > p.n_tokens) w.tokens = 0;  // not an ascending list of this call's tokens
    int64_t kv = p.kv.kv_len[b];
    w.pos0 = kv - w.tokens;
    const int64_t most = p.kv.table_stride << p.kv.page_shift;
    if (kv > most) {
        if (report) atomicOr(p.kv.err, kErrRange);
        kv = most;
    }
    w.end = kv < 0 ? 0 : kv;
    w.lo = p.window > 0 && w.pos0 + 1 > p.window ? w.pos0 + 1 - p.window : 0;
    if (w.lo < p.shared_len) w.lo = p.shared_len;
    w.sinks = p.sinks < w.lo ? p.sinks : w.lo;
    if (p.shared_len > 0) w.sinks = 0;
    if (w.sinks > w.end) w.sinks = w.end;
    w.sink_units = int((w.sinks + kUnit - 1) / kUnit);
    const int64_t win = (w.end + kUnit - 1) / kUnit - w.lo / kUnit;
    w.units = w.sink_units + (win > 0 ? int(win) : 0);
    if (w.units < 1) w.units = 1;
    w.row_tiles = (w.tokens * group + kRows - 1) / kRows;
    return w;
}

// A place on the line of units: unit u of tile (sequence b, row tile rt, key
// head hk), where the tile's units are [begin, begin + w.units) of the line.
struct Cursor {
    int b, rt, hk;
    int64_t begin;
    SeqWork w;
};
__device__ __forceinline__ void next_tile(const AttnParams& p, Cursor& c, int group) {
    c.begin += c.w.units;
    if (++c.hk < p.kv.n_heads) return;
    c.hk = 0;
    if (++c.rt < c.w.row_tiles) return;
    c.rt = 0;
    do {
        if (++c.b >= p.kv.n_seqs) return;
        c.w = seq_work(p, c.b, group, false);
    } while (c.w.row_tiles == 0);
}
// The first key of unit u of a tile, and the keys [lo, hi) of it that any row sees.
__device__ __forceinline__ int64_t unit_keys(const SeqWork& w, int u, int64_t& lo, int64_t& hi) {
    if (u < w.sink_units) {
        lo = 0, hi = w.sinks;
        return int64_t(u) * kUnit;
    }
    lo = w.lo, hi = w.end;
    return (w.lo / kUnit + (u - w.sink_units)) * kUnit;
}

struct SplitParams : AttnParams {
    float* part_o;    // not null: the rows are a part to be joined (o / l, base-2 log of the sum)
    float* part_lse;
    int beside;       // 1: launched beside the kernel before it, which belongs to the same call
};

// Quotients of non-negative numbers, in 32 bits where they fit (nearly always).
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return int64_t(uint32_t(a) / uint32_t(b));
    return a / b;
}

template <typename T, int DIM>
__global__ void __launch_bounds__(kSplitThreads, 2) attn_split_kernel(const __grid_constant__ SplitParams p) {
    using G = SplitGeom<DIM>;
    constexpr int KS = DIM / 16;  // 16-wide steps along a head
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan[kSplitWarps];
    __shared__ Cursor start;
    __shared__ int last_flag;
    // Beside a kernel that works on the same call's prefix: that one has
    // waited for the work before it, and this one reads nothing of its.
    if (!p.beside) pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.n_q_heads / p.kv.n_heads;
    const int B = p.kv.n_seqs;

    // ---- the line's length, and where this worker's share begins
    int64_t mine = 0;
    const int per = (B + kSplitThreads - 1) / kSplitThreads, b0 = threadIdx.x * per;
    SeqWork own;  // of the thread's last sequence (its only one, for up to 128 sequences)
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
    for (int w = 0; w < kSplitWarps; ++w) {
        if (w < warp) before += scan[w];
        U += scan[w];
    }
    const int64_t N = gridDim.x < U ? gridDim.x : U;
    if (blockIdx.x >= N) {
        if (p.beside) pdl_wait_prior_grid();
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
                start.b = b;
                start.w = own;
                start.begin = at + tile * own.units;
                start.rt = int(quot(tile, p.kv.n_heads));
                start.hk = int(tile - int64_t(start.rt) * p.kv.n_heads);
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    Cursor ld = start;   // of the unit being fetched
    Cursor cur = start;  // of the unit being computed

    // ---- this warp's ring
    uint8_t* ring = smem + warp * (G::kStages * G::kStageBytes);
    const uint32_t ring_a = smem_addr(ring);
    int64_t fu = first;  // the next unit to fetch
    // Sixteen keys of unit u from key 16 * warp of it on: their page, or -1
    // where no row sees any of them.
    const auto page_for = [&](const Cursor& c, int64_t u) -> int {
        int64_t lo, hi;
        const int64_t j0 = unit_keys(c.w, int(u - c.begin), lo, hi) + 16 * warp;
        if (j0 + 16 <= lo || j0 >= hi) return -1;
        return page_of(p.kv, c.b, j0);
    };
    int page = page_for(ld, fu);
    const auto fetch = [&](int stage) {
        if (fu < last) {
            int64_t lo, hi;
            const int64_t j0 = unit_keys(ld.w, int(fu - ld.begin), lo, hi) + 16 * warp;
            const int64_t base = page < 0 ? 0 : slot_offset(p.kv, page, ld.hk, j0);
            const T* ks = reinterpret_cast<const T*>(p.kv.k) + base;
            const T* vs = reinterpret_cast<const T*>(p.kv.v) + base;
            constexpr int CH = G::kRowBytes / 16;  // chunks of a row
            const uint32_t dst = ring_a + stage * G::kStageBytes;
#pragma unroll
            for (int i = 0; i < 16 * CH / 32; ++i) {
                const int r = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH;
                const bool live = page >= 0 && j0 + r >= lo && j0 + r < hi;
                const int64_t off = live ? r * p.kv.slot_stride + c * 8 : 0;
                const uint32_t d = dst + r * G::kRowBytes + ((c ^ (r & 7)) << 4);
                cp_async16(d, ks + off, live);
                cp_async16(d + 16 * G::kRowBytes, vs + off, live);
            }
            if (++fu < last) {
                if (fu == ld.begin + ld.w.units) next_tile(p, ld, group);
                page = page_for(ld, fu);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < G::kStages - 1; ++s) fetch(s);

    // ---- units
    uint32_t qf[KS][4];
    float o[DIM / 8][4], m[2], l[2];
    int64_t rpos[2];  // positions of this lane's two rows (-1: none)
    // A tile's rows: 16 rt + lane / 4 and eight further.
    const auto open_tile = [&](const Cursor& c) {
        const int rows = c.w.tokens * group;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = kRows * c.rt + (lane >> 2) + 8 * i;
            const bool live = r < rows;
            const int tok = live ? r / group : 0, g = live ? r - tok * group : 0;
            rpos[i] = live ? c.w.pos0 + tok : -1;
            const T* q = static_cast<const T*>(p.q) + int64_t(c.w.t0 + tok) * p.q_stride + int64_t(c.hk * group + g) * DIM + 2 * (lane & 3);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][i] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * k) : 0u;
                qf[k][i + 2] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8) : 0u;
            }
        }
    };
    open_tile(cur);
    float* partials = reinterpret_cast<float*>(static_cast<uint8_t*>(p.scratch) + kCounterBytes);
    unsigned* counters = static_cast<unsigned*>(p.scratch);
    float* buf = reinterpret_cast<float*>(smem + kRingBytes);  // [4 warps][8 rows][kPad], then m and l of each
    float* buf_ml = buf + kSplitWarps * 8 * G::kPad;
    int stage = 0;
    for (int64_t u = first; u < last; ++u) {
        if (u == first || u == cur.begin) {
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.0f;
#pragma unroll
            for (int d = 0; d < DIM / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.0f;
        }
        cp_async_wait<G::kStages - 2>();
        __syncwarp();
        int64_t lo, hi;
        const int64_t j0 = unit_keys(cur.w, int(u - cur.begin), lo, hi) + 16 * warp;
        if (j0 + 16 > lo && j0 < hi) {
            const uint32_t ka = ring_a + stage * G::kStageBytes, va = ka + 16 * G::kRowBytes;
            float s[2][4] = {};
            {
                // matrices: keys 0-7 and 8-15 by d 0-7 and 8-15 of each step
                const int r = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t b[4];
                    ldmatrix4(ka + r * G::kRowBytes + (((2 * k + half) ^ (r & 7)) << 4), b);
                    mma16816<T>(s[0], qf[k], b[0], b[1]);
                    mma16816<T>(s[1], qf[k], b[2], b[3]);
                }
            }
            // This lane's keys relative to the sixteen's first: 2 (lane % 4) + {0, 1, 8, 9}.
            const bool sink_unit = u - cur.begin < cur.w.sink_units;
            const int first_key = lo > j0 ? int(lo - j0) : 0, end_key = hi < j0 + 16 ? int(hi - j0) : 16;
            float mx[2] = {m[0], m[1]};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t back = rpos[i] - j0;  // the row's position among them
                const int end = back < end_key - 1 ? int(back < -1 ? -1 : back) + 1 : end_key;
                int from = first_key, sink_end = 0;
                if (p.window > 0 && !sink_unit) {
                    const int64_t f = back - p.window + 1;
                    from = f > first_key ? (f < 16 ? int(f) : 16) : first_key;
                    const int64_t e = p.sinks - j0;
                    sink_end = e < 0 ? 0 : e < 16 ? int(e) : 16;
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 8 * n + 2 * (lane & 3) + e;
                        const bool see = j < end && (j >= from || (j >= first_key && j < sink_end));
                        s[n][2 * i + e] = see ? s[n][2 * i + e] * p.scale_log2 : -INFINITY;
                        mx[i] = fmaxf(mx[i], s[n][2 * i + e]);
                    }
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
            const float base[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = exp2_approx(s[n][e] - base[e >> 1]);
                    l[e >> 1] += s[n][e];
                }
            const uint32_t pf[4] = {pack2<T>(s[0][0], s[0][1]), pack2<T>(s[0][2], s[0][3]), pack2<T>(s[1][0], s[1][1]),
                                    pack2<T>(s[1][2], s[1][3])};
            {
                const int r = lane & 15, half = lane >> 4;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t b[4];
                    ldmatrix4_t(va + r * G::kRowBytes + (((2 * k + half) ^ (r & 7)) << 4), b);
                    mma16816<T>(o[2 * k], pf, b[0], b[1]);
                    mma16816<T>(o[2 * k + 1], pf, b[2], b[3]);
                }
            }
        }
        __syncwarp();  // the stage is free again
        {
            int fs = stage + G::kStages - 1;
            if (fs >= G::kStages) fs -= G::kStages;
            fetch(fs);
        }
        if (++stage == G::kStages) stage = 0;

        const int64_t t_end = cur.begin + cur.w.units;
        if (u + 1 != last && u + 1 != t_end) continue;
        // ---- the tile ends here (for this worker).  The next one's queries
        // are on their way while its warps are joined, eight rows at a time:
        // every warp leaves its (m, l, o), and every thread then joins some
        // elements.
        const Cursor done = cur;
        if (u + 1 < last) {
            next_tile(p, cur, group);
            open_tile(cur);
        }
        const int rows = done.w.tokens * group - kRows * done.rt;  // of this tile (16 at most count)
        const int64_t wf = worker_of(done.begin), wl = worker_of(t_end - 1);  // the first and last worker of the tile
        // A worker's part of a tile lies in its first slot, or in its second
        // where another tile's end came first.
        const auto slot_of = [&](int64_t w) -> float* { return partials + 2 * w * partial_floats<DIM>(); };
        float* const wf_slot = slot_of(wf) + (begin_of(wf) < done.begin ? partial_floats<DIM>() : 0);
        const auto finish = [&](int r, int d, float M, float L, float4 v) {
            const int rr = kRows * done.rt + r;
            const int64_t row = int64_t(done.w.t0 + rr / group) * p.n_q_heads + done.hk * group + rr % group;
            const float inv = L > 0.0f ? 1.0f / L : 0.0f;
            v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
            if (p.part_o) {
                *reinterpret_cast<float4*>(p.part_o + row * DIM + d) = v;
                if (d == 0) p.part_lse[row] = L > 0.0f ? M + log2f(L) : -INFINITY;
                return;
            }
            if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * DIM + d) = v;
            else *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * DIM + d) = make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
            if (p.lse && d == 0) p.lse[row] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (8 * i >= rows) break;
            const int live = rows - 8 * i < 8 ? rows - 8 * i : 8;
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (i > 0) __syncthreads();  // the first eight are read
            if ((lane >> 2) < live) {
                float* row = buf + (8 * warp + (lane >> 2)) * G::kPad + 2 * (lane & 3);
#pragma unroll
                for (int d = 0; d < DIM / 8; ++d) *reinterpret_cast<float2*>(row + 8 * d) = make_float2(o[d][2 * i], o[d][2 * i + 1]);
                if ((lane & 3) == 0) *reinterpret_cast<float2*>(buf_ml + 2 * (8 * warp + (lane >> 2))) = make_float2(m[i], l[i]);
            }
            __syncthreads();
            for (int x = threadIdx.x; x < live * (DIM / 4); x += kSplitThreads) {
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
                    const float4 v = *reinterpret_cast<const float4*>(buf + (8 * w + r) * G::kPad + d);
                    L += a * ml[w].y;
                    acc.x += a * v.x, acc.y += a * v.y, acc.z += a * v.z, acc.w += a * v.w;
                }
                if (wf == wl) {
                    finish(8 * i + r, d, M, L, acc);
                } else {
                    float* to = (blockIdx.x == wf ? wf_slot : slot_of(blockIdx.x)) + (8 * i + r) * DIM;
                    *reinterpret_cast<float4*>(to + d) = acc;
                    if (d == 0) *reinterpret_cast<float2*>(to - (8 * i + r) * DIM + kRows * DIM + 2 * (8 * i + r)) = make_float2(M, L);
                }
            }
        }
        if (wf != wl) {
            // ---- this worker's part is written; the last to arrive joins all
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                const unsigned n = atomicAdd(&counters[wf], 1u);
                last_flag = n == unsigned(wl - wf);
                if (last_flag) counters[wf] = 0;  // for the next call
            }
            __syncthreads();
            if (last_flag) {
                __threadfence();
                const int live = rows < kRows ? rows : kRows, parts = int(wl - wf);  // beyond the first
                const float* rest = slot_of(wf + 1);
                constexpr int64_t kStep = 2 * partial_floats<DIM>();
                for (int x = threadIdx.x; x < live * (DIM / 4); x += kSplitThreads) {
                    const int r = x / (DIM / 4), d = x % (DIM / 4) * 4;
                    const int at_ml = kRows * DIM + 2 * r, at_o = r * DIM + d;
                    float2 ml = __ldcg(reinterpret_cast<const float2*>(wf_slot + at_ml));
                    float M = ml.x, L = ml.y;
                    float4 acc = __ldcg(reinterpret_cast<const float4*>(wf_slot + at_o));
                    // eight parts' loads in flight at a time
                    for (int w0 = 0; w0 < parts; w0 += 8) {
                        float2 e[8];
                        float4 v[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float* f = rest + (w0 + y < parts ? w0 + y : parts - 1) * kStep;
                            e[y] = __ldcg(reinterpret_cast<const float2*>(f + at_ml));
                            v[y] = __ldcg(reinterpret_cast<const float4*>(f + at_o));
                        }
                        float mn = M;
#pragma unroll
                        for (int y = 0; y < 8; ++y) mn = fmaxf(mn, e[y].x);
                        const float a = M == -INFINITY ? 0.0f : exp2_approx(M - mn);
                        M = mn;
                        L *= a, acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a;
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float c = w0 + y < parts && e[y].x != -INFINITY ? exp2_approx(e[y].x - mn) : 0.0f;
                            L += c * e[y].y;
                            acc.x += c * v[y].x, acc.y += c * v[y].y, acc.z += c * v[y].z, acc.w += c * v[y].w;
                        }
                    }
                    finish(r, d, M, L, acc);
                }
            }
        } else {
            __syncthreads();  // the buffer is read
        }
    }
    cp_async_wait<0>();
    if (p.beside) pdl_wait_prior_grid();  // complete only after that kernel, too
}

template <typename T, int DIM>
cudaError_t launch_split(const SplitParams& p, int sm_count, cudaStream_t s) {
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

cudaError_t launch_split_any(int dtype, const AttnParams& a, float* part_o, float* part_lse, bool beside, int sm_count,
                             cudaStream_t s) {
    SplitParams p;
    static_cast<AttnParams&>(p) = a;
    p.part_o = part_o;
    p.part_lse = part_lse;
    p.beside = beside ? 1 : 0;
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
// Rows of parts that the scratch holds: enough to split the keys of few rows
// over the GPU, and two parts of any call whose shared prefix is taken apart.
constexpr int64_t kPartRows = 65536, kMaxSharedRows = 131072;
int64_t part_rows(int64_t rows) {
    const int64_t two = 2 * (rows < kMaxSharedRows ? rows : kMaxSharedRows);
    return two > kPartRows ? (two + 63) / 64 * 64 : kPartRows;  // 256-byte multiples
}
constexpr int kMaxSplits = 31;  // of one launch: with the tails' part a row has at most 32

// CTAs that share a tile pair's keys: as many as give every SM one.
int splits_for(int64_t ctas, int64_t rows, int64_t spare_rows, int sm_count) {
    int64_t n = ctas > 0 ? sm_count / ctas : 1;
    if (n > kMaxSplits) n = kMaxSplits;
    if (n * rows > spare_rows) n = spare_rows / rows;
    return n < 1 ? 1 : int(n);
}

}  // namespace

size_t attn_scratch_bytes(int64_t n_tokens, int n_q_heads, int, int head_dim, int) {
    const int64_t rows = n_tokens * n_q_heads;
    return kSplitScratch + (head_dim == 64 || head_dim == 128 ? size_t(part_rows(rows)) * (head_dim + 1) * 4 : 0);
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
    int64_t spare = part_rows(rows);
    if (p.shared_len > 0) {
        spare -= rows;  // the tails' part
        j.parts = splits_for(tc_pairs(p.n_tokens, group, p.kv.n_seqs, true) * p.kv.n_heads, rows, spare, sm_count);
        if ((e = launch_attn_tc(dtype, p, true, j.parts, part_o, part_lse, counter, sm_count, s)) != cudaSuccess) return e;
        float* o = part_o + j.parts * rows * dim;
        float* l = part_lse + j.parts * rows;
        ++j.parts;
        e = many ? launch_attn_tc(dtype, p, false, 1, o, l, counter, sm_count, s) : launch_split_any(dtype, p, o, l, true, sm_count, s);
        return e != cudaSuccess ? e : launch_attn_join(dtype, j, s);
    }
    if (!many) return launch_split_any(dtype, p, nullptr, nullptr, false, sm_count, s);
    const int n = splits_for(tc_pairs(p.n_tokens, group, p.kv.n_seqs, false) * p.kv.n_heads, rows, spare, sm_count);
    if (n == 1) return launch_attn_tc(dtype, p, false, 1, nullptr, nullptr, counter, sm_count, s);
    if ((e = launch_attn_tc(dtype, p, false, n, part_o, part_lse, counter, sm_count, s)) != cudaSuccess) return e;
    j.parts = n;
    return launch_attn_join(dtype, j, s);
}

}  // namespace qx
