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
    static constexpr int kPad = DIM + 4;                     // floats of a row in the joining buffer
    static constexpr int kJoin = 2 * kRows * (kPad + 2) * 4;
    static constexpr size_t kSmem = kRingBytes + kJoin;
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
};

template <typename T, int DIM>
__global__ void __launch_bounds__(kSplitThreads, 2) attn_split_kernel(const __grid_constant__ SplitParams p) {
    using G = SplitGeom<DIM>;
    constexpr int KS = DIM / 16;  // 16-wide steps along a head
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan[kSplitWarps];
    __shared__ int64_t found_begin;
    __shared__ int found_b, last_flag;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.n_q_heads / p.kv.n_heads;
    const int B = p.kv.n_seqs;

    // ---- the line's length, and where this worker's share begins
    int64_t mine = 0;
    const int per = (B + kSplitThreads - 1) / kSplitThreads, b0 = threadIdx.x * per;
    for (int b = b0; b < b0 + per && b < B; ++b) {
        const SeqWork w = seq_work(p, b, group, blockIdx.x == 0);
        mine += int64_t(w.row_tiles) * p.kv.n_heads * w.units;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    if (threadIdx.x == 0) found_b = -1;
    __syncthreads();
    int64_t U = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kSplitWarps; ++w) {
        if (w < warp) before += scan[w];
        U += scan[w];
    }
    const int64_t N = gridDim.x < U ? gridDim.x : U;
    if (blockIdx.x >= N) return;
    const int64_t first = blockIdx.x * U / N, last = (blockIdx.x + 1) * U / N;  // this worker's units
    int64_t at = before + incl - mine;
    if (first >= at && first < at + mine) {
        for (int b = b0; b < b0 + per && b < B; ++b) {
            const SeqWork w = seq_work(p, b, group, false);
            const int64_t n = int64_t(w.row_tiles) * p.kv.n_heads * w.units;
            if (first < at + n) {
                found_b = b;
                found_begin = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    Cursor ld;  // of the unit being fetched
    ld.b = found_b;
    ld.w = seq_work(p, ld.b, group, false);
    {
        const int64_t tile = (first - found_begin) / ld.w.units;
        ld.begin = found_begin + tile * ld.w.units;
        ld.rt = int(tile / p.kv.n_heads);
        ld.hk = int(tile % p.kv.n_heads);
    }
    Cursor cur = ld;  // of the unit being computed

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
    float* partials = reinterpret_cast<float*>(static_cast<uint8_t*>(p.scratch) + kCounterBytes);
    unsigned* counters = static_cast<unsigned*>(p.scratch);
    int stage = 0;
    for (int64_t u = first; u < last; ++u) {
        const bool opens = u == first || u == cur.begin;
        if (opens) {
            // the tile's rows: 16 rt + lane / 4 and eight further
            const int rows = cur.w.tokens * group;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = kRows * cur.rt + (lane >> 2) + 8 * i;
                const bool live = r < rows;
                const int tok = live ? r / group : 0, g = live ? r % group : 0;
                rpos[i] = live ? cur.w.pos0 + tok : -1;
                const T* q = static_cast<const T*>(p.q) + int64_t(cur.w.t0 + tok) * p.q_stride +
                             int64_t(cur.hk * group + g) * DIM + 2 * (lane & 3);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    qf[k][i] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * k) : 0u;
                    qf[k][i + 2] = live ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8) : 0u;
                }
                m[i] = -INFINITY;
                l[i] = 0.0f;
            }
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
            const bool sink_unit = u - cur.begin < cur.w.sink_units;
            float mx[2] = {m[0], m[1]};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t j = j0 + 8 * n + 2 * (lane & 3) + (e & 1);
                    const int64_t pos = rpos[e >> 1];
                    const bool see = j >= lo && j < hi && j <= pos &&
                                     (sink_unit || p.window == 0 || j > pos - p.window || j < p.sinks);
                    s[n][e] = see ? s[n][e] * p.scale_log2 : -INFINITY;
                    mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
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

        const bool closes = u + 1 == last || u + 1 == cur.begin + cur.w.units;
        if (!closes) continue;
        // ---- the tile ends here (for this worker): join the four warps
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        float* buf = reinterpret_cast<float*>(smem + kRingBytes);
        const auto give = [&](float* to) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = (lane >> 2) + 8 * i;
                float* row = to + r * G::kPad + 2 * (lane & 3);
#pragma unroll
                for (int d = 0; d < DIM / 8; ++d)
                    *reinterpret_cast<float2*>(row + 8 * d) = make_float2(o[d][2 * i], o[d][2 * i + 1]);
                if ((lane & 3) == 0) {
                    to[kRows * G::kPad + r] = m[i];
                    to[kRows * G::kPad + kRows + r] = l[i];
                }
            }
        };
        const auto take = [&](const float* from) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = (lane >> 2) + 8 * i;
                const float om = from[kRows * G::kPad + r], ol = from[kRows * G::kPad + kRows + r];
                const float M = fmaxf(m[i], om);
                const float a = m[i] == -INFINITY ? 0.0f : exp2_approx(m[i] - M), c = om == -INFINITY ? 0.0f : exp2_approx(om - M);
                m[i] = M;
                l[i] = l[i] * a + ol * c;
                const float* row = from + r * G::kPad + 2 * (lane & 3);
#pragma unroll
                for (int d = 0; d < DIM / 8; ++d) {
                    const float2 v = *reinterpret_cast<const float2*>(row + 8 * d);
                    o[d][2 * i] = o[d][2 * i] * a + v.x * c;
                    o[d][2 * i + 1] = o[d][2 * i + 1] * a + v.y * c;
                }
            }
        };
        float* half0 = buf;
        float* half1 = buf + kRows * (G::kPad + 2);
        __syncthreads();
        if (warp >= 2) give(warp == 2 ? half0 : half1);
        __syncthreads();
        if (warp < 2) take(warp == 0 ? half0 : half1);
        __syncthreads();
        if (warp == 1) give(half0);
        __syncthreads();
        if (warp == 0) take(half0);
        // ---- write the tile, or this worker's part of it
        const int rows = cur.w.tokens * group - kRows * cur.rt;  // of this tile (16 at most count)
        const int64_t t_end = cur.begin + cur.w.units;
        const int64_t wf = ((cur.begin + 1) * N - 1) / U, wl = (t_end * N - 1) / U;  // the first and last worker of the tile
        const auto finish = [&](int r, int d, float M, float L, float x, float y) {
            const int rr = kRows * cur.rt + r;
            const int64_t row = int64_t(cur.w.t0 + rr / group) * p.n_q_heads + cur.hk * group + rr % group;
            const float inv = L > 0.0f ? 1.0f / L : 0.0f;
            if (p.part_o) {
                *reinterpret_cast<float2*>(p.part_o + row * DIM + d) = make_float2(x * inv, y * inv);
                if (d == 0) p.part_lse[row] = L > 0.0f ? M + log2f(L) : -INFINITY;
                return;
            }
            if (p.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + row * DIM + d) = make_float2(x * inv, y * inv);
            else *reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + row * DIM + d) = pack2<T>(x * inv, y * inv);
            if (p.lse && d == 0) p.lse[row] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
        };
        if (wf == wl) {
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = (lane >> 2) + 8 * i;
                    if (r < rows)
#pragma unroll
                        for (int d = 0; d < DIM / 8; ++d)
                            finish(r, 8 * d + 2 * (lane & 3), m[i], l[i], o[d][2 * i], o[d][2 * i + 1]);
                }
            }
        } else {
            const auto slot_of = [&](int64_t w) { return partials + (2 * w + (w == wf && wf * U / N < cur.begin ? 1 : 0)) * partial_floats<DIM>(); };
            if (warp == 0) {
                float* to = slot_of(blockIdx.x);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = (lane >> 2) + 8 * i;
                    if (r < rows) {
#pragma unroll
                        for (int d = 0; d < DIM / 8; ++d)
                            *reinterpret_cast<float2*>(to + r * DIM + 8 * d + 2 * (lane & 3)) = make_float2(o[d][2 * i], o[d][2 * i + 1]);
                        if ((lane & 3) == 0) to[kRows * DIM + r] = m[i], to[kRows * DIM + kRows + r] = l[i];
                    }
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    const unsigned n = atomicAdd(&counters[wf], 1u);
                    last_flag = n == unsigned(wl - wf);
                    if (last_flag) counters[wf] = 0;  // for the next call
                }
            }
            __syncthreads();
            if (last_flag) {
                __threadfence();
                const int live = rows < kRows ? rows : kRows;
                for (int i = threadIdx.x; i < live * (DIM / 4); i += kSplitThreads) {
                    const int r = i / (DIM / 4), d = i % (DIM / 4) * 4;
                    float M = -INFINITY, L = 0.0f;
                    for (int64_t w = wf; w <= wl; ++w) M = fmaxf(M, __ldcg(slot_of(w) + kRows * DIM + r));
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int64_t w = wf; w <= wl; ++w) {
                        const float* f = slot_of(w);
                        const float wm = __ldcg(f + kRows * DIM + r), wlen = __ldcg(f + kRows * DIM + kRows + r);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(f + r * DIM + d));
                        const float a = wm == -INFINITY ? 0.0f : exp2_approx(wm - M);
                        L += a * wlen;
                        acc.x += a * v.x, acc.y += a * v.y, acc.z += a * v.z, acc.w += a * v.w;
                    }
                    finish(r, d, M, L, acc.x, acc.y);
                    finish(r, d + 2, M, L, acc.z, acc.w);
                }
            }
        }
        if (u + 1 < last) next_tile(p, cur, group);
    }
    cp_async_wait<0>();
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

cudaError_t launch_split_any(int dtype, const AttnParams& a, float* part_o, float* part_lse, int sm_count, cudaStream_t s) {
    SplitParams p;
    static_cast<AttnParams&>(p) = a;
    p.part_o = part_o;
    p.part_lse = part_lse;
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
        e = many ? launch_attn_tc(dtype, p, false, 1, o, l, counter, sm_count, s) : launch_split_any(dtype, p, o, l, sm_count, s);
        return e != cudaSuccess ? e : launch_attn_join(dtype, j, s);
    }
    if (!many) return launch_split_any(dtype, p, nullptr, nullptr, sm_count, s);
    const int n = splits_for(tc_pairs(p.n_tokens, group, p.kv.n_seqs, false) * p.kv.n_heads, rows, spare, sm_count);
    if (n == 1) return launch_attn_tc(dtype, p, false, 1, nullptr, nullptr, counter, sm_count, s);
    if ((e = launch_attn_tc(dtype, p, false, n, part_o, part_lse, counter, sm_count, s)) != cudaSuccess) return e;
    j.parts = n;
    return launch_attn_join(dtype, j, s);
}

}  // namespace qx
