// qx_attn.cu -- attention over the paged cache.
//
// Row (token t, query head h) at position pos: with s_j = scale q . k_j over
// the keys it sees, m the running maximum, l the running sum of exp(s_j - m)
// and o the running sum of exp(s_j - m) v_j, a block of keys with maximum m'
// turns (m, l, o) into (M, l e^(m-M) + sum e^(s_j-M), o e^(m-M) + ...), M =
// max(m, m'); the output is o / l.  Exponents are taken to base 2 with
// scale * log2(e) folded into the scores.
#include "qx_attn.cuh"
#include "qx_attn_line.cuh"
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
// 128.  (T: queries and output, C: the cache, codes of int8_t.)
template <typename T, typename C>
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
    row_sums<C, 4>(p, seq, pos, hk, 0, INT64_MAX, 32 * warp, 32 * kRowWarps,
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

    Line line;
    if (!open_line<kRows>(p, B, group, scan, start, line)) {
        if (pp.beside) pdl_wait_prior_grid();
        return;
    }
    const int64_t first = line.first;
    int64_t left = line.last - first;  // units to go

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
                line.describe<kRows>(p, cur, ui, group, x);
                info[slot] = x;
                mbar_arrive(&full[slot]);
            }
            __syncwarp();
            if (left > 1) {  // the next unit's pages are looked up while its room is awaited
                if (++ui == cur.w.units) {
                    next_tile<kRows>(p, cur, group, B);
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

template <typename T, typename C = T>
cudaError_t launch_row(const AttnParams& p, cudaStream_t s) {
    return launch_serial(attn_row_kernel<T, C>, dim3(unsigned(p.n_tokens), unsigned(p.n_q_heads)), 32 * kRowWarps, 0, s, p);
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

// Where a call's parts lie in its scratch, and how many a row of prompts has (0:
// none).
struct Parts {
    float *o, *lse;
    unsigned* counter;
    int slots;
};
Parts parts_of(const AttnParams& p, int sm_count) {
    const int group = p.n_q_heads / p.kv.n_heads;
    const int64_t rows = int64_t(p.n_tokens) * p.n_q_heads, spare = part_rows(rows);
    Parts x;
    x.lse = reinterpret_cast<float*>(static_cast<char*>(p.scratch) + kSplitScratch);
    x.o = x.lse + spare;
    x.counter = static_cast<unsigned*>(p.scratch) + kMaxWorkers;
    int64_t keys = p.kv.table_stride << p.kv.page_shift;
    if (p.window > 0 && p.window + p.sinks + 256 < keys) keys = p.window + p.sinks + 256;
    const int64_t pairs = tc_pairs(p.n_tokens, group, p.kv.n_seqs, false) * p.kv.n_heads;
    x.slots = slots_for(pairs, (keys + 127) / 128, p.kv.n_seqs, rows, spare, sm_count);
    return x;
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
    const Parts parts = parts_of(p, sm_count);
    // a scale that is not positive is an oddity that only the split kernel serves
    if (rows > kMaxSharedRows || p.n_tokens < 2 || p.scale_log2 <= 0.0f) p.shared_len = 0;
    // Rows of a key head a sequence, on average: the split kernel reads a
    // sequence's keys once for every 16 of them, the tensor cores' once for
    // 256, but only they need whole tiles to be efficient.
    const bool many = int64_t(p.n_tokens) * group >= 64 * int64_t(p.kv.n_seqs) && p.scale_log2 > 0.0f;
    JoinParams j;
    j.a = p;
    j.part_o = parts.o;
    j.part_lse = parts.lse;
    j.parts = 0;
    cudaError_t e;
    if (p.shared_len > 0) {
        // A short prefix for few rows: the split kernel takes it with the
        // tails, though it reads it once for every 16 rows.  (16 sequences
        // behind 2000 keys: 23 us, against 32 with a launch of its own; 64
        // behind 2000 or 16 behind 8000: 49 and 41 against 46 and 37; 4 behind
        // 8000, whose tiles many workers share: 36 against 28.)
        const int64_t units = (int64_t(p.n_tokens) * group + kRows - 1) / kRows * p.kv.n_heads * ((p.shared_len + kUnit - 1) / kUnit);
        if (!many && p.shared_len <= kShortPrefix && units <= int64_t(kPrefixUnits) * 2 * sm_count) {
            j.parts = 2;
            e = launch_split_any(dtype, p, parts.o, parts.lse, false, true, sm_count, s);
            return e != cudaSuccess ? e : launch_attn_join(dtype, j, s);
        }
        // the prefix, the tails beside it, and both joined
        const int slots = slots_for(0, (p.shared_len + 127) / 128, 1, rows, part_rows(rows) - rows, sm_count);
        if ((e = launch_attn_tc(dtype, p, true, slots, parts.o, parts.lse, parts.counter, sm_count, s)) != cudaSuccess) return e;
        j.parts = slots > 0 ? slots : 1;
        float* o = parts.o + j.parts * rows * dim;
        float* l = parts.lse + j.parts * rows;
        ++j.parts;
        e = many ? launch_attn_tc(dtype, p, false, 0, o, l, parts.counter, sm_count, s) : launch_split_any(dtype, p, o, l, true, false, sm_count, s);
        return e != cudaSuccess ? e : launch_attn_join(dtype, j, s);
    }
    if (!many) return launch_split_any(dtype, p, nullptr, nullptr, false, false, sm_count, s);
    if (parts.slots == 0) return launch_attn_tc(dtype, p, false, 0, nullptr, nullptr, parts.counter, sm_count, s);
    if ((e = launch_attn_tc(dtype, p, false, parts.slots, parts.o, parts.lse, parts.counter, sm_count, s)) != cudaSuccess) return e;
    j.parts = parts.slots;
    return launch_attn_join(dtype, j, s);
}

cudaError_t launch_attn_q8(int dtype, const AttnParams& p, int sm_count, cudaStream_t s) {
    const int dim = p.kv.head_dim;
    if (dim != 64 && dim != 128) return dtype == QX_F16 ? launch_row<__half, int8_t>(p, s) : launch_row<__nv_bfloat16, int8_t>(p, s);
    const int group = p.n_q_heads / p.kv.n_heads;
    // Rows of a key head a sequence, on average: up to the split kernel's largest tile
    // at head size 128 (16 sequences over 8000 keys, 24 rows: 97 us against the tensor
    // cores' 145; 32 rows, two tiles: 160 against 145), two at 64 (42 rows: 41 against
    // 53; 56: 53 against 53).  Scales of the scores: as in 16 bits.
    const int64_t most = (dim == 128 ? 24 : 48) * int64_t(p.kv.n_seqs);
    if (int64_t(p.n_tokens) * group <= most || p.scale_log2 <= 0.0f) return launch_attn_split_q8(dtype, p, sm_count, s);
    const Parts parts = parts_of(p, sm_count);
    if (parts.slots == 0) return launch_attn_tc_q8(dtype, p, 0, nullptr, nullptr, parts.counter, sm_count, s);
    const cudaError_t e = launch_attn_tc_q8(dtype, p, parts.slots, parts.o, parts.lse, parts.counter, sm_count, s);
    if (e != cudaSuccess) return e;
    JoinParams j;
    j.a = p;
    j.part_o = parts.o;
    j.part_lse = parts.lse;
    j.parts = parts.slots;
    return launch_attn_join(dtype, j, s);
}

}  // namespace qx
