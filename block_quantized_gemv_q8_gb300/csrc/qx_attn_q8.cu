// qx_attn_q8.cu -- attention of few rows a sequence over a cache in 8 bits.
//
// The line of units, the ring and the joins are those of 16 bits (qx_attn.cu);
// what a warp does with its keys is not.  Codes become f16, which holds them
// exactly, on the plain units, and that is most of this kernel's work: five
// instructions for four codes.  So the tensor cores' products are turned over --
// S^T = K Q^T and O^T = V^T P^T, the codes the operand of sixteen rows, the
// queries that of eight columns -- and a tile has as many rows as its sequences
// bring, in eights: a converted code meets all of them, and none of the softmax
// is spent on rows that are not there.
//
// Scales: the key's multiplies its scores.  The value's multiplies its
// probability, and that product is rounded to f16; for its range, a row's running
// base counts the scales with the scores.
//
// It is bound by DRAM until its instructions take longer.  Measured: 64 tokens over
// windows of 4096 keys and 4 first ones (8 key heads of 128, bf16, 0.49 GB) 96 us, 5.1
// TB/s, 74 % of the measured copy rate (without the products 87, without the tiles'
// ends 83, without either 70); one token over 131072 keys 55.9 us (73 %); one over
// 1023 keys 8.1; five tokens of 16 sequences over 2000 to 20001 keys, 20 rows, 126 us
// (47 %).
#include "qx_attn.cuh"
#include "qx_attn_codes.cuh"
#include "qx_attn_line.cuh"
#include "qx_layer.cuh"

namespace qx {

namespace {

template <int DIM, int NT>
struct Q8Geom {
    static constexpr int kRowsT = 8 * NT;                 // rows of a tile
    static constexpr int kHalfStage = kUnit * DIM;        // a unit's keys; its values follow
    // Units of a worker at least: a part costs its join, the more rows the more.  (2
    // sequences over 3000 keys, 8 key heads, with two units: 12, 16 and 24 rows 35, 39
    // and 55 us; so 27, 29 and 39.)
    static constexpr int kLeastUnits = NT == 1 ? 2 : NT == 2 ? 8 : 6;
    static constexpr int kRing = 80 * 1024;
    // (24 rows of 128 elements: 133 us for five drafts of 16 sequences, with the split
    // of the others, of which their consumers need more, 142)
    static constexpr int kConsumers = DIM == 128 && NT == 3 ? 208 : kConsumerRegs, kProducers = kConsumerRegs + kProducerRegs - kConsumers;
    static constexpr int kStages = kRing / (2 * kHalfStage);
    static constexpr int kScales = kStages * 2 * kUnit * 4;
    static constexpr int kJoin = (kSplitWarps * 8 * (DIM + 2)) * 4;
    static constexpr int kQueries = NT * (DIM / 16) * 32 * 8;  // the tile's, as the products take them
    static constexpr int kMisc = 1024 + 2 * kRowsT * 4;
    static constexpr size_t kSmem = kRing + kScales + kJoin + kQueries + kMisc;
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
    // workers whose parts the scratch has room for
    static constexpr int kWorkers = int(int64_t(kMaxWorkers) * partial_floats<128>() / partial_floats<DIM, kRowsT>());
};

// A pair of bf16 times f, as f16.
__device__ __forceinline__ uint32_t bf16_to_f16(uint32_t u, float f) {
    const float2 v = unpack2<__nv_bfloat16>(u);
    return pack2<__half>(v.x * f, v.y * f);
}
// An 8 x 8 matrix of 16-bit elements, two of a row in each lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t u) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(u));
    return r;
}

// Probabilities are raised by 2^15 above the row's base (its largest score plus the
// power that the scales stay below), so that times a scale they are below 2^15.
constexpr float kLiftQ8 = 15.0f;

template <typename T, int DIM, int NT>
__global__ void __launch_bounds__(kSplitThreads, 2) attn_split_q8_kernel(const __grid_constant__ SplitParams pp) {
    using G = Q8Geom<DIM, NT>;
    constexpr int ROWS = G::kRowsT, KS = DIM / 16, NS = G::kStages;
    constexpr bool kBf16 = IsBf16<T>::value;
    const AttnParams& p = pp.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* scales = reinterpret_cast<float*>(smem + G::kRing);          // [NS][keys, values][64]
    float* buf = reinterpret_cast<float*>(smem + G::kRing + G::kScales);  // [4 warps][8 rows][DIM], then m and l of each
    float* buf_ml = buf + kSplitWarps * 8 * DIM;
    uint2* queries = reinterpret_cast<uint2*>(smem + G::kRing + G::kScales + G::kJoin);  // [NT][KS][lane]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kRing + G::kScales + G::kJoin + G::kQueries);
    uint64_t* empty = full + NS;
    int64_t* scan = reinterpret_cast<int64_t*>(empty + NS);  // [8]
    Cursor* start = reinterpret_cast<Cursor*>(scan + 2 * kSplitWarps);
    UnitInfo* info = reinterpret_cast<UnitInfo*>(start + 1);  // [NS]
    float* row_scale = reinterpret_cast<float*>(info + NS);  // [ROWS] of bf16: the rows' queries were divided by these powers of two
    int* row_pos = reinterpret_cast<int*>(row_scale + ROWS);  // [ROWS] (-1: none)
    int* last_flag = row_pos + ROWS;
    static_assert((2 * NS + 2 * kSplitWarps) * 8 + sizeof(Cursor) + NS * sizeof(UnitInfo) + 2 * ROWS * 4 + 4 <= G::kMisc,
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
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int group = p.n_q_heads / p.kv.n_heads, B = p.kv.n_seqs;
    Line line;
    if (!open_line<ROWS, G::kLeastUnits>(p, B, group, scan, start, line)) return;
    int64_t left = line.last - line.first;  // units to go

    if (warp >= kSplitWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kProducers));
        // ---- producers, which all walk the line, a lane for each page of a unit: two
        // fetch the codes, of every other unit, and two the scales, and describe the unit.
        // (One warp for all took longer for a unit than its copies: 131072 keys of one
        // token 72.6 us; one for the codes and one for the scales 58.)
        const int role = warp - kSplitWarps;
        const bool describes = role & 1;
        Cursor cur = *start;
        int ui = int(line.first - cur.begin);  // unit of the tile
        const int page_keys = (1 << p.kv.page_shift) < kUnit ? (1 << p.kv.page_shift) : kUnit;
        const int in_page_mask = (1 << p.kv.page_shift) - 1;
        const int boxes = kUnit / page_keys;  // at most 4
        UnitInfo x;
        int page, in_page;  // the lane's page of the unit, or -1 where no row sees any of its keys
        const auto look_up = [&]() {
            int lo, hi;
            const int j = unit_keys(cur.w, ui, lo, hi) + lane * page_keys;
            page = lane < boxes && j + page_keys > lo && j < hi ? page_of(p.kv, cur.b, j) : -1;
            in_page = j & in_page_mask;
        };
        const auto advance = [&]() {
            if (++ui < cur.w.units) return;
            next_tile<ROWS>(p, cur, group, B);
            ui = 0;
            if (describes) line.describe_tile<ROWS>(p, cur, group, x);
        };
        if (describes) line.describe_tile<ROWS>(p, cur, group, x);
        int slot = role >> 1;
        uint32_t phase = 1;  // the ring is empty at first: the wait for the phase before the first returns
        left -= slot;        // units from this warp's first on
        if (slot > 0 && left > 0) advance();
        if (left > 0) look_up();
        int issued = 0;  // (as many as the ring may still hold)
        for (; left > 0; left -= 2) {
            if (describes) line.describe_unit(p, cur, ui, x);
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&empty[slot], phase, kSplitWaitNs, p.kv.err, kErrTimeoutEmpty))) break;
            const unsigned live = __ballot_sync(0xffffffffu, page >= 0);
            if (lane == 0) {
                if (describes) info[slot] = x;
                mbar_arrive_expect_tx(&full[slot], __popc(live) * page_keys * (describes ? 8 : 2 * DIM));
            }
            __syncwarp();
            if (page >= 0) {
                if (describes) {
                    const int64_t from = scale_offset(p.kv, page, cur.hk, in_page);
                    float* to = scales + slot * 2 * kUnit + lane * page_keys;
                    bulk_g2s(to, p.kv.k_scale + from, page_keys * 4, &full[slot]);
                    bulk_g2s(to + kUnit, p.kv.v_scale + from, page_keys * 4, &full[slot]);
                } else {
                    uint8_t* dst = smem + slot * 2 * G::kHalfStage + lane * page_keys * DIM;
                    tma_load_4d(dst, &pp.k_map, 0, in_page, cur.hk, page, &full[slot]);
                    tma_load_4d(dst + G::kHalfStage, &pp.v_map, 0, in_page, cur.hk, page, &full[slot]);
                }
            }
            __syncwarp();
            if (left > 2) {  // the next unit's pages are looked up while its room is awaited
                advance();
                advance();
                look_up();
            }
            if (issued < NS) ++issued;
            slot += 2;
            if (slot >= NS) {
                slot -= NS;
                phase ^= 1;
            }
        }
        // keep the CTA alive until every copy it issued has landed: those of this warp
        // among the last NS units (in earlier ones' slots others have been since, and
        // their barriers are further on).  `left`: 0 where the last unit of all is the
        // other warp's, -1 where it is this one's.
        if (lane == 0) {
            const int most = left <= 0 ? (NS - int(left)) / 2 : (NS + 1) / 2;
            for (int i = issued < most ? issued : most; i > 0; --i) {
                slot -= 2;
                if (slot < 0) {
                    slot += NS;
                    phase ^= 1;
                }
                mbar_wait_bounded(&full[slot], phase ^ 1, kSplitWaitNs, p.kv.err, kErrTimeoutDrain);
            }
        }
        return;
    }

    // ---- consumers.  Two warps take a unit, 32 keys each, and the other two the
    // next: sixteen keys at a time a warp's products and its softmax waited for one
    // another.  Lane 4 g + c has keys g and g + 8 of sixteen, and of each eight rows
    // rows 2 c and 2 c + 1 (of the queries: row g).
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kConsumers));
    const int g = lane >> 2, c = lane & 3;
    float o[KS][NT][4], m[NT][2], l[NT][2];
    int pos_first, pos_last; // of the tile's rows
    // A tile's queries: warp t fetches those of rows 8 t and on (load_tile), and
    // leaves them for all when the tile before is done with its own (open_tile).
    uint4 q[KS / 2];
    const auto load_tile = [&](const UnitInfo& x) {
        const int r = 8 * warp + g;
        const bool live = warp < NT && r < x.rows;
        // a step's elements lie side by side in the codes of a key: lanes c share
        // them in quarters
        const int rr = x.r0 + (live ? r : 0);
        const T* from = static_cast<const T*>(p.q) + int64_t(x.t0 + rr / group) * p.q_stride + int64_t(x.hk * group + rr % group) * DIM +
                        c * (DIM / 4);
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) q[k] = live ? *reinterpret_cast<const uint4*>(from + 8 * k) : make_uint4(0u, 0u, 0u, 0u);
    };
    const auto open_tile = [&](const UnitInfo& x) {
        const int live_rows = x.rows < ROWS ? x.rows : ROWS;
        const int low = x.pos0 + x.r0 / group, high = x.pos0 + (x.r0 + live_rows - 1) / group;
        pos_first = low < 0 ? -1 : low;
        pos_last = high < 0 ? -1 : high;
        if (warp >= NT) return;
        const int r = 8 * warp + g, pos = x.pos0 + (x.r0 + r) / group;
        int e = 14;
        if constexpr (kBf16) {
            // f16 has fewer powers: the row's largest element is brought to 2^14 ..
            // 2^15, which keeps all bits of those above 2^-28 of it, and of the others
            // what 2^-39 of it leaves
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < KS / 2; ++k) {
                const uint32_t u[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
                for (int x = 0; x < 4; ++x) top = max(top, max(u[x] << 16 & 0x7fff0000u, u[x] & 0x7fff0000u));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            e = max(int(top >> 23), 15);
            const float f = power_of_two(268 - e);
#pragma unroll
            for (int k = 0; k < KS / 2; ++k)
                q[k] = make_uint4(bf16_to_f16(q[k].x, f), bf16_to_f16(q[k].y, f), bf16_to_f16(q[k].z, f), bf16_to_f16(q[k].w, f));
        }
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) {
            queries[(warp * KS + 2 * k) * 32 + lane] = make_uint2(q[k].x, q[k].y);
            queries[(warp * KS + 2 * k + 1) * 32 + lane] = make_uint2(q[k].z, q[k].w);
        }
        if (c == 0) {
            row_scale[r] = power_of_two(e - 14);
            row_pos[r] = r < live_rows && pos >= 0 ? pos : -1;
        }
    };
    {
        UnitInfo x;
        x.t0 = start->w.t0, x.pos0 = start->w.pos0, x.hk = start->hk;
        x.r0 = ROWS * start->rt, x.rows = start->w.tokens * group - x.r0;
        load_tile(x);
        open_tile(x);
        consumers_sync();
    }
    float* partials = reinterpret_cast<float*>(static_cast<uint8_t*>(p.scratch) + kCounterBytes);
    unsigned* counters = static_cast<unsigned*>(p.scratch);
    const int window = p.window > 0 && p.window < INT32_MAX ? int(p.window) : INT32_MAX;
    const int sinks = p.sinks < INT32_MAX ? int(p.sinks) : INT32_MAX;
    const uint32_t ring = smem_addr(smem);
    const int first_key = 32 * (warp & 1);  // of a unit
    // 16-byte chunk `chunk` of a key's codes in the swizzle of the copies
    const auto place = [](int key, int chunk) { return key * DIM + ((DIM == 128 ? chunk ^ (key & 7) : chunk ^ ((key >> 1) & 3)) << 4); };
    int slot = 0;
    uint32_t phase = 0;
    // (waits that run out: as in the kernel of 16 bits)
    bool ok = true, together = true;
    const auto arrived = [&]() {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[slot], phase, kSplitWaitNs, p.kv.err, kErrTimeoutFull));
    };
    arrived();
    for (int turn = warp >> 1; left > 0 && ok; --left, turn ^= 1) {
        const int flags = info[slot].flags, lo = info[slot].lo, hi = info[slot].hi;
        const int j0 = info[slot].j0 + first_key;  // this warp's keys
        if (flags & kOpens) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int i = 0; i < 2; ++i) m[t][i] = -INFINITY, l[t][i] = 0.0f;
#pragma unroll
                for (int d = 0; d < KS; ++d) o[d][t][0] = o[d][t][1] = o[d][t][2] = o[d][t][3] = 0.0f;
            }
        }
        if (turn == 0 && j0 + 32 > lo && j0 < hi) {
            const uint8_t* const keys = smem + slot * 2 * G::kHalfStage;
            const uint32_t values = ring + slot * 2 * G::kHalfStage + G::kHalfStage;
            const float* const sc = scales + slot * 2 * kUnit + first_key + g;
            float s[2][NT][4] = {}, dv[2][2];  // of sixteen keys each
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += 4) {
                uint32_t w[2][2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint4 u = *reinterpret_cast<const uint4*>(keys + place(first_key + 16 * h + 8 * x + g, c * (KS / 4) + k0 / 4));
                        w[h][x][0] = u.x ^ 0x80808080u, w[h][x][1] = u.y ^ 0x80808080u;
                        w[h][x][2] = u.z ^ 0x80808080u, w[h][x][3] = u.w ^ 0x80808080u;
                    }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint2 b[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) b[t] = queries[(t * KS + k0 + k) * 32 + lane];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a[4] = {code_pair<0, 1>(w[h][0][k]), code_pair<0, 1>(w[h][1][k]), code_pair<2, 3>(w[h][0][k]),
                                               code_pair<2, 3>(w[h][1][k])};
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma16816<__half>(s[h][t], a, b[t].x, b[t].y);
                    }
                }
            }
            float2 rows_f[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) rows_f[t] = kBf16 ? *reinterpret_cast<const float2*>(row_scale + 8 * t + 2 * c) : make_float2(1.0f, 1.0f);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    // A scale that is no number makes no numbers of the scores, of the rows
                    // that see it; the product of probability and scale is every row's.
                    float d = sc[16 * h + 8 * x], e = sc[kUnit + 16 * h + 8 * x];
                    const bool sound = fabsf(d) < INFINITY && fabsf(e) < INFINITY;
                    dv[h][x] = sound ? e : 0.0f;
                    const float f = sound ? d * inner_scale(p.scale_log2) : __uint_as_float(0x7fffffffu);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (kBf16) s[h][t][2 * x] *= rows_f[t].x, s[h][t][2 * x + 1] *= rows_f[t].y;
                        s[h][t][2 * x] *= f;
                        s[h][t][2 * x + 1] *= f;
                    }
                }
            if (fabsf(p.scale_log2) > 1.0f) {
                const float f = outer_scale(p.scale_log2);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[h][t][x] *= f;
            }
            const bool sink_unit = flags & kSink;
            if (j0 < lo || j0 + 32 > hi || j0 + 31 > pos_first || (!sink_unit && pos_last - window >= j0)) {
                // some row does not see some of them
                const int a = lo - j0, b = hi - j0, f = sinks - j0;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int pos = row_pos[8 * t + 2 * c + i];
                        const int end = pos - j0 + 1 < b ? pos - j0 + 1 : b;
                        const int low = pos >= window ? pos - window + 1 : 0;  // of the row's window
                        const int from = sink_unit || low - j0 < a ? a : low - j0;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int j = 16 * h + 8 * x + g;
                                if (!(j < end && (j >= from || (j >= a && j < f)))) s[h][t][2 * x + i] = -INFINITY;
                            }
                    }
            }
            // A row's base moves less and less often: the lanes meet, and o is rescaled, only
            // when one asks for it (a lane asks for all of its keys, and counts those that
            // the row sees).
            const float power = scale_power(fmaxf(fmaxf(fabsf(dv[0][0]), fabsf(dv[0][1])), fmaxf(fabsf(dv[1][0]), fabsf(dv[1][1]))));
            float mx[NT][2];
            bool moved = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mx[t][i] = fmaxf(fmaxf(s[0][t][i], s[0][t][2 + i]), fmaxf(s[1][t][i], s[1][t][2 + i]));
                    moved |= mx[t][i] + power > m[t][i];
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float d = 0.0f;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int x = 0; x < 2; ++x) d = fmaxf(d, s[h][t][2 * x + i] == -INFINITY ? 0.0f : fabsf(dv[h][x]));
                        float top = fmaxf(m[t][i], mx[t][i] + scale_power(d));
#pragma unroll
                        for (int w = 4; w <= 16; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                        const float h = top == -INFINITY ? 1.0f : exp2_approx(0.5f * (m[t][i] - top)), a = h * h;
                        l[t][i] = twice(l[t][i], h);
                        m[t][i] = top;
#pragma unroll
                        for (int k = 0; k < KS; ++k) o[k][t][i] *= a, o[k][t][2 + i] *= a;
                    }
            }
            uint32_t pf[2][NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float base[2] = {m[t][0] == -INFINITY ? 0.0f : m[t][0] - kLiftQ8, m[t][1] == -INFINITY ? 0.0f : m[t][1] - kLiftQ8};
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            w[i] = exp2_approx(s[h][t][2 * x + i] - base[i]);
                            l[t][i] += w[i];
                            w[i] *= dv[h][x];
                        }
                        pf[h][t][x] = transposed(pack2<__half>(w[0], w[1]));
                    }
            }
            // As pairs of codes the 16-byte chunks of the values are what ldmatrix
            // transposes: a register has elements 2 g and 2 g + 1 of two keys.  The
            // sixteen rows of the product are a chunk's even elements, then its odd ones.
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t b[4];
                    ldmatrix4_t(values + place(first_key + 16 * h + (lane & 15), k + (lane >> 4)), b);
#pragma unroll
                    for (int x = 0; x < 4; ++x) b[x] ^= 0x80808080u;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t a[4] = {code_pair<0, 2>(b[2 * y]), code_pair<1, 3>(b[2 * y]), code_pair<0, 2>(b[2 * y + 1]),
                                               code_pair<1, 3>(b[2 * y + 1])};
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma16816<__half>(o[k + y][t], a, pf[h][t][0], pf[h][t][1]);
                    }
                }
        }
        UnitInfo done;
        if (flags & kCloses) done = info[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (++slot == NS) {
            slot = 0;
            phase ^= 1;
        }
        if (left > 1) arrived();
        if (!(flags & kCloses)) continue;
        // ---- the tile ends here (for this worker).  The next one's queries are on
        // their way while its warps are joined, eight rows at a time: every warp
        // leaves its (m, l, o), and every thread then joins some elements.
        if (left > 1 && ok) load_tile(info[slot]);
        const int rows = done.rows;  // (ROWS at most count)
        const auto part_at = [&](int i) -> float* { return partials + int64_t(i) * partial_floats<DIM, ROWS>(); };
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (8 * t >= rows) break;
            const int live = rows - 8 * t < 8 ? rows - 8 * t : 8;
#pragma unroll
            for (int w = 4; w <= 16; w <<= 1)
#pragma unroll
                for (int i = 0; i < 2; ++i) l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], w);
            if (t > 0) consumers_sync();  // the eight before are read
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * c + i;
                if (r >= live) continue;
                // (groups of eight elements permuted by the row, for the banks)
                float* row = buf + (8 * warp + r) * DIM + 2 * (g & 3);
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    *reinterpret_cast<float2*>(row + 8 * ((2 * k + (g >> 2)) ^ r)) = make_float2(o[k][t][i], o[k][t][2 + i]);
                if (g == 0) *reinterpret_cast<float2*>(buf_ml + 2 * (8 * warp + r)) = make_float2(m[t][i] - kLiftQ8, l[t][i]);
            }
            if (t > 0) consumers_sync();
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
                    const float h = ml[w].x == -INFINITY ? 0.0f : exp2_approx(0.5f * (ml[w].x - M)), a = h * h;
                    const float4 v = *reinterpret_cast<const float4*>(buf + (8 * w + r) * DIM + (d ^ (8 * r)));
                    L += twice(ml[w].y, h);
                    acc.x += a * v.x, acc.y += a * v.y, acc.z += a * v.z, acc.w += a * v.w;
                }
                if (done.parts == 0) {
                    write_four<T, DIM>(pp, done, 8 * t + r, d, M, L, acc, false);
                } else {
                    float* to = part_at(int(blockIdx.x) == done.wf ? done.part : 2 * int(blockIdx.x));
                    *reinterpret_cast<float4*>(to + (8 * t + r) * DIM + d) = acc;
                    if (d == 0) *reinterpret_cast<float2*>(to + ROWS * DIM + 2 * (8 * t + r)) = make_float2(M, L);
                }
            }
        }
        if (!together) break;
        if (left > 1) open_tile(info[slot]);  // (all warps are past the tile's products)
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
            if (*last_flag) join_parts<T, DIM, ROWS, true>(pp, done, buf, false);
        }
        consumers_sync();  // the buffer is read, and the next tile's queries are there
    }
    if (!ok && together) consumers_agree(false);
}

template <typename T, int DIM, int NT>
cudaError_t launch_split_q8(const AttnParams& a, int sm_count, cudaStream_t s) {
    using G = Q8Geom<DIM, NT>;
    SplitParams p;
    p.a = a;
    p.part_o = p.part_lse = nullptr;
    p.beside = p.prefix = 0;
    if (!encode_code_maps(a.kv, kUnit, &p.k_map, &p.v_map)) return cudaErrorInvalidValue;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(attn_split_q8_kernel<T, DIM, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(G::kSmem));
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    int workers = 2 * sm_count < kMaxWorkers ? 2 * sm_count : kMaxWorkers;
    if (workers > G::kWorkers) workers = G::kWorkers;
    return launch_serial(attn_split_q8_kernel<T, DIM, NT>, dim3(unsigned(workers)), kSplitThreads, G::kSmem, s, p);
}

template <typename T, int DIM>
cudaError_t launch_rows_q8(const AttnParams& p, int sm_count, cudaStream_t s) {
    // Rows of a key head a sequence, on average.
    const int64_t rows = int64_t(p.n_tokens) * (p.n_q_heads / p.kv.n_heads), seqs = p.kv.n_seqs;
    if (rows <= 8 * seqs) return launch_split_q8<T, DIM, 1>(p, sm_count, s);
    if (rows <= 16 * seqs) return launch_split_q8<T, DIM, 2>(p, sm_count, s);
    return launch_split_q8<T, DIM, 3>(p, sm_count, s);
}

}  // namespace

cudaError_t launch_attn_split_q8(int dtype, const AttnParams& p, int sm_count, cudaStream_t s) {
    const bool f16 = dtype == QX_F16;
    if (p.kv.head_dim == 128) return f16 ? launch_rows_q8<__half, 128>(p, sm_count, s) : launch_rows_q8<__nv_bfloat16, 128>(p, sm_count, s);
    return f16 ? launch_rows_q8<__half, 64>(p, sm_count, s) : launch_rows_q8<__nv_bfloat16, 64>(p, sm_count, s);
}

}  // namespace qx
