// ibp_select.hip -- which pages of a cache a query reads: per-page bounds of
// the keys, and the choice of the pages with the highest bound on the score.
//
// For a page with lo[d] <= k[d] <= hi[d], q.k <= sum over d of
// max(q[d] lo[d], q[d] hi[d]), for finite bounds the sum of max(q,0) hi +
// min(q,0) lo: a product of the vector (q+, q-) with (hi, lo), twice head_dim
// long.  (With infinite bounds the product has 0 times infinity where the
// maximum has none; such pages are left to the sums in 64 bits.)  Neighbouring
// scores decide which pages are read, so the definition sums in 64 bits and
// rounds once; the kernels get there in two steps:
//   1. k_scores multiplies on the matrix cores in 32 bits, and a second
//      product of the absolute values bounds how far each sum can be off;
//   2. k_choose finds the n-th largest of these, roughly, and sums again in 64
//      bits only the pages that lie within that bound of it, usually a few,
//      and those whose 32-bit sums say nothing (infinities, NaN, overflow).
// The result is the one that 64-bit sums of all pages give.  Short rows with
// pages of their own take both steps in one launch, k_select.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/ibp.h"
#include "ibp_host.hpp"
#include "ibp_kv_math.hpp"

namespace ibp {

// ---------------------------------------------------------------------------
// Bounds.  One wave per page, as the decode of small tensors: a lane holds
// eight numbers (four words) of one token per vector, and since a page row is
// a power of two of words and at most 256 of them, the same eight dims in
// every vector.  So a lane keeps its dims' running bounds over its vectors and
// the lanes of one dim group are joined at the end.  Bound by the pages' bytes
// (65,536 pages of 4 KiB under a whole-page period: 64.3 us, 4.7 TB/s read and
// written, what a large copy reaches; 67 pages: 4.2 us, one launch's latency).
// ---------------------------------------------------------------------------
constexpr uint32_t kBoundWaves = 4;

__device__ __forceinline__ void join_bounds(float& lo, float& hi, float x_lo, float x_hi) {
    // (minimum and maximum that pass a NaN on)
    lo = __builtin_elementwise_minimum(lo, x_lo);
    hi = __builtin_elementwise_maximum(hi, x_hi);
}

template <class E, int NV, bool TAB_LDS>
__global__ __launch_bounds__(kWave * kBoundWaves) void k_page_bounds(Pool pool, uint32_t row_words,
                                                                     const int64_t* __restrict__ ids,
                                                                     const int32_t* __restrict__ tokens, uint64_t n,
                                                                     uint32_t* __restrict__ bounds) {
    extern __shared__ __align__(16) uint32_t smem[];
    const uint32_t lane = lane_id(), wib = uniform(threadIdx.x / kWave);
    const uint32_t tab_words = TAB_LDS ? page_tab_words(pool.Mw, pool.runs) : 0u;
    if (TAB_LDS) {
        stage_page_tables(pool, smem);
        __syncthreads();
    }
    const PageTab tab = page_tab(pool, smem, TAB_LDS);
    uint32_t* stage = smem + tab_words + wib * page_stage_words<NV>();
    const uint32_t row_lanes = row_words / 4;  // lanes that one token takes
    const uint32_t row_shift = 31 - __builtin_clz(row_words);
    const uint64_t stride = (uint64_t)gridDim.x * kBoundWaves;
    for (uint64_t i = (uint64_t)blockIdx.x * kBoundWaves + wib; i < n; i += stride) {
        const int64_t id64 = (int64_t)uniform64((uint64_t)ids[i]);
        const int32_t held = tokens ? (int32_t)uniform((uint32_t)tokens[i]) : 0x7FFFFFFF;
        if (id64 == -1 || held <= 0) continue;
        const uint32_t id = page_id(id64, pool.n_slots);
        if (id == kNoPage) {
            latch_error(pool.err, kErrRange);
            continue;
        }
        __builtin_amdgcn_wave_barrier();
        u32x4 st[NV];
        load_page<NV>(st, pool.slots, id);
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            lo[j] = __builtin_inff();
            hi[j] = -__builtin_inff();
        }
        auto take = [&](uint32_t w, const u32x4& x) __attribute__((always_inline)) {
            if ((int32_t)(w >> row_shift) >= held) return;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y = E::from_bits(x[j >> 1] >> (16 * (j & 1)));
                join_bounds(lo[j], hi[j], y, y);
            }
        };
        if (uniform(page_bit(pool.bitmask, id))) {
            stage_page<NV>(st, stage);
            if (!rebuild_page<NV, 2>(pool, tab, stage, take)) latch_error(pool.err, kErrCorrupt);
        } else {
#pragma unroll
            for (int r = 0; r < NV; ++r) take(256u * r + 4u * lane, st[r]);
        }
        for (uint32_t o = row_lanes; o < kWave; o <<= 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                join_bounds(lo[j], hi[j], __shfl_xor(lo[j], (int)o), __shfl_xor(hi[j], (int)o));
        }
        if (lane < row_lanes) {
            u32x4 a, b;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = E::pack(lo[2 * j], lo[2 * j + 1]);
                b[j] = E::pack(hi[2 * j], hi[2 * j + 1]);
            }
            u32x4* out = reinterpret_cast<u32x4*>(bounds + (uint64_t)id * 2 * row_words);
            out[lane] = a;
            out[row_lanes + lane] = b;
        }
    }
}

// ---------------------------------------------------------------------------
// Scores.  A operand: 16 columns of (row, query head), lane l holding column
// l % 16; B operand: the bounds of 16 pages.  D then holds, in lane l, page
// l % 16 and columns 4 (l / 16) .. + 3, so the maximum over a group's heads is
// taken inside a lane for groups of up to four heads and across the four
// lanes of a page for larger ones.  Groups are padded to `pad` heads (1, 2, 4,
// 8 or a multiple of 16), so that no group straddles tiles.
//
// A wave takes 64 blocks of one head for CT tiles of columns.
//   k_scores, decoding, where every row has pages of its own: CT = 1, other
//     blocks in every wave, operands straight from memory.  Bound by the
//     bounds' bytes (16 rows of 2,048 blocks by 8 heads of 128 dims, 134 MB:
//     21.6 us, 6.2 TB/s out of the last-level cache).
//   k_scores_shared, rows that share a sequence: the four waves of a workgroup
//     take the same blocks for rows of their own, and bring the bounds to LDS
//     once.  An operand's 16 lanes are 16 pages, so that a load from memory
//     takes the cache 64 lookups instead of 8: read that way, with each wave
//     on its own, the cache's one lookup per cycle was the limit (512 rows of
//     4,096 blocks by 8 heads of 128 dims: 138 us, 77 through LDS, of which
//     the matrix cores work 27).  Workgroups whose rows belong to several
//     sequences, and 256 dims, which LDS has no room for, still read that way.
// Heads are the fastest index of the grid, so that with eight of them each
// XCD's L2 holds the bounds of one (decoding: 22.6 us otherwise).
// ---------------------------------------------------------------------------
struct SelectArgs {
    const void* q;
    const void* bounds;
    const int64_t* table;
    const int32_t* lens;
    const int32_t* row_seq;
    float* scores;   // [n_rows][kv heads][pitch]
    float* slack;    // [n_rows][kv heads][chunks]: sum of absolute products, the largest of 64 blocks
    int32_t* out;
    uint32_t* err;
    uint64_t n_rows, n_seqs, n_slots, blocks, pitch, chunks;
    int64_t q_row, q_head;
    uint32_t kv_heads, group, page_tokens, keep_first, keep_last, n_out;
    uint32_t pad;            // heads a group takes in a tile's columns
    uint32_t log2_pad;       // its logarithm, 31 for groups of several tiles
    uint32_t rows_per_tile;  // 16 / pad, or 1
    uint32_t head_tiles;     // column tiles of one row (pad / 16, or 1)
    uint32_t wave_rows;      // rows of one wave
    uint32_t span;           // times 64 blocks per wave
};

constexpr uint32_t kScoreWaves = 4;
constexpr uint32_t kWaveBlocks = 64;

// Error of a 32-bit sum of 2 * dim products, relative to the sum of their
// absolute values: 2 * dim additions, each off by at most 2^-23 (which covers
// rounding towards zero inside the matrix cores); the products are exact.
__host__ __device__ constexpr float sum_error(int dim) { return (float)dim / 4194304.0f; }

// And beside that: products and sums below the normal range of 32 bits may be
// off by as much as its smallest number (in 64 bits such a sum is a score of
// its own).
__host__ __device__ constexpr float sum_underflow(int dim) { return (float)dim * 0x1p-125f; }

// Sums of absolute values from here on may overflow in another order.
constexpr float kLargestSum = 1e38f;

__device__ __forceinline__ float max_or_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// The score m of a block whose absolute values sum up to e, as it is stored:
// NaN where e says nothing of it, being infinite, nearly so, or a NaN (an
// infinity, a NaN in the bounds, an overflow of 32 bits): k_choose sums such
// blocks in 64 bits before it does anything else.  Other blocks' e counts for
// the row's slack.
__device__ __forceinline__ void settle(float& m, float e, float& slack) {
    const bool known = e < kLargestSum;
    m = known ? m : __builtin_nanf("");
    slack = fmaxf(slack, known ? e : 0.f);
}

// Blocks of row r (0 where its sequence or length is not valid).
__device__ __forceinline__ uint32_t row_blocks(const SelectArgs& a, uint64_t r, int64_t* seq) {
    *seq = a.row_seq ? (int64_t)a.row_seq[r] : (int64_t)r;
    const int64_t len = a.lens[r];
    if (*seq < 0 || (uint64_t)*seq >= a.n_seqs || len < 0) return 0;
    const uint64_t nb = ((uint64_t)len + a.page_tokens - 1) / a.page_tokens;
    return (uint32_t)(nb < a.blocks ? nb : a.blocks);
}

// The bounds of 64 blocks in LDS, rows padded so that 16 blocks' operands
// spread over all banks.
template <int D>
struct BoundTile {
    static constexpr uint32_t stride = 4 * D + 16, bytes = kWaveBlocks * stride;
    static constexpr bool fits = D <= 128;
};

// Of a workgroup whose waves' rows all belong to one sequence: that sequence
// and its most blocks (`tile` as well, else NULL).
struct Together {
    char* tile;
    uint32_t seq, nb;
};

// One wave: rows r0 .. of head h, blocks b_first .. of a.span * 64.  STAGED:
// the whole workgroup, which brings the bounds to LDS 64 blocks at a time.
template <class E, int D, int CT, bool ONE_ROW, bool STAGED>
__device__ __forceinline__ void score_blocks(const SelectArgs& a, uint64_t r0, uint32_t h, uint32_t b_first,
                                             const Together wg = {}) {
    using V8 = typename E::V8;
    constexpr int DK = D / 32;
    const uint32_t lane = lane_id();
    const uint32_t col = lane & 15u, g = lane >> 4;
    // lane l: row r0 + l of the wave (at most 64), its sequence and blocks
    int64_t my_seq = -1;
    uint32_t my_nb = 0;
    if (lane < a.wave_rows && r0 + lane < a.n_rows) my_nb = row_blocks(a, r0 + lane, &my_seq);
    uint64_t todo = ballot(my_nb > b_first);
    bool first_turn = STAGED;
    while (todo || first_turn) {  // one sequence after another; usually there is one
        first_turn = false;
        const uint32_t seq = STAGED ? wg.seq : lane_value((uint32_t)my_seq, (int)__builtin_ctzll(todo));
        const uint64_t mine = todo & ballot((uint32_t)my_seq == seq && my_nb > b_first);
        todo &= ~mine;
        uint32_t nb = wg.nb;
        if (!STAGED)
            for (uint64_t m = mine; m; m &= m - 1) nb = max(nb, lane_value(my_nb, (int)__builtin_ctzll(m)));
        // 64 page ids at once
        auto ids_at = [&](uint32_t b) __attribute__((always_inline)) -> uint32_t {
            if (b + lane >= nb) return kNoPage;
            const uint32_t id =
                page_id(a.table[((uint64_t)seq * a.kv_heads + h) * a.blocks + b + lane], (uint32_t)a.n_slots);
            if (id == kNoPage) atomicCAS(a.err, 0u, (uint32_t)kErrRange);
            return id;
        };
        const uint32_t b_end = min(nb, b_first + kWaveBlocks * a.span);
        const uint32_t col_tiles = a.head_tiles * ((a.wave_rows + a.rows_per_tile - 1) / a.rows_per_tile);
        for (uint32_t ct0 = 0; ct0 < col_tiles; ct0 += CT) {
            // the numbers above zero, and those below, of each column; a head
            // with a NaN, whose scores are all the lowest, becomes zeros and no
            // column's head
            V8 qp[CT][DK], qm[CT][DK];
            uint32_t with_nan[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const uint32_t x = (ct0 + c) * 16 + col;  // column of the wave
                const uint32_t row = x >> a.log2_pad, head = x - (row << a.log2_pad);
                const bool on = head < a.group && row < a.wave_rows && ((mine >> (row & 63u)) & 1u);
                const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)(r0 + row) * a.q_row +
                                    (int64_t)(h * a.group + head) * a.q_head;
                u32x4 v[DK];
                u16x2 top = {0, 0};
#pragma unroll
                for (int kk = 0; kk < DK; ++kk) {
                    v[kk] = on ? load_eight(q + 32 * kk + 8 * g) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        top = __builtin_elementwise_max(top, bits_as<u16x2>(v[kk][j] & 0x7FFF7FFFu));
                }
                const uint64_t nan = ballot(top.x > E::kExponent || top.y > E::kExponent);
                with_nan[c] = (uint32_t)((nan | nan >> 16 | nan >> 32 | nan >> 48) & 0xFFFFu);
                const uint32_t keep = ((with_nan[c] >> col) & 1u) - 1u;
#pragma unroll
                for (int kk = 0; kk < DK; ++kk) {
                    u32x4 p, m;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t x = v[kk][j] & keep, neg = (x >> 15 & 0x10001u) * 0xFFFFu;
                        p[j] = x & ~neg;
                        m[j] = x & neg;
                    }
                    qp[c][kk] = bits_as<V8>(p);
                    qm[c][kk] = bits_as<V8>(m);
                }
            }
            // of columns 4 g + i of each tile: which hold a head, the row of
            // the first, and the blocks of each row they belong to
            constexpr int ROWS = ONE_ROW ? 1 : 4;
            uint32_t heads[CT], row_nb[CT][ROWS];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                heads[c] = 0;
                const uint32_t x0 = (ct0 + c) * 16 + 4 * g;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t row = (x0 + i) >> a.log2_pad;
                    if (x0 + i - (row << a.log2_pad) < a.group && !((with_nan[c] >> (4 * g + i)) & 1u))
                        heads[c] |= 1u << i;
                    if (i < ROWS) {
                        const bool live = row < a.wave_rows && ((mine >> (row & 63u)) & 1u);
                        const uint32_t n = (uint32_t)__shfl((int)my_nb, (int)(row & 63u));
                        row_nb[c][i] = live ? n : 0u;
                    }
                }
            }
            uint32_t id_next = ids_at(b_first);
            for (uint32_t b0 = b_first; b0 < b_end; b0 += kWaveBlocks) {
                const uint32_t id = id_next;
                id_next = b0 + kWaveBlocks < b_end ? ids_at(b0 + kWaveBlocks) : kNoPage;
                const uint32_t tiles = min((b_end - b0 + 15) / 16, kWaveBlocks / 16);
                if constexpr (STAGED) {
                    // a wave brings 16 blocks, each lane 16 bytes at a time
                    constexpr uint32_t PIECES = D / 4, AT_ONCE = kWave / PIECES;
                    const uint32_t wib = uniform(threadIdx.x / kWave);
                    u32x4 piece[16 / AT_ONCE];
#pragma unroll
                    for (uint32_t i = 0; i < 16 / AT_ONCE; ++i) {
                        const uint32_t pid = (uint32_t)__shfl((int)id, (int)(16 * wib + AT_ONCE * i + lane / PIECES));
                        piece[i] = *reinterpret_cast<const u32x4*>(
                            static_cast<const char*>(a.bounds) + (uint64_t)(pid == kNoPage ? 0u : pid) * (4ull * D) +
                            16 * (lane % PIECES));
                    }
                    __syncthreads();  // the 64 blocks before have been read
#pragma unroll
                    for (uint32_t i = 0; i < 16 / AT_ONCE; ++i)
                        *reinterpret_cast<u32x4*>(wg.tile + (16 * wib + AT_ONCE * i + lane / PIECES) * BoundTile<D>::stride +
                                                  16 * (lane % PIECES)) = piece[i];
                    __syncthreads();
                }
                float slack[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) slack[c] = 0.f;
#pragma unroll 1
                for (uint32_t t = 0; t < tiles; ++t) {
                    V8 lo[DK], hi[DK];
                    auto read = [&](const char* base) __attribute__((always_inline)) {
#pragma unroll
                        for (int kk = 0; kk < DK; ++kk) {
                            lo[kk] = *reinterpret_cast<const V8*>(base + 64 * kk);
                            hi[kk] = *reinterpret_cast<const V8*>(base + 2 * D + 64 * kk);
                        }
                    };
                    if constexpr (STAGED) {
                        read(wg.tile + (16 * t + col) * BoundTile<D>::stride + 16 * g);
                    } else {
                        const uint32_t pid = (uint32_t)__shfl((int)id, (int)(16 * t + col));
                        read(static_cast<const char*>(a.bounds) + (uint64_t)(pid == kNoPage ? 0u : pid) * (4ull * D) +
                             16 * g);
                    }
                    f32x4 sum[CT], sum_p[CT], sum_m[CT];
#pragma unroll
                    for (int kk = 0; kk < DK; ++kk) {
                        const V8 hi_abs = bits_as<V8>(bits_as<u32x4>(hi[kk]) & 0x7FFF7FFFu);
                        const V8 lo_abs = bits_as<V8>(bits_as<u32x4>(lo[kk]) & 0x7FFF7FFFu);
#pragma unroll
                        for (int c = 0; c < CT; ++c) {
                            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                            sum[c] = E::mfma(qp[c][kk], hi[kk], kk ? sum[c] : zero);
                            sum_p[c] = E::mfma(qp[c][kk], hi_abs, kk ? sum_p[c] : zero);
                            sum_m[c] = E::mfma(qm[c][kk], lo_abs, kk ? sum_m[c] : zero);
                            sum[c] = E::mfma(qm[c][kk], lo[kk], sum[c]);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        const f32x4 s = sum[c], wp = sum_p[c], wm = sum_m[c];
                        const uint32_t x0 = (ct0 + c) * 16 + 4 * g, row0 = x0 >> a.log2_pad;
                        const uint32_t b = b0 + 16 * t + col;
                        float v[4], w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // a NaN is left out: fmaxf takes its other argument
                            v[i] = (heads[c] >> i) & 1u ? fmaxf(s[i], -__builtin_inff()) : -__builtin_inff();
                            w[i] = wp[i] - wm[i];
                        }
                        if constexpr (ONE_ROW) {
                            float m = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                            float e = max_or_nan(max_or_nan(w[0], w[1]), max_or_nan(w[2], w[3]));
                            if (a.pad >= 8) {
                                m = fmaxf(m, __shfl_xor(m, 16));
                                e = max_or_nan(e, __shfl_xor(e, 16));
                            }
                            if (a.pad >= 16) {
                                m = fmaxf(m, __shfl_xor(m, 32));
                                e = max_or_nan(e, __shfl_xor(e, 32));
                            }
                            if (b < row_nb[c][0]) {
                                settle(m, e, slack[c]);
                                const bool later = a.head_tiles > 1 && ct0 + c > 0;
                                if (x0 == (row0 << a.log2_pad) || (later && g == 0)) {
                                    float* to = a.scores + ((r0 + row0) * a.kv_heads + h) * a.pitch + b;
                                    // a row of several tiles: the highest so far, or a NaN
                                    if (later) m = max_or_nan(m, *to);
                                    *to = m;
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (a.pad == 2 && (i & 1)) continue;
                                float m = a.pad == 2 ? fmaxf(v[i], v[i | 1]) : v[i];
                                const float e = a.pad == 2 ? max_or_nan(w[i], w[i | 1]) : w[i];
                                if (b < row_nb[c][i]) {
                                    settle(m, e, slack[c]);
                                    a.scores[((r0 + ((x0 + i) >> a.log2_pad)) * a.kv_heads + h) * a.pitch + b] = m;
                                }
                            }
                        }
                    }
                }
                // The largest sum of the 64 blocks for the rows of lane l's
                // columns.  Rows that share a lane share the larger one: a bound
                // may be too large.
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    float e = slack[c];
                    for (int o = 1; o < 16; o <<= 1) e = fmaxf(e, __shfl_xor(e, o));
                    const uint32_t x0 = (ct0 + c) * 16 + 4 * g;
#pragma unroll
                    for (uint32_t i = 0; i < (uint32_t)ROWS; ++i) {
                        const uint32_t row = (x0 + i) >> a.log2_pad;
                        const bool first = a.head_tiles > 1 ? g == 0 && i == 0 : x0 + i == (row << a.log2_pad);
                        if (col == 0 && first && row_nb[c][i] > b0) {
                            float* to = a.slack + ((r0 + row) * a.kv_heads + h) * a.chunks + b0 / kWaveBlocks;
                            if (a.head_tiles > 1 && ct0 + c > 0) e = fmaxf(e, *to);
                            *to = e;
                        }
                    }
                }
            }
        }
    }
}

template <class E, int D, int CT, bool ONE_ROW>
__global__ __launch_bounds__(kWave * kScoreWaves, 2) void k_scores(SelectArgs a) {
    const uint32_t wib = uniform(threadIdx.x / kWave);
    score_blocks<E, D, CT, ONE_ROW, false>(a, (uint64_t)blockIdx.z * a.wave_rows, blockIdx.x,
                                           (blockIdx.y * kScoreWaves + wib) * kWaveBlocks * a.span);
}

template <class E, int D, int CT, bool ONE_ROW>
__global__ __launch_bounds__(kWave * kScoreWaves, D == 128 && ONE_ROW ? 3 : 2) void k_scores_shared(SelectArgs a) {
    const uint32_t lane = lane_id(), wib = uniform(threadIdx.x / kWave);
    const uint64_t r0 = ((uint64_t)blockIdx.z * kScoreWaves + wib) * a.wave_rows;
    const uint32_t b_first = blockIdx.y * kWaveBlocks * a.span;
    if constexpr (BoundTile<D>::fits) {
        __shared__ __align__(16) char tile[BoundTile<D>::bytes];
        __shared__ uint32_t seq_sh[kScoreWaves], nb_sh[kScoreWaves], mixed_sh[kScoreWaves];
        int64_t seq = -1;
        uint32_t nb = 0;
        if (lane < a.wave_rows && r0 + lane < a.n_rows) nb = row_blocks(a, r0 + lane, &seq);
        const uint64_t on = ballot(nb > b_first);
        const uint32_t lead = on ? (uint32_t)__builtin_ctzll(on) : 0u;
        const uint32_t wave_seq = lane_value((uint32_t)seq, (int)lead);
        const uint64_t others = ballot(nb > b_first && (uint32_t)seq != wave_seq);
        for (int o = 32; o > 0; o >>= 1) nb = max(nb, (uint32_t)__shfl_xor((int)nb, o));
        if (lane == 0) {
            seq_sh[wib] = wave_seq;
            nb_sh[wib] = on ? nb : 0u;
            mixed_sh[wib] = others != 0;
        }
        __syncthreads();
        Together wg{tile, 0, 0};
        bool mixed = false;
        for (uint32_t w = 0; w < kScoreWaves; ++w) {
            if (!nb_sh[w]) continue;
            mixed = mixed || mixed_sh[w] || (wg.nb && seq_sh[w] != wg.seq);
            wg.seq = seq_sh[w];
            wg.nb = max(wg.nb, nb_sh[w]);
        }
        wg.seq = uniform(wg.seq);
        wg.nb = uniform(wg.nb);
        if (wg.nb == 0) return;
        if (!mixed) {
            score_blocks<E, D, CT, ONE_ROW, true>(a, r0, blockIdx.x, b_first, wg);
            return;
        }
    }
    score_blocks<E, D, CT, ONE_ROW, false>(a, r0, blockIdx.x, b_first);
}

// ---------------------------------------------------------------------------
// The choice.  One workgroup per (row, head).  A thread has consecutive
// blocks, whose keys (scores as ordered integers) lie in LDS, or for rows too
// long for that are made anew from the scores in each pass.  The loops are
// kept rolled: unrolled over keys in registers the kernel took twice as long
// on a short row, most of it instruction fetches.  Bound by its chain of
// barriers and gathers (16 rows of 2,048 blocks by 8 heads: 15 us).
// ---------------------------------------------------------------------------
constexpr uint64_t kLdsKeys = 8192;
constexpr uint64_t kMaxBlocks = 1u << 17;  // near blocks are marked in 16 KiB of LDS

// Ascending order as unsigned numbers; NaN the lowest.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);  // both zeros are one value
    const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return x != x ? 0u : k;
}

__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

constexpr uint32_t kMaxChooseWaves = 16;
constexpr uint32_t kBins = 2048;
constexpr uint32_t kNearList = kWave;  // near blocks that one wave ranks

struct ChooseShared {
    uint32_t hist[kBins];
    uint32_t sums[2][2][kMaxChooseWaves];
    uint32_t digit, left, n_near;
    uint32_t near_block[kNearList], near_key[kNearList];
};

// Sums of two numbers over the workgroup, and over the threads in front.
// `turn` alternates between two rows of LDS, so one barrier per call is
// enough.
struct Sums {
    uint32_t all[2], before[2];
};
__device__ __forceinline__ Sums choose_sums(uint32_t v0, uint32_t v1, ChooseShared& sh, uint32_t& turn) {
    const uint32_t w = threadIdx.x / kWave, waves = blockDim.x / kWave;
    const uint32_t i0 = wave_incl_scan(v0), i1 = wave_incl_scan(v1);
    if (lane_id() == kWave - 1) {
        sh.sums[turn][0][w] = i0;
        sh.sums[turn][1][w] = i1;
    }
    __syncthreads();
    Sums s{{0, 0}, {i0 - v0, i1 - v1}};
    for (uint32_t i = 0; i < waves; ++i) {
        const uint32_t x = sh.sums[turn][0][i], y = sh.sums[turn][1][i];
        if (i < w) {
            s.before[0] += x;
            s.before[1] += y;
        }
        s.all[0] += x;
        s.all[1] += y;
    }
    turn ^= 1;
    return s;
}

// Maxima of two numbers over the workgroup.
__device__ __forceinline__ void choose_max2(uint32_t& v0, uint32_t& v1, ChooseShared& sh, uint32_t& turn) {
    for (int o = 32; o > 0; o >>= 1) {
        v0 = max(v0, (uint32_t)__shfl_xor((int)v0, o));
        v1 = max(v1, (uint32_t)__shfl_xor((int)v1, o));
    }
    if (lane_id() == 0) {
        sh.sums[turn][0][threadIdx.x / kWave] = v0;
        sh.sums[turn][1][threadIdx.x / kWave] = v1;
    }
    __syncthreads();
    for (uint32_t i = 0; i < blockDim.x / kWave; ++i) {
        v0 = max(v0, sh.sums[turn][0][i]);
        v1 = max(v1, sh.sums[turn][1][i]);
    }
    turn ^= 1;
}

// One pass over the bins that each() calls back with: the bin of the left-th
// largest; `left` becomes its rank within the bin.
template <class Each>
__device__ __forceinline__ uint32_t find_bin(uint32_t n_bins, uint32_t& left, ChooseShared& sh, uint32_t& turn,
                                             Each each) {
    for (uint32_t i = threadIdx.x; i < n_bins; i += blockDim.x) sh.hist[i] = 0;
    __syncthreads();
    each([&](uint32_t bin) __attribute__((always_inline)) { atomicAdd(&sh.hist[bin], 1u); });
    __syncthreads();
    // thread t: `per` bins from the top downwards
    const uint32_t per = (n_bins + blockDim.x - 1) / blockDim.x;
    const uint32_t top = n_bins - 1 - min(threadIdx.x * per, n_bins - 1);
    const uint32_t mine = threadIdx.x * per < n_bins ? min(per, n_bins - threadIdx.x * per) : 0u;
    uint32_t sum = 0;
    for (uint32_t j = 0; j < mine; ++j) sum += sh.hist[top - j];
    const Sums s = choose_sums(sum, 0u, sh, turn);
    uint32_t before = s.before[0];
    if (before < left && before + sum >= left) {
        uint32_t j = 0;
        while (before + sh.hist[top - j] < left) before += sh.hist[top - j++];
        sh.digit = top - j;
        sh.left = left - before;
    }
    __syncthreads();
    left = sh.left;
    return sh.digit;
}

// The want-th largest (want >= 1) of the keys for which each() calls back;
// *above: how many are larger.  lo, hi: the smallest and the largest of them.
template <class Each>
__device__ __forceinline__ uint32_t nth_largest(uint32_t want, uint32_t lo, uint32_t hi, ChooseShared& sh,
                                                uint32_t& turn, uint32_t* above, Each each) {
    *above = 0;
    if (lo == hi) return lo;
    const uint32_t lz = (uint32_t)__builtin_clz(hi - lo);
    uint32_t prefix = 0, left = want;
    for (int shift = 24; shift > -8; shift -= 8) {
        if (shift + 8 <= (int)lz) break;  // the bits below are zeros of the shift
        const uint32_t digit = find_bin(256, left, sh, turn, [&](auto f) __attribute__((always_inline)) {
            each([&](uint32_t key) __attribute__((always_inline)) {
                const uint32_t k = (key - lo) << lz;
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) f((k >> shift) & 255u);
            });
        });
        prefix |= digit << shift;
    }
    *above = want - left;
    return lo + (prefix >> lz);
}

// max(y lo, y hi), or a NaN of either.
__device__ __forceinline__ double larger_product(double y, double lo, double hi) {
    const double to_lo = y * lo, to_hi = y * hi;
    return to_lo != to_lo || to_lo > to_hi ? to_lo : to_hi;
}

// One wave: the score of page b of (row r, head h) summed in 64 bits, as a
// key.  Sixteen lanes take a query head, eight dims each at a time.
template <class E, int D>
__device__ __forceinline__ uint32_t exact_key(const SelectArgs& a, uint64_t r, uint32_t h, const uint16_t* bounds) {
    const uint32_t lane = lane_id(), part = lane & 15u;
    float best = -__builtin_inff();
    for (uint32_t j0 = 0; j0 < a.group; j0 += 4) {
        const uint32_t j = j0 + (lane >> 4);
        const uint16_t* q =
            static_cast<const uint16_t*>(a.q) + (int64_t)r * a.q_row + (int64_t)(h * a.group + min(j, a.group - 1)) * a.q_head;
        double s = 0.0;
#pragma unroll
        for (int d = 0; d < D; d += 128) {
            if (d + 8 * part < (uint32_t)D) {
                const u32x4 x = load_eight(q + d + 8 * part);
                const u32x4 lo = *reinterpret_cast<const u32x4*>(bounds + d + 8 * part);
                const u32x4 hi = *reinterpret_cast<const u32x4*>(bounds + D + d + 8 * part);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int sh = 16 * (e & 1);
                    const double y = (double)E::from_bits(x[e >> 1] >> sh);
                    s += larger_product(y, (double)E::from_bits(lo[e >> 1] >> sh), (double)E::from_bits(hi[e >> 1] >> sh));
                }
            }
        }
        for (int o = 8; o > 0; o >>= 1) s += __shfl_xor(s, o);
        best = fmaxf(best, (float)s);  // a head listed twice at the end changes no maximum
    }
    best = fmaxf(best, __shfl_xor(best, 16));
    best = fmaxf(best, __shfl_xor(best, 32));
    return order_of(best);
}

// One thread: the same, for the rare pages of which a 32-bit sum says nothing.
// Rolled up, so that it takes few registers.
template <class E, int D>
__device__ __forceinline__ uint32_t lone_key(const SelectArgs& a, uint64_t r, uint32_t h, const uint16_t* bounds) {
    float best = -__builtin_inff();
#pragma unroll 1
    for (uint32_t j = 0; j < a.group; ++j) {
        const uint16_t* q =
            static_cast<const uint16_t*>(a.q) + (int64_t)r * a.q_row + (int64_t)(h * a.group + j) * a.q_head;
        double s = 0.0;
#pragma unroll 2
        for (int d = 0; d < D; ++d) {
            const double y = (double)E::from_bits(q[d]);
            s += larger_product(y, (double)E::from_bits(bounds[d]), (double)E::from_bits(bounds[D + d]));
        }
        best = fmaxf(best, (float)s);
    }
    return order_of(best);
}

// Whether a head of (row r, key/value head h) has a number that is not zero,
// and no NaN.  A wave takes a head at a time.
template <class E, int D>
__device__ __forceinline__ bool any_number(const SelectArgs& a, uint64_t r, uint32_t h, ChooseShared& sh,
                                           uint32_t& turn) {
    uint32_t any = 0, zero = 0;
#pragma unroll 1
    for (uint32_t j = threadIdx.x / kWave; j < a.group; j += blockDim.x / kWave) {
        const uint16_t* q =
            static_cast<const uint16_t*>(a.q) + (int64_t)r * a.q_row + (int64_t)(h * a.group + j) * a.q_head;
        uint32_t top = 0;
#pragma unroll 1
        for (uint32_t d = lane_id(); d < (uint32_t)D; d += kWave) top = max(top, q[d] & 0x7FFFu);
        if (ballot(top != 0) != 0 && ballot(top > E::kExponent) == 0) any = 1;
    }
    choose_max2(any, zero, sh, turn);
    return any != 0;
}

template <class E, int D, bool KEYS>
__device__ __forceinline__ void choose_blocks(const SelectArgs& a, ChooseShared& sh, uint32_t* smem) {
    uint32_t* const near_words = smem;  // blocks to be summed in 64 bits
    uint32_t* const keys = smem + (a.blocks + 31) / 32;
    const uint64_t rh = blockIdx.x;
    const uint64_t r = rh / a.kv_heads;
    const uint32_t h = (uint32_t)(rh % a.kv_heads);
    const uint32_t tid = threadIdx.x, nt = blockDim.x, lane = lane_id(), wib = tid / kWave;
    int32_t* out = a.out + rh * a.n_out;
    float* scores = a.scores + rh * a.pitch;
    // the first scores and bounds are on their way while the row's length is
    // (their addresses lie inside the workspace whatever it is)
    float first = 0.f, slack = 0.f;
    if (KEYS && tid < a.blocks) first = scores[tid];
    for (uint32_t c = tid; c < a.chunks; c += nt) slack = a.slack[rh * a.chunks + c];
    int64_t seq;
    const uint32_t nb = row_blocks(a, r, &seq);
    if (tid == 0) {
        const int64_t len = a.lens[r];
        if (seq < 0 || (uint64_t)seq >= a.n_seqs || len < 0 || (uint64_t)len > a.blocks * a.page_tokens)
            atomicCAS(a.err, 0u, (uint32_t)kErrRange);
    }
    if (nb <= a.n_out) {
        for (uint32_t i = tid; i < a.n_out; i += nt) out[i] = i < nb ? (int32_t)i : -1;
        return;
    }
    const uint32_t f_end = a.keep_first, l_begin = nb - a.keep_last;  // keep_first + keep_last <= n_out < nb
    // this thread's blocks [at, end)
    const uint32_t per = (nb + nt - 1) / nt;
    const uint32_t at = min(tid * per, nb), end = min(at + per, nb);
    if (KEYS) {
        if (tid < nb) keys[tid] = order_of(first);
        for (uint32_t b = tid + nt; b < nb; b += nt) keys[b] = order_of(scores[b]);
    }
    for (uint32_t w = tid; w < (nb + 31) / 32; w += nt) near_words[w] = 0;
    auto key_of = [&](uint32_t b) __attribute__((always_inline)) { return KEYS ? keys[b] : order_of(scores[b]); };
    auto is_near = [&](uint32_t b) __attribute__((always_inline)) {
        return ((near_words[b >> 5] >> (b & 31)) & 1u) != 0;
    };
    uint32_t turn = 0;
    const uint32_t want = a.n_out - a.keep_first - a.keep_last;
    // Chosen: keys above `cut`, and the first `ties` equal to it.  Where pages
    // were summed again, `near` ones among them are those whose mark is left,
    // or (many of them) those that `cut` and `ties` say, and the others those
    // above `over`.
    uint32_t cut = 0xFFFFFFFFu, ties = 0, over = 0xFFFFFFFFu;
    bool marked = false, ranked = false;
    if (want > 0) {
        if (a.chunks <= nt) {
            if (tid >= (nb + kWaveBlocks - 1) / kWaveBlocks) slack = 0.f;
        } else {
            slack = 0.f;
            for (uint32_t c = tid; c < (nb + kWaveBlocks - 1) / kWaveBlocks; c += nt)
                slack = fmaxf(slack, a.slack[rh * a.chunks + c]);
        }
        if (tid == 0) sh.n_near = 0;
        uint32_t slack_bits = __float_as_uint(slack), zero = 0;
        choose_max2(slack_bits, zero, sh, turn);  // (and the keys are in LDS)
        slack = sum_error(D) * __uint_as_float(slack_bits);
        // (rows of zeros or NaNs, as a batch may be padded with, have no products)
        if (slack_bits != 0 || any_number<E, D>(a, r, h, sh, turn)) slack += sum_underflow(D);
        const uint32_t own_at = max(at, f_end), own_end = min(end, l_begin);
        const int64_t* table = a.table + ((uint64_t)seq * a.kv_heads + h) * a.blocks;
        const uint16_t* bounds = static_cast<const uint16_t*>(a.bounds);
        auto bounds_of = [&](uint32_t b) __attribute__((always_inline)) {
            const uint32_t id = page_id(table[b], (uint32_t)a.n_slots);
            return bounds + (uint64_t)(id == kNoPage ? 0u : id) * (2ull * D);
        };
        auto own = [&](auto f) __attribute__((always_inline)) {
#pragma unroll 1
            for (uint32_t b = own_at; b < own_end; ++b) f(b, key_of(b));
        };
        auto own_keys = [&](auto f) __attribute__((always_inline)) {
            own([&](uint32_t, uint32_t k) __attribute__((always_inline)) { f(k); });
        };
        uint32_t not_lo, hi;
        auto range_of = [&](auto each) __attribute__((always_inline)) {
            not_lo = hi = 0;
            each([&](uint32_t k) __attribute__((always_inline)) {
                not_lo = max(not_lo, ~k);
                hi = max(hi, k);
            });
            choose_max2(not_lo, hi, sh, turn);
        };
        range_of(own_keys);
        // Pages with key 0, a NaN: nothing is known of them yet.  A thread sums
        // its own in 64 bits if no thread has more than two; else all pages
        // are near.
        bool unbounded = false;
        if (not_lo == 0xFFFFFFFFu) {
            uint32_t mine = 0, zero2 = 0;
            own_keys([&](uint32_t k) __attribute__((always_inline)) { mine += k == 0; });
            choose_max2(mine, zero2, sh, turn);
            unbounded = mine > 2;
            if (!unbounded) {
                own([&](uint32_t b, uint32_t k) __attribute__((always_inline)) {
                    if (k != 0) return;
                    k = lone_key<E, D>(a, r, h, bounds_of(b));
                    if (KEYS)
                        keys[b] = k;
                    else
                        scores[b] = value_of(k);
                });
                range_of(own_keys);
            }
        }
        const uint32_t lo = ~not_lo;
        // One pass: the bin of kBins between lo and hi that holds the want-th
        // largest sum.  Keys of scores that lie close together differ in
        // their low bits only, so bins are counted from lo.
        const uint32_t bits = 32 - (uint32_t)__builtin_clz((hi - lo) | 1u), drop = bits > 11 ? bits - 11 : 0u;
        uint32_t left = want, above;
        const uint32_t bin = find_bin(kBins, left, sh, turn, [&](auto f) __attribute__((always_inline)) {
            own_keys([&](uint32_t k) __attribute__((always_inline)) { f((k - lo) >> drop); });
        });
        const float t_lo = value_of(lo + (bin << drop));
        const float t_hi = value_of(min(hi, lo + (bin << drop) + ((1u << drop) - 1)));
        if (slack > 0.f || unbounded) {
            // Every true score is within `slack` of its sum, so the want-th
            // largest true one lies between t_lo and t_hi widened by slack;
            // pages that are further than two of them outside are decided
            // (a third covers the roundings of these bounds and of the score).
            const uint32_t near_lo = unbounded ? 0u : order_of(t_lo - 3.f * slack);
            const uint32_t near_hi = unbounded ? 0xFFFFFFFFu : order_of(t_hi + 3.f * slack);
            uint32_t n_above = 0, n_near = 0;
            own([&](uint32_t b, uint32_t k) __attribute__((always_inline)) {
                if (k > near_hi) {
                    ++n_above;
                } else if (k >= near_lo) {
                    atomicOr(&near_words[b >> 5], 1u << (b & 31));
                    const uint32_t i = atomicAdd(&sh.n_near, 1u);
                    if (i < kNearList) sh.near_block[i] = b;
                    ++n_near;
                }
            });
            const Sums n = choose_sums(n_above, n_near, sh, turn);
            over = near_hi;
            if (n.all[0] + n.all[1] == want) {
                cut = near_lo - 1;  // the near ones are exactly those still wanted
            } else {
                const uint32_t rest = want - n.all[0];
                marked = true;
                if (n.all[1] <= kNearList) {
                    // the usual case: a few, in a list, ranked by one wave
                    for (uint32_t i = wib; i < n.all[1]; i += nt / kWave) {
                        const uint32_t k = exact_key<E, D>(a, r, h, bounds_of(uniform(sh.near_block[i])));
                        if (lane == 0) sh.near_key[i] = k;
                    }
                    __syncthreads();
                    if (wib == 0) {
                        const uint32_t b = lane < n.all[1] ? sh.near_block[lane] : 0u;
                        const uint32_t k = lane < n.all[1] ? sh.near_key[lane] : 0u;
                        uint32_t better = 0;
                        for (uint32_t i = 0; i < n.all[1]; ++i) {
                            const uint32_t ki = lane_value(k, (int)i), bi = lane_value(b, (int)i);
                            better += ki > k || (ki == k && bi < b);
                        }
                        if (lane < n.all[1] && better >= rest) atomicAnd(&near_words[b >> 5], ~(1u << (b & 31)));
                    }
                    __syncthreads();
                    ranked = true;
                } else {
                    for (uint32_t w = wib; w < (nb + 31) / 32; w += nt / kWave) {
                        for (uint32_t m = uniform(near_words[w]); m; m &= m - 1) {
                            const uint32_t b = 32 * w + (uint32_t)__builtin_ctz(m);
                            const uint32_t k = exact_key<E, D>(a, r, h, bounds_of(b));
                            if (lane == 0) {
                                if (KEYS)
                                    keys[b] = k;
                                else
                                    scores[b] = value_of(k);
                            }
                        }
                    }
                    __threadfence_block();
                    __syncthreads();
                    auto near_keys = [&](auto f) __attribute__((always_inline)) {
                        own([&](uint32_t b, uint32_t k) __attribute__((always_inline)) {
                            if (is_near(b)) f(k);
                        });
                    };
                    range_of(near_keys);
                    cut = nth_largest(rest, ~not_lo, hi, sh, turn, &above, near_keys);
                    ties = rest - above;
                }
            }
        } else {
            // no slack (a row of zeros or NaNs): the sums, all alike
            cut = nth_largest(want, lo, hi, sh, turn, &above, own_keys);
            ties = want - above;
        }
    }
    // which of this thread's blocks are in, ties in order of their block
    auto state_of = [&](uint32_t b) __attribute__((always_inline)) -> uint32_t {  // 0 out, 1 in, 2 tie
        if (b < f_end || b >= l_begin) return 1u;
        const uint32_t k = key_of(b);
        if (marked) {
            const bool near = is_near(b);
            if (ranked) return near || k > over ? 1u : 0u;
            if (!near) return k > over ? 1u : 0u;
        }
        return k > cut ? 1u : (k == cut ? 2u : 0u);
    };
    uint32_t n_ties = 0, n_in = 0;
#pragma unroll 1
    for (uint32_t b = at; b < end; ++b) {
        const uint32_t s = state_of(b);
        n_in += s == 1u;
        n_ties += s == 2u;
    }
    const Sums n = choose_sums(n_in, n_ties, sh, turn);
    // rank of this thread's first block: those in front of it, and the ties
    // in front of it as far as they are taken
    uint32_t tie_rank = n.before[1], rank = n.before[0] + min(tie_rank, ties);
    const uint32_t total = n.all[0] + min(n.all[1], ties);
#pragma unroll 1
    for (uint32_t b = at; b < end; ++b) {
        const uint32_t s = state_of(b);
        if (s == 1u || (s == 2u && tie_rank++ < ties)) {
            if (rank < a.n_out) out[rank] = (int32_t)b;
            ++rank;
        }
    }
    for (uint32_t i = total + tid; i < a.n_out; i += nt) out[i] = -1;
}

// 64 registers for pages of up to 128 dims, so that eight waves fit a SIMD: the
// 64-bit sums read from everywhere and wait (512 rows of 4,096 blocks on 8
// heads: 86 us, 124 us with the 94 registers the compiler takes by itself).
// 256 dims would spill.
template <class E, int D, bool KEYS>
__global__ __launch_bounds__(1024, D <= 128 ? 8 : 4) void k_choose(SelectArgs a) {
    __shared__ ChooseShared sh;
    extern __shared__ __align__(16) uint32_t smem[];
    choose_blocks<E, D, KEYS>(a, sh, smem);
}

// Both in one launch, for rows with pages of their own in tables of at most
// kOneLaunchBlocks blocks: the workgroup of a (row, head) scores its blocks,
// 64 a wave at a time, and chooses among them.  (A row of 256 blocks and 8
// heads of 128 dims: 14 us, as much as the two launches, 8 and 6, without the
// 4 to 5 us that the second one costs the host.)
constexpr uint32_t kSelectWaves = 8;
constexpr uint64_t kOneLaunchBlocks = 1024;

template <class E, int D>
__global__ __launch_bounds__(kWave * kSelectWaves) void k_select(SelectArgs a) {
    __shared__ ChooseShared sh;
    extern __shared__ __align__(16) uint32_t smem[];
    const uint64_t r = blockIdx.x / a.kv_heads;
    const uint32_t h = blockIdx.x % a.kv_heads;
#pragma unroll 1
    for (uint32_t b = uniform(threadIdx.x / kWave) * kWaveBlocks; b < a.blocks; b += kSelectWaves * kWaveBlocks)
        score_blocks<E, D, 1, true, false>(a, r, h, b);
    __threadfence_block();
    __syncthreads();
    choose_blocks<E, D, true>(a, sh, smem);
}

}  // namespace ibp

using namespace ibp;

extern "C" {

ibp_status ibp_page_bounds(const ibp_pages* k, uint32_t dtype, uint32_t head_dim, const int64_t* ids,
                           const int32_t* tokens, uint64_t n, void* bounds, hipStream_t stream) {
    if (!k || !k->meta) return IBP_ERR_INVALID_ARG;
    if (n == 0) return IBP_OK;
    ibp_meta_t h = k->meta;
    DeviceGuard guard(h->device);
    if (!guard.ok) return IBP_ERR_DEVICE;
    if (dtype > IBP_FP16 || n > kMaxPoolSlots) return IBP_ERR_INVALID_ARG;
    Pool pool;
    ibp_status st = make_pool(k, h->device, &pool);
    if (st != IBP_OK) return st;
    const uint64_t L = h->params.tensor_bytes;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return IBP_ERR_UNSUPPORTED;
    if (L < 2048 || L > kMaxPageBytes || (L & (L - 1)) != 0) return IBP_ERR_UNSUPPORTED;
    if (!device_only(ids, h->device) || !device_only(bounds, h->device) ||
        (tokens && !device_only(tokens, h->device)) || reinterpret_cast<uintptr_t>(bounds) % 16)
        return IBP_ERR_INVALID_ARG;
    const uint32_t row_words = head_dim / 2;
    const uint64_t tab = 4ull * page_tab_words(pool.Mw, pool.runs);
    auto launch = [&](auto e, auto nv) {
        using E = decltype(e);
        constexpr int NV = decltype(nv)::value;
        const uint64_t stage = 4ull * kBoundWaves * page_stage_words<NV>();
        // tables that leave no room for a second workgroup on a compute unit
        // (and none in the LDS that a launch has by itself) stay in device memory
        const bool lds = pool.Mw < 4 || tab + stage <= kMaxLdsPerBlock;
        const uint64_t waves = std::min<uint64_t>(n, 4ull * kBoundWaves * 4 * h->cu_count);
        const dim3 grid((uint32_t)((waves + kBoundWaves - 1) / kBoundWaves));
        if (lds)
            hipLaunchKernelGGL((k_page_bounds<E, NV, true>), grid, dim3(kWave * kBoundWaves), (uint32_t)(tab + stage),
                               stream, pool, row_words, ids, tokens, n, static_cast<uint32_t*>(bounds));
        else
            hipLaunchKernelGGL((k_page_bounds<E, NV, false>), grid, dim3(kWave * kBoundWaves), (uint32_t)stage, stream,
                               pool, row_words, ids, tokens, n, static_cast<uint32_t*>(bounds));
        return hipGetLastError();
    };
    auto by_size = [&](auto e) {
        if (L == 2048) return launch(e, std::integral_constant<int, 2>{});
        if (L == 4096) return launch(e, std::integral_constant<int, 4>{});
        return launch(e, std::integral_constant<int, 8>{});
    };
    return from_hip(dtype == IBP_BF16 ? by_size(Bf16{}) : by_size(Fp16{}));
}

static uint64_t select_chunks(const ibp_attention* a) { return (a->table_blocks + kWaveBlocks - 1) / kWaveBlocks; }
static uint64_t select_pitch(const ibp_attention* a) { return (a->table_blocks + 3) & ~3ull; }

uint64_t ibp_select_pages_workspace(const ibp_attention* a) {
    if (!a) return 0;
    return 4 * a->n_rows * a->n_kv_heads * (select_pitch(a) + select_chunks(a));
}

ibp_status ibp_select_pages(ibp_meta_t h, const ibp_attention* a, const void* q, const void* bounds, uint64_t n_slots,
                            const int64_t* k_table, const int32_t* lens, const int32_t* row_seq, uint32_t keep_first,
                            uint32_t keep_last, int32_t* blocks, uint32_t n_blocks, void* workspace,
                            uint64_t workspace_bytes, hipStream_t stream) {
    if (!h || !a) return IBP_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (!guard.ok) return IBP_ERR_DEVICE;
    ibp_status st = check_attention(a);
    if (st != IBP_OK) return st;
    if (a->n_rows == 0) return IBP_OK;
    if (n_blocks == 0 || (uint64_t)keep_first + keep_last > n_blocks || n_slots == 0 || n_slots > kMaxPoolSlots)
        return IBP_ERR_INVALID_ARG;
    if (!row_seq && a->n_rows > a->n_seqs) return IBP_ERR_INVALID_ARG;
    if (a->table_blocks > kMaxBlocks) return IBP_ERR_UNSUPPORTED;
    for (const void* p : {q, bounds, (const void*)k_table, (const void*)lens, (const void*)blocks,
                          (const void*)workspace})
        if (!device_only(p, h->device)) return IBP_ERR_INVALID_ARG;
    if (row_seq && !device_only(row_seq, h->device)) return IBP_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(bounds) % 16 || reinterpret_cast<uintptr_t>(workspace) % 16 ||
        workspace_bytes < ibp_select_pages_workspace(a))
        return IBP_ERR_INVALID_ARG;
    SelectArgs s{};
    s.q = q;
    s.bounds = bounds;
    s.table = k_table;
    s.lens = lens;
    s.row_seq = row_seq;
    s.blocks = a->table_blocks;
    s.pitch = select_pitch(a);
    s.chunks = select_chunks(a);
    s.scores = static_cast<float*>(workspace);
    s.slack = s.scores + a->n_rows * a->n_kv_heads * s.pitch;
    s.out = blocks;
    s.err = h->d_err;
    s.n_rows = a->n_rows;
    s.n_seqs = a->n_seqs;
    s.n_slots = n_slots;
    s.q_row = a->q_row_stride;
    s.q_head = a->q_head_stride;
    s.kv_heads = a->n_kv_heads;
    s.group = a->n_q_heads / a->n_kv_heads;
    s.page_tokens = a->page_tokens;
    s.keep_first = keep_first;
    s.keep_last = keep_last;
    s.n_out = n_blocks;
    // Many rows per sequence share the pages' bounds, two tiles of rows a wave
    // (one of 256 dims, for the registers); few rows take a wave each, whose
    // lanes then always hold columns of one row.
    const bool shared = a->n_rows >= 4 * a->n_seqs && s.group <= 16;
    s.pad = shared ? 1 : 4;
    while (s.pad < s.group && s.pad < 16) s.pad *= 2;
    if (s.group > 16) s.pad = (s.group + 15) / 16 * 16;
    s.log2_pad = s.pad > 16 ? 31 : (uint32_t)__builtin_ctz(s.pad);
    s.rows_per_tile = s.pad < 16 ? 16 / s.pad : 1;
    s.head_tiles = s.pad > 16 ? s.pad / 16 : 1;
    const uint32_t ct = shared && a->head_dim <= 128 ? 2 : 1;
    s.wave_rows = shared ? ct * s.rows_per_tile : 1;
    // A wave that shares pays for its queries once: as many blocks as give one
    // round of workgroups, three on a compute unit of 256.  (512 rows by 4,096
    // blocks by 8 heads of 128 dims, read without LDS: 136 us in 768 workgroups,
    // 162 in 1,024, 156 in 2,048.)
    const uint64_t row_groups = (a->n_rows + ct * s.rows_per_tile * kScoreWaves - 1) / (ct * s.rows_per_tile * kScoreWaves);
    const uint64_t all_chunks = row_groups * a->n_kv_heads * select_chunks(a);
    s.span = shared ? (uint32_t)std::min<uint64_t>(std::max<uint64_t>(1, (all_chunks + 767) / 768), 64) : 1;
    const uint64_t per_wg_rows = (uint64_t)s.wave_rows * (shared ? kScoreWaves : 1);
    const uint64_t groups = (a->n_rows + per_wg_rows - 1) / per_wg_rows;
    const bool scored = a->table_blocks > n_blocks && n_blocks > keep_first + keep_last;
    const bool one_launch = scored && !shared && a->table_blocks <= kOneLaunchBlocks;
    const bool keys = a->table_blocks <= kLdsKeys;
    // waves that choose: eight blocks per thread
    uint32_t waves = kMaxChooseWaves;
    if (one_launch)
        waves = kSelectWaves;
    else if (keys)
        waves = (uint32_t)std::min<uint64_t>(waves, std::max<uint64_t>(4, (a->table_blocks + 8 * kWave - 1) / (8 * kWave)));
    if (a->n_rows * a->n_kv_heads > max_workgroups(kWave * waves) || (scored && !one_launch && groups > 65535))
        return IBP_ERR_UNSUPPORTED;
    auto launch = [&](auto e, auto dc) {
        using E = decltype(e);
        constexpr int D = decltype(dc)::value;
        const dim3 grid((uint32_t)(a->n_rows * a->n_kv_heads));
        const uint32_t marks = (uint32_t)(4 * ((a->table_blocks + 31) / 32));
        if (one_launch) {
            hipLaunchKernelGGL((k_select<E, D>), grid, dim3(kWave * waves),
                               marks + (uint32_t)(4 * a->table_blocks), stream, s);
            return hipGetLastError();
        }
        if (scored) {  // no row can have more pages than it may read otherwise
            const uint64_t per_wg = (uint64_t)(shared ? 1 : kScoreWaves) * kWaveBlocks * s.span;
            const dim3 tiles(a->n_kv_heads, (uint32_t)((a->table_blocks + per_wg - 1) / per_wg), (uint32_t)groups);
            auto by_rows = [&](auto ct_tiles, dim3 g) {
                constexpr int CT = decltype(ct_tiles)::value;
                if (s.pad >= 4)
                    hipLaunchKernelGGL((k_scores_shared<E, D, CT, true>), g, dim3(kWave * kScoreWaves), 0, stream, s);
                else
                    hipLaunchKernelGGL((k_scores_shared<E, D, CT, false>), g, dim3(kWave * kScoreWaves), 0, stream, s);
            };
            if (shared)
                by_rows(std::integral_constant<int, D == 256 ? 1 : 2>{}, tiles);
            else
                hipLaunchKernelGGL((k_scores<E, D, 1, true>), tiles, dim3(kWave * kScoreWaves), 0, stream, s);
            const hipError_t err = hipGetLastError();
            if (err != hipSuccess) return err;
        }
        if (keys)
            hipLaunchKernelGGL((k_choose<E, D, true>), grid, dim3(kWave * waves),
                               marks + (uint32_t)(4 * a->table_blocks), stream, s);
        else
            hipLaunchKernelGGL((k_choose<E, D, false>), grid, dim3(kWave * waves), marks, stream, s);
        return hipGetLastError();
    };
    auto by_dim = [&](auto e) {
        if (a->head_dim == 64) return launch(e, std::integral_constant<int, 64>{});
        if (a->head_dim == 128) return launch(e, std::integral_constant<int, 128>{});
        return launch(e, std::integral_constant<int, 256>{});
    };
    return from_hip(a->dtype == IBP_BF16 ? by_dim(Bf16{}) : by_dim(Fp16{}));
}

}  // extern "C"
