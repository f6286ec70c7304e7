// ibp_select.hip -- which pages of a cache a query reads: per-page bounds of
// the keys, and the choice of the pages with the highest bound on the score.
//
// For a page with lo[d] <= k[d] <= hi[d], q.k <= sum over d of
// max(q[d] lo[d], q[d] hi[d]) = sum of max(q,0) hi + min(q,0) lo: a product
// of the vector (q+, q-) with (hi, lo), twice head_dim long.  Neighbouring
// scores decide which pages are read, so the definition sums in 64 bits and
// rounds once; the kernels get there in two steps:
//   1. k_scores multiplies on the matrix cores in 32 bits, and a second
//      product of the absolute values bounds how far each sum can be off;
//   2. k_choose finds the n-th largest of these, and sums again in 64 bits
//      only the pages whose distance from it is within that bound, usually
//      none or one.
// The result is the one that 64-bit sums of all pages give.
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
// the lanes of one dim group are joined at the end.
// ---------------------------------------------------------------------------
constexpr uint32_t kBoundWaves = 4;

__device__ __forceinline__ void join_bounds(float& lo, float& hi, float x_lo, float x_hi) {
    // comparisons with NaN are false: a NaN on either side is kept
    lo = (x_lo < lo || x_lo != x_lo) ? x_lo : lo;
    hi = (x_hi > hi || x_hi != x_hi) ? x_hi : hi;
}

template <class E, int NV, bool TAB_LDS>
__global__ __launch_bounds__(kWave * kBoundWaves) void k_page_bounds(Pool pool, uint32_t row_words,
                                                                     const int64_t* __restrict__ ids,
                                                                     const int32_t* __restrict__ tokens, uint64_t n,
                                                                     uint32_t* __restrict__ bounds) {
    extern __shared__ uint32_t smem[];
    const uint32_t lane = lane_id(), wib = uniform(threadIdx.x / kWave);
    const uint32_t tab_words = TAB_LDS ? page_tab_words(pool.Mw, pool.runs) : 0u;
    if (TAB_LDS) {
        stage_page_tables(pool, smem);
        __syncthreads();
    }
    const PageTab tab = TAB_LDS ? page_tab(pool, smem) : page_tab_global(pool);
    uint32_t* stage = smem + tab_words + wib * page_stage_words<NV>();
    const uint32_t row_lanes = row_words / 4;  // lanes that one token takes
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
        u32x4 st[NV];
        load_page<NV>(st, pool.slots, id);
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            lo[j] = __builtin_inff();
            hi[j] = -__builtin_inff();
        }
        auto take = [&](uint32_t w, const u32x4& x) __attribute__((always_inline)) {
            if ((int32_t)(w / row_words) >= held) return;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y = E::from_bits(x[j >> 1] >> (16 * (j & 1)));
                join_bounds(lo[j], hi[j], y, y);
            }
        };
        if (uniform(page_bit(pool.bitmask, id))) {
            if (!rebuild_page<NV>(st, pool, tab, stage, take)) latch_error(pool.err, kErrCorrupt);
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
// Scores.  One wave takes 16 * kPageTiles blocks of one (row tile, head): the
// bounds of 16 pages are the A operand (lane l: page l % 16, eight dims), 16
// columns of (row, query head) the B operand, so D holds the scores of 16
// pages by 16 columns.  A row tile is 16 / group rows (one, and several column
// tiles, for groups of more than 16 heads).
// ---------------------------------------------------------------------------
struct SelectArgs {
    const void* q;
    const void* bounds;
    const int64_t* table;
    const int32_t* lens;
    const int32_t* row_seq;
    float* scores;   // [n_rows][kv heads][blocks]
    float* slack;    // [n_rows][kv heads][chunks]: bound on the error of a chunk's scores
    int32_t* out;
    uint32_t* err;
    uint64_t n_rows, n_seqs, n_slots, blocks, chunks;
    int64_t q_row, q_head;
    uint32_t kv_heads, group, page_tokens, keep_first, keep_last, n_out;
    uint32_t rows_per_tile, col_tiles;
    uint32_t vec;    // q rows may be read as 16-byte vectors
};

constexpr uint32_t kScoreWaves = 4;
constexpr uint32_t kPageTiles = 4;  // tiles of 16 blocks per wave
constexpr uint32_t kScoreChunk = kScoreWaves * kPageTiles * 16;

// Error of a 32-bit sum of 2 * head_dim products, relative to the sum of
// their absolute values: head_dim <= 256, so at most 512 additions of 2^-24
// each, 2^-15; the products themselves are exact.
constexpr float kSumError = 1.0f / 32768.0f;

// Blocks of row r, and whether its sequence and length are valid.
__device__ __forceinline__ uint64_t row_blocks(const SelectArgs& a, uint64_t r, int64_t* seq) {
    *seq = a.row_seq ? a.row_seq[r] : (int64_t)r;
    const int64_t len = a.lens[r];
    if (*seq < 0 || (uint64_t)*seq >= a.n_seqs || len < 0) return 0;
    const uint64_t nb = ((uint64_t)len + a.page_tokens - 1) / a.page_tokens;
    return nb < a.blocks ? nb : a.blocks;
}

template <class E, int D>
__global__ __launch_bounds__(kWave * kScoreWaves) void k_scores(SelectArgs a) {
    using V8 = typename E::V8;
    const uint32_t lane = lane_id(), wib = uniform(threadIdx.x / kWave);
    const uint32_t col = lane & 15u, g = lane >> 4;
    const uint32_t h = blockIdx.y;
    const uint64_t r0 = (uint64_t)blockIdx.z * a.rows_per_tile;
    const uint64_t b0 = (uint64_t)blockIdx.x * kScoreChunk + wib * (kPageTiles * 16);
    // the tile's rows that have not been done yet, one sequence after another
    int64_t row_seq = -1;
    uint64_t row_nb = 0;
    if (lane < a.rows_per_tile && r0 + lane < a.n_rows) row_nb = row_blocks(a, r0 + lane, &row_seq);
    uint64_t todo = ballot(row_nb > b0);
    const bool one_tile = a.col_tiles == 1;
    while (todo) {
        const uint32_t lead = (uint32_t)__builtin_ctzll(todo);
        const int64_t seq = (int64_t)(((uint64_t)lane_value((uint32_t)((uint64_t)row_seq >> 32), lead) << 32) |
                                      lane_value((uint32_t)row_seq, lead));
        const uint64_t mine = todo & ballot(row_seq == seq && row_nb > b0);
        todo &= ~mine;
        uint64_t nb = 0;
        for (uint64_t m = mine; m; m &= m - 1) {
            const uint32_t l = (uint32_t)__builtin_ctzll(m);
            nb = max(nb, (uint64_t)lane_value((uint32_t)row_nb, l));
        }
        const int64_t* table = a.table + ((uint64_t)seq * a.kv_heads + h) * a.blocks;
        for (uint32_t t = 0; t < kPageTiles; ++t) {
            const uint64_t bt = b0 + 16 * t;
            if (bt >= nb) break;
            const uint64_t bl = bt + col;
            uint32_t id = kNoPage;
            if (bl < nb) {
                id = page_id(table[bl], (uint32_t)a.n_slots);
                if (id == kNoPage) atomicCAS(a.err, 0u, (uint32_t)kErrRange);
            }
            const char* base = static_cast<const char*>(a.bounds) + (uint64_t)(id == kNoPage ? 0u : id) * (4ull * D);
            V8 lo[D / 32], hi[D / 32];
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
                lo[kk] = *reinterpret_cast<const V8*>(base + 64 * kk + 16 * g);
                hi[kk] = *reinterpret_cast<const V8*>(base + 2 * D + 64 * kk + 16 * g);
            }
            float best[4], off[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                best[i] = -__builtin_inff();
                off[i] = 0.f;
            }
            for (uint32_t ct = 0; ct < a.col_tiles; ++ct) {
                // column -> (row of the tile, query head of the group)
                const uint32_t c = ct * 16 + col;
                const uint32_t row = one_tile ? c / a.group : 0u, head = one_tile ? c - row * a.group : c;
                const bool on = head < a.group && row < a.rows_per_tile && r0 + row < a.n_rows;
                f32x4 s = {0.f, 0.f, 0.f, 0.f}, w = {0.f, 0.f, 0.f, 0.f};
                const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (int64_t)(r0 + row) * a.q_row +
                                     (int64_t)(h * a.group + head) * a.q_head;
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) {
                    const u32x4 x = on ? load_eight(qp + 32 * kk + 8 * g, a.vec != 0) : u32x4{0u, 0u, 0u, 0u};
                    u32x4 p, m, pa, ma;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // the numbers above zero, and those below, of two at a time
                        const uint32_t neg = (x[j] >> 15 & 0x10001u) * 0xFFFFu;
                        p[j] = x[j] & ~neg;
                        m[j] = x[j] & neg;
                        pa[j] = p[j] & 0x7FFF7FFFu;
                        ma[j] = m[j] & 0x7FFF7FFFu;
                    }
                    s = E::mfma(hi[kk], bits_as<V8>(p), s);
                    s = E::mfma(lo[kk], bits_as<V8>(m), s);
                    w = E::mfma(bits_as<V8>(bits_as<u32x4>(hi[kk]) & 0x7FFF7FFFu), bits_as<V8>(pa), w);
                    w = E::mfma(bits_as<V8>(bits_as<u32x4>(lo[kk]) & 0x7FFF7FFFu), bits_as<V8>(ma), w);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!on) s[i] = -__builtin_inff();
                    if (!on || !(w[i] < __builtin_inff())) w[i] = 0.f;
                    best[i] = fmaxf(best[i], s[i]);  // a NaN is left out
                    off[i] = fmaxf(off[i], w[i]);
                }
            }
            // the highest over a row's heads: its columns, or (one row) all 16
            float slack = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = best[i], e = off[i];
                if (one_tile) {
                    for (uint32_t k = 1; k < a.group; ++k) {
                        v = fmaxf(v, __shfl(best[i], (int)(lane + k) & 63));
                        e = fmaxf(e, __shfl(off[i], (int)(lane + k) & 63));
                    }
                } else {
                    for (int o = 1; o < 16; o <<= 1) {
                        v = fmaxf(v, __shfl_xor(v, o));
                        e = fmaxf(e, __shfl_xor(e, o));
                    }
                }
                const uint32_t row = one_tile ? col / a.group : 0u;
                const bool lead_col = one_tile ? col == row * a.group : col == 0;
                const uint64_t b = bt + 4 * g + i;
                const bool live = lead_col && row < a.rows_per_tile && ((mine >> row) & 1u) != 0;
                const uint64_t nb_row = (uint64_t)__shfl((int)(uint32_t)row_nb, (int)min(row, 63u));
                if (live && b < nb_row) {
                    a.scores[((r0 + row) * a.kv_heads + h) * a.blocks + b] = v;
                    slack = fmaxf(slack, e);
                }
            }
            // the largest error bound of these 16 blocks, per row
            slack = fmaxf(slack, __shfl_xor(slack, 16));
            slack = fmaxf(slack, __shfl_xor(slack, 32));
            const uint32_t row = one_tile ? col / a.group : 0u;
            const bool lead_col = one_tile ? col == row * a.group : col == 0;
            if (g == 0 && lead_col && row < a.rows_per_tile && ((mine >> row) & 1u))
                a.slack[((r0 + row) * a.kv_heads + h) * a.chunks + bt / 16] = slack * kSumError;
        }
    }
}

// ---------------------------------------------------------------------------
// The choice.  One workgroup per (row, head).
// ---------------------------------------------------------------------------
constexpr uint32_t kChooseThreads = 512;
constexpr uint32_t kChooseWaves = kChooseThreads / kWave;
constexpr uint64_t kMaxBlocks = 1u << 17;  // near blocks are marked in 16 KiB of LDS

// Ascending order as unsigned numbers; NaN the lowest.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x);
    if (x != x) return 0u;
    const uint32_t k = (u >> 31) ? ~u : u | 0x80000000u;
    return x == 0.f ? 0x80000000u : k;  // both zeros are one value
}

__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

struct ChooseShared {
    uint32_t hist[256];
    uint32_t sums[kChooseWaves];
    float slack[kChooseWaves];
    uint32_t digit, left, in_count;
};

__device__ __forceinline__ uint32_t choose_sum(uint32_t v, ChooseShared& sh) {
    v = wave_sum(v);
    __syncthreads();
    if (lane_id() == 0) sh.sums[threadIdx.x / kWave] = v;
    __syncthreads();
    uint32_t s = 0;
    for (uint32_t i = 0; i < kChooseWaves; ++i) s += sh.sums[i];
    return s;
}

// The want-th largest (want >= 1) of key(b) over the blocks b in [0, nb) for
// which on(b); *above: how many are larger.  Four passes of eight bits.
template <class On, class Key>
__device__ __forceinline__ uint32_t nth_largest(uint64_t nb, uint32_t want, ChooseShared& sh, uint32_t* above, On on,
                                                Key key) {
    uint32_t prefix = 0, left = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (uint32_t i = threadIdx.x; i < 256; i += kChooseThreads) sh.hist[i] = 0;
        __syncthreads();
        for (uint64_t b = threadIdx.x; b < nb; b += kChooseThreads) {
            if (!on(b)) continue;
            const uint32_t k = key(b);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < kWave) {
            // lane l: digits 255 - 4 l .. 252 - 4 l, from the largest
            const uint32_t lane = lane_id();
            uint32_t c[4], tot = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[j] = sh.hist[255 - 4 * lane - j];
                tot += c[j];
            }
            const uint32_t incl = wave_incl_scan(tot);
            uint32_t before = incl - tot;
            const uint64_t has = ballot(incl >= left);
            if (has && lane == (uint32_t)__builtin_ctzll(has)) {
                uint32_t j = 0;
                while (j < 3 && before + c[j] < left) before += c[j++];
                sh.digit = 255 - 4 * lane - j;
                sh.left = left - before;
            }
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        left = sh.left;
        __syncthreads();
    }
    *above = want - left;
    return prefix;
}

template <class E, int D>
__global__ __launch_bounds__(kChooseThreads) void k_choose(SelectArgs a) {
    __shared__ ChooseShared sh;
    extern __shared__ uint32_t near_bits[];  // blocks to be summed in 64 bits
    const uint64_t rh = blockIdx.x;
    const uint64_t r = rh / a.kv_heads;
    const uint32_t h = (uint32_t)(rh % a.kv_heads);
    const uint32_t tid = threadIdx.x, lane = lane_id(), wib = tid / kWave;
    int32_t* out = a.out + rh * a.n_out;
    int64_t seq;
    const uint64_t nb = row_blocks(a, r, &seq);
    if (tid == 0) {
        const int64_t len = a.lens[r];
        if (seq < 0 || (uint64_t)seq >= a.n_seqs || len < 0 || (uint64_t)len > a.blocks * a.page_tokens)
            atomicCAS(a.err, 0u, (uint32_t)kErrRange);
    }
    if (nb <= a.n_out) {
        for (uint32_t i = tid; i < a.n_out; i += kChooseThreads) out[i] = i < nb ? (int32_t)i : -1;
        return;
    }
    float* scores = a.scores + rh * a.blocks;
    const uint64_t f_end = a.keep_first, l_begin = nb - a.keep_last;  // keep_first + keep_last <= n_out < nb
    auto kept = [&](uint64_t b) { return b < f_end || b >= l_begin; };
    const uint32_t want = a.n_out - a.keep_first - a.keep_last;
    uint32_t cut = 0xFFFFFFFFu, ties = 0;  // chosen: above `cut` in order, and the first `ties` equal to it
    uint32_t nth_key = 0;  // pages that are not near are chosen above this
    bool any_near = false;
    if (want > 0) {
        float slack = 0.f;
        for (uint64_t c = tid; c < (nb + 15) / 16; c += kChooseThreads) slack = fmaxf(slack, a.slack[rh * a.chunks + c]);
        for (int o = 32; o > 0; o >>= 1) slack = fmaxf(slack, __shfl_xor(slack, o));
        if (lane == 0) sh.slack[wib] = slack;
        __syncthreads();
        for (uint32_t i = 0; i < kChooseWaves; ++i) slack = fmaxf(slack, sh.slack[i]);
        uint32_t above;
        const uint32_t nth = nth_largest(
            nb, want, sh, &above, [&](uint64_t b) { return !kept(b); }, [&](uint64_t b) { return order_of(scores[b]); });
        const float t = value_of(nth);
        // Every true score is within `slack` of its sum, so the want-th
        // largest true one is within slack of t; pages further than two of
        // them from t are decided, and two more cover the final rounding.
        const float lo_near = t - 4.f * slack, hi_near = t + 4.f * slack;
        // with no slack (all products zero, or not finite) the sums are taken as they are
        const bool finite = t - t == 0.f && slack > 0.f;
        // pages to be summed again, and how many lie above them
        for (uint64_t w = tid; w < (nb + 31) / 32; w += kChooseThreads) near_bits[w] = 0;
        __syncthreads();
        uint32_t n_above = 0, n_near = 0;
        for (uint64_t b = tid; b < nb; b += kChooseThreads) {
            if (kept(b)) continue;
            const float s = scores[b];
            if (finite && s >= lo_near && s <= hi_near) {
                atomicOr(&near_bits[b >> 5], 1u << (b & 31));
                ++n_near;
            } else if (order_of(s) > nth) {
                ++n_above;
            }
        }
        n_above = choose_sum(n_above, sh);
        n_near = choose_sum(n_near, sh);
        any_near = finite;
        if (!finite) {
            cut = nth;
            ties = want - above;
        } else if (n_above + n_near == want) {
            cut = 0;  // every near one: their keys are above 0, a NaN's
        } else {
            const int64_t* table = a.table + ((uint64_t)seq * a.kv_heads + h) * a.blocks;
            // one wave per page: lane l sums the dims l, l + 64, ... of every
            // head of the group in 64 bits
            for (uint64_t w = wib; w < (nb + 31) / 32; w += kChooseWaves) {
                for (uint32_t m = uniform(near_bits[w]); m; m &= m - 1) {
                    const uint64_t b = 32 * w + (uint32_t)__builtin_ctz(m);
                    const uint32_t id = page_id(table[b], (uint32_t)a.n_slots);
                    if (id == kNoPage) continue;
                    const uint16_t* bp = static_cast<const uint16_t*>(a.bounds) + (uint64_t)id * (2ull * D);
                    float best = -__builtin_inff();
                    for (uint32_t j = 0; j < a.group; ++j) {
                        const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (int64_t)r * a.q_row +
                                             (int64_t)(h * a.group + j) * a.q_head;
                        double s = 0.0;
                        for (uint32_t d = lane; d < (uint32_t)D; d += kWave) {
                            const double x = (double)E::from_bits(qp[d]);
                            s += (x > 0.0 ? x : 0.0) * (double)E::from_bits(bp[D + d]) +
                                 (x < 0.0 ? x : 0.0) * (double)E::from_bits(bp[d]);
                        }
                        for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
                        best = fmaxf(best, (float)s);
                    }
                    if (lane == 0) scores[b] = best;
                }
            }
            __threadfence_block();
            __syncthreads();
            uint32_t above_near;
            const uint32_t rest = want - n_above;
            cut = nth_largest(
                nb, rest, sh, &above_near, [&](uint64_t b) { return ((near_bits[b >> 5] >> (b & 31)) & 1u) != 0; },
                [&](uint64_t b) { return order_of(scores[b]); });
            ties = rest - above_near;
        }
        nth_key = nth;
    }
    // ascending order: a running count over slices of kChooseThreads blocks
    uint32_t at = 0, ties_used = 0;
    for (uint64_t base = 0; base < nb; base += kChooseThreads) {
        const uint64_t b = base + tid;
        bool in = false, tie = false;
        if (b < nb) {
            if (kept(b)) {
                in = true;
            } else if (want > 0) {
                const uint32_t k = order_of(scores[b]);
                const bool near = any_near && ((near_bits[b >> 5] >> (b & 31)) & 1u);
                if (any_near && !near) {
                    in = k > nth_key;
                } else {
                    in = k > cut;
                    tie = !in && k == cut;
                }
            }
        }
        // ties in order of their block
        const uint64_t tb = ballot(tie);
        __syncthreads();
        if (lane == 0) sh.sums[wib] = (uint32_t)__builtin_popcountll(tb);
        __syncthreads();
        uint32_t tie_rank = ties_used + bits_below(tb), slice_ties = 0;
        for (uint32_t i = 0; i < kChooseWaves; ++i) {
            if (i < wib) tie_rank += sh.sums[i];
            slice_ties += sh.sums[i];
        }
        ties_used += slice_ties;
        if (tie && tie_rank < ties) in = true;
        const uint64_t ib = ballot(in);
        __syncthreads();
        if (lane == 0) sh.sums[wib] = (uint32_t)__builtin_popcountll(ib);
        __syncthreads();
        uint32_t rank = at + bits_below(ib);
        for (uint32_t i = 0; i < kChooseWaves; ++i) {
            if (i < wib) rank += sh.sums[i];
            at += sh.sums[i];
        }
        if (in && rank < a.n_out) out[rank] = (int32_t)b;
    }
    for (uint32_t i = at + tid; i < a.n_out; i += kChooseThreads) out[i] = -1;
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
        // stay in device memory
        const bool lds = pool.Mw < 4 || tab + stage <= kLdsPerCu / 2;
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

static uint64_t select_chunks(const ibp_attention* a) { return (a->table_blocks + 15) / 16; }

uint64_t ibp_select_pages_workspace(const ibp_attention* a) {
    if (!a) return 0;
    return 4 * a->n_rows * a->n_kv_heads * (a->table_blocks + select_chunks(a)) + 16;
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
    if (reinterpret_cast<uintptr_t>(bounds) % 16 || reinterpret_cast<uintptr_t>(workspace) % 8 ||
        workspace_bytes < ibp_select_pages_workspace(a))
        return IBP_ERR_INVALID_ARG;
    SelectArgs s{};
    s.q = q;
    s.bounds = bounds;
    s.table = k_table;
    s.lens = lens;
    s.row_seq = row_seq;
    s.blocks = a->table_blocks;
    s.chunks = select_chunks(a);
    s.scores = static_cast<float*>(workspace);
    s.slack = s.scores + a->n_rows * a->n_kv_heads * a->table_blocks;
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
    s.rows_per_tile = s.group <= 16 ? 16 / s.group : 1;
    s.col_tiles = (s.group + 15) / 16;
    s.vec = vectors_ok(q, a->q_row_stride, a->q_head_stride);
    const uint64_t tiles = (a->n_rows + s.rows_per_tile - 1) / s.rows_per_tile;
    if (tiles > 65535 || a->n_kv_heads > 65535 || a->n_rows * a->n_kv_heads > 0x7FFFFFFFull) return IBP_ERR_UNSUPPORTED;
    const bool scored = a->table_blocks > n_blocks && n_blocks > keep_first + keep_last;
    auto launch = [&](auto e, auto dc) {
        using E = decltype(e);
        constexpr int D = decltype(dc)::value;
        if (scored) {  // no row can have more pages than it may read otherwise
            const dim3 grid((uint32_t)((a->table_blocks + kScoreChunk - 1) / kScoreChunk), a->n_kv_heads,
                            (uint32_t)tiles);
            hipLaunchKernelGGL((k_scores<E, D>), grid, dim3(kWave * kScoreWaves), 0, stream, s);
            const hipError_t err = hipGetLastError();
            if (err != hipSuccess) return err;
        }
        hipLaunchKernelGGL((k_choose<E, D>), dim3((uint32_t)(a->n_rows * a->n_kv_heads)), dim3(kChooseThreads),
                           (uint32_t)(4 * ((a->table_blocks + 31) / 32)), stream, s);
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
