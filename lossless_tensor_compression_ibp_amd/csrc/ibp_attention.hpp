// ibp_attention.hpp -- attention over a cache's pages: the kernels, for one
// number type.  Each number type is compiled in a file of its own.
//
// Mathematics.  For the rows of one key/value head, t_j = scale * q.k_j,
// o = sum_j exp(t_j - m) v_j / sum_j exp(t_j - m) with the running maximum m.
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T: a lane of the
// matrix cores' result then holds four tokens (S^T) or four dims (O^T) of ONE
// row, its column l % 16, so m, the sum and the rescaling are one number per
// lane, and the weights that a lane computes from S^T are exactly the eight it
// has to supply to O^T's product: tokens 4 g + 0..3 of two tiles of 16, where
// g = l / 16.  (The product sums over tokens, so their order is free as long
// as V^T's operand has the same: two transposed LDS reads of four tokens.)
//
// Pages.  A wave loads a slot linearly (16 bytes per lane and instruction),
// rebuilds it in registers if it holds a record, and writes it to LDS as rows
// of tokens, padded so that the operand reads spread over the banks.  The next
// page's loads are in flight meanwhile.
//
// Two shapes of work:
//   SHARED = false: few rows (16 MR).  Every wave walks pages of its own for
//     all rows, without a barrier, and the waves' results are joined at the
//     end.  Bound by the pages' bytes (or their rebuild).
//   SHARED = true: many rows.  The workgroup's waves load a step's pages
//     together, each rebuilding its share, and each multiplies all of them
//     with 16 MR rows of its own.
// A long context is split over workgroups; k_join adds the parts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ibp_kv_math.hpp"

namespace ibp {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kAttnWaves = 4;

struct AttnArgs {
    Pool k, v;
    const uint16_t* q;
    const int64_t* k_table;
    const int64_t* v_table;
    const int32_t* lens;
    const int32_t* new_rows;   // tree
    const uint16_t* k_new;
    const uint16_t* v_new;
    const uint32_t* mask;      // tree: 2 * mask_words per row
    const int32_t* row_seq;    // sparse
    const int32_t* blocks;     // sparse: n_list per (row, head)
    uint16_t* out;
    float* lse;
    float* part;               // [row][head][split][D], then [row][head][split][2]
    float* part_ml;
    uint64_t n_rows, n_seqs, table_blocks;
    int64_t q_row, q_head, new_row, new_head;
    uint32_t n_list, mask_words2, max_new;
    uint32_t kv_heads, group, splits, row_tiles, work;  // work: (sequence or row) * kv_heads
    uint32_t tab_words_k, tab_words_v;  // LDS words of the tables (0: not staged)
    uint32_t tab_lds_k, tab_lds_v;      // staged in LDS, else read where they lie in device memory
    uint32_t same_tab;                  // values have the keys' tables
    float scale2;              // |scale| * log2(e), not zero
    uint32_t q_sign;           // both sign bits for a negative scale
};

typedef short i16x4 __attribute__((ext_vector_type(4)));

// Four tokens' numbers of one dim: within 16 lanes, lane i addresses four
// consecutive dims of token i / 4 and receives dim i of the four tokens.
__device__ __forceinline__ u32x2 read_transposed(const char* lds) {
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)lds));
}

template <int D, int T, bool SHARED>
struct AttnShape {
    static constexpr int NV = D * T / 512;                 // vectors per lane of a page
    static constexpr int STEP = SHARED ? (T == 64 ? 128 : 64) : (T < 32 ? 32 : T);
    static constexpr int PP = STEP / T;                    // pages per step
    static constexpr bool BOTH = !SHARED || T == 16;       // a wave loads keys and values
    static constexpr int PW = SHARED ? 1 : PP;             // pages per step, wave and kind
    static constexpr int RK = 2 * D + 16, RV = 2 * D + 32; // bytes per token row in LDS
    static constexpr uint32_t stage_bytes = 4 * page_stage_words<NV>();
    static constexpr int CHUNK = SHARED ? 64 : STEP;       // tokens per pass of the softmax
    static constexpr bool ONE = !SHARED && PW * NV > 8;    // one register buffer for keys and values in turn
    static constexpr uint32_t wave_bytes = PW * stage_bytes + (SHARED ? 0 : STEP * RV);
    static_assert(stage_bytes % 16 == 0, "areas are vectors");
    static constexpr uint32_t shared_bytes = SHARED ? STEP * (RK + RV) : 0;
    static constexpr uint32_t join_bytes = SHARED ? 0 : kAttnWaves * (16 * (D + 4) * 4);
    static constexpr uint32_t area_bytes =
        kAttnWaves * wave_bytes + shared_bytes > join_bytes ? kAttnWaves * wave_bytes + shared_bytes : join_bytes;
};

// Infinities and NaNs of eight numbers become zero; whether there was one.
template <class E>
__device__ __forceinline__ bool clear_odd(u32x4& x) {
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t lo = x[j] & E::kExponent, hi = (x[j] >> 16) & E::kExponent;
        if (lo == E::kExponent) x[j] &= 0xFFFF0000u;
        if (hi == E::kExponent) x[j] &= 0x0000FFFFu;
        odd = odd || lo == E::kExponent || hi == E::kExponent;
    }
    return odd;
}

// x of lane l joined with x of lanes l ^ 16, l ^ 32 and l ^ 48: exchanges of
// whole rows of 16 and 32 lanes, which take no LDS round trip.
template <class F>
__device__ __forceinline__ float over_four(float x, F f) {
    const uint32_t a = __float_as_uint(x);
    const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    x = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const uint32_t b = __float_as_uint(x);
    const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return f(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float max_over_four(float x) {
    return over_four(x, [](float a, float b) __attribute__((always_inline)) { return fmaxf(a, b); });
}
__device__ __forceinline__ float sum_over_four(float x) {
    return over_four(x, [](float a, float b) __attribute__((always_inline)) { return a + b; });
}

__device__ __forceinline__ void lds_order() { asm volatile("" ::: "memory"); }

// The kernel's arguments once more.  What only rare or final steps need is
// read through this pointer where it is needed: the compiler cannot tell that
// it is the arguments', so it does not keep them in scalar registers (with all
// of them live the loop spent a tenth of its instructions on saving them).
typedef const __attribute__((address_space(4))) AttnArgs* ArgsPtr;
__device__ __forceinline__ ArgsPtr args_again() {
    ArgsPtr p = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}

template <class E, int D, int T, int MR, bool SHARED, bool TREE>
__global__ __launch_bounds__(kWave * kAttnWaves, 2) void k_attend(AttnArgs a) {
    using S = AttnShape<D, T, SHARED>;
    using V8 = typename E::V8;
    constexpr int NV = S::NV, STEP = S::STEP, PP = S::PP, PW = S::PW, TILES = S::CHUNK / 16;
    constexpr int DK = D / 32, DN = D / 16;
    constexpr uint32_t kRowsWg = 16u * MR * (SHARED ? kAttnWaves : 1u);
    constexpr uint32_t kStride = SHARED ? 1u : kAttnWaves;  // steps between a wave's steps
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ float join_m[kAttnWaves][16], join_l[kAttnWaves][16];
    __shared__ uint32_t odd_values;  // an infinity or NaN among the drafted values
    const uint32_t lane = lane_id(), wib = uniform(threadIdx.x / kWave);
    const uint32_t col = lane & 15u, g = lane >> 4;

    // the first vector per thread of each pool's tables is on its way while
    // the wave finds its pages
    u32x4 tab_k = {0u, 0u, 0u, 0u}, tab_v = {0u, 0u, 0u, 0u};
    if (4 * threadIdx.x < a.tab_words_k) tab_k = page_table_vector(a.k, threadIdx.x);
    if (4 * threadIdx.x < a.tab_words_v) tab_v = page_table_vector(a.v, threadIdx.x);
    if (TREE && threadIdx.x == 0) odd_values = 0;

    // which part of the work: split, (sequence or row, head), row tile
    const uint32_t split = blockIdx.x % a.splits;
    const uint32_t wg = (blockIdx.x / a.splits) % a.work, rt = blockIdx.x / a.splits / a.work;
    const uint32_t h = wg % a.kv_heads;
    const uint32_t item = wg / a.kv_heads;  // sequence (tree) or row
    uint32_t seq = item, first_row = TREE ? 0u : item, n_new = TREE ? 0u : 1u;
    int32_t len = a.lens[item];
    bool bad = len < 0 || (uint64_t)len > a.table_blocks * T;
    if (TREE) {
        const int32_t r0 = a.new_rows[item], r1 = a.new_rows[item + 1];
        const uint32_t n = (uint32_t)(r1 - r0);
        if (r0 < 0 || r1 < r0 || (uint64_t)r1 > a.n_rows || n > a.max_new || n > 32u * a.mask_words2) {
            bad = true;
        } else {
            first_row = (uint32_t)r0;
            n_new = n;
        }
    } else if (a.row_seq) {
        const int32_t s = a.row_seq[item];
        bad = bad || s < 0 || (uint64_t)s >= a.n_seqs;
        seq = (uint32_t)s;
    }
    if (bad) {
        latch_error(a.k.err, kErrRange);
        if (TREE) return;
        seq = 0;
        len = 0;
    }
    const uint32_t rows = n_new * a.group;
    if (rt * kRowsWg >= rows) return;
    const uint32_t row0 = rt * kRowsWg + (SHARED ? wib * 16u * MR : 0u);

    // steps of this split: the context's, then the drafted tokens'
    const uint32_t ctx_pages = TREE ? ((uint32_t)len + T - 1) / T : (len > 0 ? a.n_list : 0u);
    const uint32_t ctx_steps = (ctx_pages + PP - 1) / PP;
    const uint32_t all_steps = ctx_steps + (TREE ? (n_new + STEP - 1) / STEP : 0u);
    const uint32_t per = (all_steps + a.splits - 1) / a.splits;
    const uint32_t s_lo = min(split * per, all_steps), s_hi = min(s_lo + per, all_steps);
    const uint32_t s_first = s_lo + (SHARED ? 0u : wib);
    const uint32_t n_steps = s_first < s_hi ? (s_hi - s_first + kStride - 1) / kStride : 0u;

    char* const area = reinterpret_cast<char*>(smem + a.tab_words_k + a.tab_words_v);
    uint32_t* const stage = reinterpret_cast<uint32_t*>(area + wib * S::wave_bytes);
    char* const k_tile =
        SHARED ? area + kAttnWaves * S::wave_bytes : reinterpret_cast<char*>(stage) + PW * S::stage_bytes;
    char* const v_tile = SHARED ? k_tile + STEP * S::RK : k_tile;

    // a wave of SHARED pages of 32 or 64 tokens loads keys or values only
    const bool only_v = !S::BOTH && (wib & 1u);
    const uint32_t page_in_step = SHARED ? (T == 16 ? wib : wib >> 1) : 0u;

    // --- the wave's next pages: lane l has page l % PW of its step base + l / PW
    uint32_t id_a = 0, id_b = 0, held = 0, comp = 0;
    auto refill = [&](uint32_t base) __attribute__((always_inline)) {
        const ArgsPtr c = args_again();
        const uint32_t s = s_first + (base + lane / PW) * kStride;
        id_a = id_b = held = comp = 0;
        if (s < s_hi && s < ctx_steps) {
            const uint32_t n = s * PP + (SHARED ? page_in_step : lane % PW);
            int32_t block = n < ctx_pages ? (int32_t)n : -1;
            if (!TREE && n < ctx_pages) block = c->blocks[((uint64_t)item * a.kv_heads + h) * c->n_list + n];
            if (block >= 0 && (int64_t)block * T < len) {
                held = (uint32_t)min(T, len - block * T);
                const uint64_t at = ((uint64_t)seq * a.kv_heads + h) * c->table_blocks + (uint32_t)block;
                // both ids, then both bits, each pair in one latency
                const bool keys = S::BOTH || !only_v, values = S::BOTH || only_v;
                const int64_t k64 = keys ? c->k_table[at] : 0, v64 = values ? c->v_table[at] : 0;
                const uint32_t k = page_id(k64, c->k.n_slots), v = page_id(v64, c->v.n_slots);
                const bool missing = (keys && k == kNoPage) || (values && v == kNoPage);
                const uint32_t k_at = !keys || k == kNoPage ? 0u : k, v_at = !values || v == kNoPage ? 0u : v;
                const uint32_t k_word = c->k.bitmask[k_at >> 5], v_word = c->v.bitmask[v_at >> 5];
                const uint32_t k_bit = keys && k != kNoPage ? (k_word >> (k_at & 31u)) & 1u : 0u;
                const uint32_t v_bit = values && v != kNoPage ? (v_word >> (v_at & 31u)) & 1u : 0u;
                id_a = S::BOTH || !only_v ? k_at : v_at;
                id_b = v_at;
                comp = S::BOTH ? k_bit | v_bit << 1 : k_bit | v_bit;
                if (missing) atomicCAS(c->k.err, 0u, (uint32_t)kErrRange);
            }
        }
    };
    // The pages of local step i -> registers: T rows of D numbers each, of a
    // slot, or of the drafted tokens' dense rows (where rows past the last
    // token read the last one).  What they hold beyond the page's tokens is
    // masked (keys) or cleared (values) later.
    auto load = [&](u32x4* st, uint32_t i, bool values, uint32_t ids) __attribute__((always_inline)) {
        const uint32_t s = s_first + i * kStride;
        if (!TREE || s < ctx_steps) {
#pragma unroll
            for (int p = 0; p < PW; ++p)
                load_page<NV>(st + p * NV, values ? a.v.slots : a.k.slots,
                              lane_value(ids, (int)((i % (64 / PW)) * PW + p)));
        } else {
            const ArgsPtr c = args_again();
            const uint16_t* base = (values ? c->v_new : c->k_new) + (int64_t)h * c->new_head;
            const int64_t row = c->new_row;
#pragma unroll
            for (int p = 0; p < PW; ++p) {
                const uint32_t j0 = (s - ctx_steps) * STEP + (SHARED ? page_in_step : (uint32_t)p) * T;
#pragma unroll
                for (int r = 0; r < NV; ++r) {
                    const uint32_t w = 256u * r + 4u * lane, token = min(j0 + w / (D / 2), n_new - 1);
                    st[p * NV + r] = load_eight(base + (int64_t)(first_row + token) * row + 2 * (w % (D / 2)));
                }
            }
        }
    };
    // The wave's pages as rows of tokens in LDS.  A record goes through the
    // stage; values behind a page's last token become zero.  Lane-wise words
    // of a page: four at w, of token w / (D / 2).
    auto put = [&](const u32x4* st, bool values, uint32_t records, const uint32_t* keep, char* tile, int stride)
                   __attribute__((always_inline)) {
        auto row_of = [&](uint32_t p, uint32_t n, uint32_t w, u32x4 x) __attribute__((always_inline)) {
            const uint32_t token = w / (D / 2), b = 4 * (w % (D / 2));
            if (token >= n) x = u32x4{0u, 0u, 0u, 0u};
            *reinterpret_cast<u32x4*>(tile + ((SHARED ? page_in_step : p) * T + token) * stride + b) = x;
        };
        lds_order();
#pragma unroll
        for (int p = 0; p < PW; ++p) {
            const uint32_t n = values ? keep[p] : (uint32_t)T;
            if ((records >> p) & 1u) {
                stage_page<NV>(st + p * NV, stage + p * (S::stage_bytes / 4));
            } else if (n == (uint32_t)T) {
#pragma unroll
                for (int r = 0; r < NV; ++r) row_of(p, T, 256u * r + 4u * lane, st[p * NV + r]);
            } else {
#pragma unroll
                for (int r = 0; r < NV; ++r) row_of(p, n, 256u * r + 4u * lane, st[p * NV + r]);
            }
        }
        const Pool& pool = values ? a.v : a.k;
        const PageTab tab = page_tab(pool, smem + (values && !a.same_tab ? a.tab_words_k : 0u),
                                     values ? a.tab_lds_v : a.tab_lds_k);
        for (; records; records &= records - 1) {
            const uint32_t p = PW == 1 ? 0u : (uint32_t)__builtin_ctz(records);
            const uint32_t n = !values ? (uint32_t)T : PW == 1 || p == 0 ? keep[0] : keep[PW - 1];
            if (!rebuild_page<NV>(pool, tab, stage + p * (S::stage_bytes / 4),
                                  [&](uint32_t w, u32x4 x) __attribute__((always_inline)) { row_of(p, n, w, x); }))
                latch_error(args_again()->k.err, kErrCorrupt);
        }
        lds_order();
    };

    // --- the rows' queries (B operand) and running state
    V8 qf[MR][DK];
    float m[MR], l[MR];
    f32x4 o[MR][DN];
    uint32_t q_row[MR];  // of lane's column; kNoPage past the last row
    auto row_head = [&](uint32_t rho, uint32_t* j) __attribute__((always_inline)) {
        const uint32_t i = rho / a.group;
        *j = rho - i * a.group;
        return first_row + i;
    };
    {
        const ArgsPtr c = args_again();
#pragma unroll
        for (int t = 0; t < MR; ++t) {
            const uint32_t rho = row0 + 16 * t + col;
            uint32_t j;
            q_row[t] = row_head(rho, &j);
            if (rho >= rows) q_row[t] = kNoPage;
            const uint16_t* qp = c->q + (int64_t)q_row[t] * c->q_row + (int64_t)(h * a.group + j) * c->q_head;
#pragma unroll
            for (int kk = 0; kk < DK; ++kk) {
                u32x4 x = {0u, 0u, 0u, 0u};
                if (rho < rows) x = load_eight(qp + 32 * kk + 8 * g);
                qf[t][kk] = bits_as<V8>(x ^ c->q_sign);  // (a negative scale is taken into the queries)
            }
            m[t] = -__builtin_inff();
            l[t] = 0.f;
#pragma unroll
            for (int n = 0; n < DN; ++n) o[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
    // tables of the record formats, once the first pages are on their way
    auto put_tables = [&]() __attribute__((always_inline)) {
        if (4 * threadIdx.x < a.tab_words_k) reinterpret_cast<u32x4*>(smem)[threadIdx.x] = tab_k;
        if (4 * threadIdx.x < a.tab_words_v) reinterpret_cast<u32x4*>(smem + a.tab_words_k)[threadIdx.x] = tab_v;
        if (a.tab_words_k > 4 * kWave * kAttnWaves) stage_page_tables(a.k, smem, kWave * kAttnWaves);
        if (a.tab_words_v > 4 * kWave * kAttnWaves) stage_page_tables(a.v, smem + a.tab_words_k, kWave * kAttnWaves);
    };

    u32x4 st_a[PW * NV], st_b[S::BOTH && !S::ONE ? PW * NV : 1];
    bool odd = false;
    // of the step at work and of the next: tokens of each page that the wave
    // loads, and the rows' mask words of drafted steps; which pages at work
    // are records (keys, then values); ids of the value pages at work (ONE)
    uint32_t n_held[PW], next_held[PW], records = 0, ids_b = 0;
    uint32_t sees[TREE ? MR : 1][STEP / 32], next_sees[TREE ? MR : 1][STEP / 32];
    auto facts = [&](uint32_t j) __attribute__((always_inline)) {
        const uint32_t sn = s_first + j * kStride;
#pragma unroll
        for (int p = 0; p < PW; ++p) {
            next_held[p] = lane_value(held, (int)((j % (64 / PW)) * PW + p));
            if (TREE && sn >= ctx_steps) {
                const uint32_t j0 = (sn - ctx_steps) * STEP + (SHARED ? page_in_step : (uint32_t)p) * T;
                next_held[p] = n_new > j0 ? min(n_new - j0, (uint32_t)T) : 0u;
            }
        }
        if (TREE && sn >= ctx_steps) {
            const ArgsPtr x = args_again();
#pragma unroll
            for (int t = 0; t < MR; ++t) {
#pragma unroll
                for (int w = 0; w < STEP / 32; ++w) {
                    const uint32_t word = (sn - ctx_steps) * (STEP / 32) + w;
                    next_sees[t][w] = 0;
                    if (q_row[t] != kNoPage && word < x->mask_words2)
                        next_sees[t][w] = x->mask[(uint64_t)q_row[t] * x->mask_words2 + word];
                }
            }
        }
    };
    // step j becomes the one at work (after its loads have been sent: the
    // records' bits come a latency after the ids)
    auto advance = [&](uint32_t j) __attribute__((always_inline)) {
        records = 0;
        ids_b = id_b;
#pragma unroll
        for (int p = 0; p < PW; ++p) {
            n_held[p] = next_held[p];
            const uint32_t c = lane_value(comp, (int)((j % (64 / PW)) * PW + p));
            records |= (c & 1u) << p | (c >> 1) << (PW + p);
        }
    };
    auto take_sees = [&]() __attribute__((always_inline)) {
        if constexpr (TREE) {
#pragma unroll
            for (int t = 0; t < MR; ++t) {
#pragma unroll
                for (int w = 0; w < STEP / 32; ++w) sees[t][w] = next_sees[t][w];
            }
        }
    };
#pragma unroll
    for (int t = 0; t < (TREE ? MR : 1); ++t) {
#pragma unroll
        for (int w = 0; w < STEP / 32; ++w) sees[t][w] = next_sees[t][w] = 0;
    }
    if (n_steps) {
        refill(0);
        facts(0);
        load(st_a, 0, only_v, id_a);
        if constexpr (S::BOTH && !S::ONE) load(st_b, 0, true, id_b);
    }
    put_tables();
    if (n_steps) {
        advance(0);
        take_sees();
    }
    if constexpr (!SHARED) __syncthreads();  // (the loop of SHARED begins with one)

    for (uint32_t i = 0; i < n_steps; ++i) {
        const bool more = i + 1 < n_steps;
        const uint32_t s = s_first + i * kStride;
        const bool draft = TREE && s >= ctx_steps;
        auto put_keys = [&]() __attribute__((always_inline)) {
            put(st_a, false, records & ((1u << PW) - 1), n_held, k_tile, S::RK);
        };
        auto put_values = [&](u32x4* st, uint32_t shift) __attribute__((always_inline)) {
            // Infinities and NaNs of drafted values are taken out, so that
            // they reach no row through a product with a weight of zero, and
            // added at the end to the rows that see them.
            if (draft) {
#pragma unroll
                for (int r = 0; r < PW * NV; ++r) odd |= clear_odd<E>(st[r]);
            }
            put(st, true, records >> shift, n_held, v_tile, S::RV);
        };
        if constexpr (SHARED) {
            __syncthreads();  // the tiles are free, and the tables there
            if (S::BOTH) {
                put_keys();
                put_values(st_b, PW);
            } else if (only_v) {
                put_values(st_a, 0);
            } else {
                put_keys();
            }
        } else {
            put_keys();
        }
        const uint32_t step_held_all =
            draft ? min(n_new - (s - ctx_steps) * STEP, (uint32_t)STEP) : min((uint32_t)len - s * STEP, (uint32_t)STEP);
        uint32_t tiles_held[!TREE && !SHARED ? PW : 1];  // tokens of the pages at work, for the masks
        if constexpr (!TREE && !SHARED) {
#pragma unroll
            for (int p = 0; p < PW; ++p) tiles_held[p] = n_held[p];
        }
        if constexpr (S::ONE) load(st_a, i, true, ids_b);
        if (more) {
            if ((i + 1) % (64 / PW) == 0) refill(i + 1);
            facts(i + 1);
            if constexpr (!S::ONE) load(st_a, i + 1, only_v, id_a);
            if constexpr (SHARED && S::BOTH) load(st_b, i + 1, true, id_b);
        }
        if constexpr (SHARED) {
            if (more) advance(i + 1);
            __syncthreads();
        }
#pragma unroll 1
        for (uint32_t c = 0; c < (uint32_t)(STEP / S::CHUNK); ++c) {
            // valid tokens of each tile of 16
            const uint32_t t0 = c * S::CHUNK;
            auto tile_held = [&](int u) __attribute__((always_inline)) -> uint32_t {
                if constexpr (TREE || SHARED) {
                    const uint32_t before = t0 + 16u * u;
                    return step_held_all > before ? step_held_all - before : 0u;
                } else {
                    const uint32_t n = tiles_held[(u * 16) / T < PW ? (u * 16) / T : 0];
                    return n > (uint32_t)(u * 16 % T) ? n - (uint32_t)(u * 16 % T) : 0u;
                }
            };
            const char* const kt = k_tile + t0 * S::RK;
            const char* const vt = v_tile + t0 * S::RV;
            // S^T = K Q^T
            f32x4 sc[MR][TILES];
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
#pragma unroll
                for (int t = 0; t < MR; ++t) sc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < DK; ++kk) {
                    const V8 kf = *reinterpret_cast<const V8*>(kt + (16 * u + col) * S::RK + 64 * kk + 16 * g);
#pragma unroll
                    for (int t = 0; t < MR; ++t) sc[t][u] = E::mfma(kf, qf[t][kk], sc[t][u]);
                }
            }
            // masked scores -infinity, the running maximum, weights
            bool whole = !draft;
#pragma unroll
            for (int u = 0; u < TILES; ++u) whole = whole && tile_held(u) >= 16u;
            if (!whole) {
#pragma unroll
                for (int t = 0; t < MR; ++t) {
#pragma unroll
                    for (int u = 0; u < TILES; ++u) {
                        // bit j of `seen`: the lane's row sees token j of the tile
                        uint32_t seen = tile_held(u) >= 16u ? 0xFFFFu : (1u << tile_held(u)) - 1u;
                        if (draft) {
                            uint32_t bits = sees[TREE ? t : 0][u / 2];
                            if constexpr (STEP > S::CHUNK) bits = c ? sees[TREE ? t : 0][STEP / 64 + u / 2] : bits;
                            seen &= bits >> (16 * (u & 1));
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[t][u][e] = (seen >> (4 * g + e)) & 1u ? sc[t][u][e] : -__builtin_inff();
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < MR; ++t) {
                float top = -__builtin_inff();
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[t][u][e]);
                }
                top = max_over_four(top) * a.scale2;
                // The maximum is moved only when a score passes it by more
                // than 8 (weights then stay below 2^8 and sums far from
                // overflow), so most steps rescale nothing.
                if (ballot(top > m[t] + 8.f || (m[t] == -__builtin_inff() && top != -__builtin_inff()))) {
                    const float m_new = fmaxf(m[t], top);
                    const float f = m_new == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(m[t] - m_new);
                    m[t] = m_new;
                    l[t] *= f;
#pragma unroll
                    for (int n = 0; n < DN; ++n) o[t][n] *= f;
                }
                const float base = m[t] == -__builtin_inff() ? 0.f : -m[t];
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][u][e], a.scale2, base));
                        sc[t][u][e] = p;
                    }
                    l[t] += (sc[t][u][0] + sc[t][u][1]) + (sc[t][u][2] + sc[t][u][3]);
                }
            }

            if constexpr (!SHARED) put_values(S::ONE ? st_a : st_b, PW);
            if constexpr (!SHARED) {
                if (more) {
                    if constexpr (S::ONE)
                        load(st_a, i + 1, false, id_a);
                    else
                        load(st_b, i + 1, true, id_b);
                    advance(i + 1);
                }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int u = 0; u < TILES; u += 2) {
                V8 pf[MR];
#pragma unroll
                for (int t = 0; t < MR; ++t) {
                    const u32x4 x = {E::pack(sc[t][u][0], sc[t][u][1]), E::pack(sc[t][u][2], sc[t][u][3]),
                                     E::pack(sc[t][u + 1][0], sc[t][u + 1][1]),
                                     E::pack(sc[t][u + 1][2], sc[t][u + 1][3])};
                    pf[t] = bits_as<V8>(x);
                }
                const char* vp = vt + (16 * u + 4 * g + (col >> 2)) * S::RV + 8 * (col & 3);
#pragma unroll
                for (int n = 0; n < DN; ++n) {
                    const u32x2 x = read_transposed(vp + 32 * n), y = read_transposed(vp + 16 * S::RV + 32 * n);
                    const V8 vf = bits_as<V8>(u32x4{x[0], x[1], y[0], y[1]});
#pragma unroll
                    for (int t = 0; t < MR; ++t) o[t][n] = E::mfma(vf, pf[t], o[t][n]);
                }
            }
            lds_order();
        }
        if (more) take_sees();
    }

    // --- the sums over the four lanes of a row, then the result or this split's part
    const ArgsPtr c = args_again();
    const uint32_t nq = c->kv_heads * c->group, splits = c->splits;
    auto finish = [&](uint32_t row, uint32_t head, uint32_t d, f32x4 x, float mm, float ll) __attribute__((
                      always_inline)) {
        const uint64_t rh = (uint64_t)row * nq + head;
        if (splits == 1) {
            const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
            const u32x2 y = {E::pack(x[0] * inv, x[1] * inv), E::pack(x[2] * inv, x[3] * inv)};
            *reinterpret_cast<u32x2*>(c->out + rh * D + d) = y;
            if (d == 0 && c->lse)
                c->lse[rh] = ll > 0.f || ll != ll ? (mm + __builtin_amdgcn_logf(ll)) * kLn2 : -__builtin_inff();
        } else {
            *reinterpret_cast<f32x4*>(c->part + (rh * splits + split) * D + d) = x;
            if (d == 0) {
                c->part_ml[(rh * splits + split) * 2] = mm;
                c->part_ml[(rh * splits + split) * 2 + 1] = ll;
            }
        }
    };
#pragma unroll
    for (int t = 0; t < MR; ++t) {
        l[t] = sum_over_four(l[t]);
        if constexpr (SHARED) {
            uint32_t j;
            const uint32_t row = row_head(row0 + 16 * t + col, &j);
            if (q_row[t] != kNoPage) {
#pragma unroll
                for (int n = 0; n < DN; ++n) finish(row, h * a.group + j, 16 * n + 4 * g, o[t][n], m[t], l[t]);
            }
        } else {
            // the waves' rows joined through LDS: [wave][row][D + 4]
            float* const buf = reinterpret_cast<float*>(area);
            __syncthreads();
#pragma unroll
            for (int n = 0; n < DN; ++n)
                *reinterpret_cast<f32x4*>(buf + (wib * 16 + col) * (D + 4) + 16 * n + 4 * g) = o[t][n];
            if (g == 0) {
                join_m[wib][col] = m[t];
                join_l[wib][col] = l[t];
            }
            __syncthreads();
#pragma unroll 1
            for (uint32_t e = threadIdx.x; e < 16 * (D / 4); e += kWave * kAttnWaves) {
                const uint32_t cc = e / (D / 4), d = 4 * (e % (D / 4));
                const uint32_t rho = row0 + 16 * t + cc;
                if (rho >= rows) break;
                float mm = -__builtin_inff(), ll = 0.f;
#pragma unroll
                for (uint32_t w = 0; w < kAttnWaves; ++w) mm = fmaxf(mm, join_m[w][cc]);
                const float base = mm == -__builtin_inff() ? 0.f : mm;
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (uint32_t w = 0; w < kAttnWaves; ++w) {
                    const float f = __builtin_amdgcn_exp2f(join_m[w][cc] - base);
                    ll += f * join_l[w][cc];
                    x += f * *reinterpret_cast<const f32x4*>(buf + (w * 16 + cc) * (D + 4) + d);
                }
                uint32_t j;
                const uint32_t row = row_head(rho, &j);
                finish(row, h * a.group + j, d, x, mm, ll);
            }
        }
    }
    if constexpr (TREE) {
        // Drafted values that are infinite or NaN: added to what the rows
        // that see them have in memory.
        if (ballot(odd) && lane == 0) odd_values = 1;
        __syncthreads();
        if (odd_values) {
            const uint32_t j_lo = s_lo > ctx_steps ? (s_lo - ctx_steps) * STEP : 0u;
            const uint32_t j_hi = s_hi > ctx_steps ? min((s_hi - ctx_steps) * STEP, n_new) : 0u;
            const uint32_t n_rows = min(rows - rt * kRowsWg, kRowsWg);
            for (uint32_t e = threadIdx.x; e < n_rows * D; e += kWave * kAttnWaves) {
                const uint32_t d = e % D;
                uint32_t j;
                const uint32_t row = row_head(rt * kRowsWg + e / D, &j);
                float sum = 0.f;
                bool any = false;
                for (uint32_t k = j_lo; k < j_hi; ++k) {
                    if (!((c->mask[(uint64_t)row * c->mask_words2 + k / 32] >> (k % 32)) & 1u)) continue;
                    const uint32_t v = c->v_new[(int64_t)(first_row + k) * c->new_row + (int64_t)h * c->new_head + d];
                    if ((v & E::kExponent) != E::kExponent) continue;
                    sum += E::from_bits(v);
                    any = true;
                }
                if (!any) continue;
                const uint64_t rh = (uint64_t)row * nq + h * a.group + j;
                if (splits == 1)
                    c->out[rh * D + d] = (uint16_t)E::pack(E::from_bits(c->out[rh * D + d]) + sum, 0.f);
                else
                    c->part[(rh * splits + split) * D + d] += sum;
            }
        }
    }
}

// The splits' parts joined: D / 4 lanes per (row, head).
template <class E, int D>
__global__ __launch_bounds__(256) void k_join(AttnArgs a) {
    const uint32_t nq = a.kv_heads * a.group;
    const uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    const uint64_t rh = e / (D / 4);
    const uint32_t d = 4 * (uint32_t)(e % (D / 4));
    uint64_t rows = a.n_rows;
    if (a.new_rows) {
        const int64_t last = a.new_rows[a.n_seqs];
        rows = last < 0 ? 0 : min(rows, (uint64_t)last);
    }
    if (rh >= rows * nq) return;
    if (a.new_rows && a.new_rows[0] > 0 && rh < (uint64_t)a.new_rows[0] * nq) return;
    const float* ml = a.part_ml + rh * a.splits * 2;
    const float* part = a.part + rh * a.splits * D + d;
    float mm = -__builtin_inff(), ll = 0.f;
    for (uint32_t s = 0; s < a.splits; ++s) mm = fmaxf(mm, ml[2 * s]);
    const float base = mm == -__builtin_inff() ? 0.f : mm;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t s = 0; s < a.splits; ++s) {
        const float f = __builtin_amdgcn_exp2f(ml[2 * s] - base);
        ll += f * ml[2 * s + 1];
        x += f * *reinterpret_cast<const f32x4*>(part + (uint64_t)s * D);
    }
    const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
    const u32x2 y = {E::pack(x[0] * inv, x[1] * inv), E::pack(x[2] * inv, x[3] * inv)};
    *reinterpret_cast<u32x2*>(a.out + rh * D + d) = y;
    if (d == 0 && a.lse) a.lse[rh] = ll > 0.f || ll != ll ? (mm + __builtin_amdgcn_logf(ll)) * kLn2 : -__builtin_inff();
}

// Shape of a launch, chosen by the host (plan_attention).
struct AttnPlan {
    int mr = 1;              // tiles of 16 rows per wave
    bool shared = false;
    uint32_t step = 0;       // tokens per step
    uint32_t area_bytes = 0; // LDS besides the tables
    uint32_t row_tiles = 1, splits = 1;
};

hipError_t launch_attention_bf16(const AttnArgs& a, const AttnPlan& p, uint32_t head_dim, uint32_t page_tokens,
                                 bool tree, uint32_t lds, hipStream_t s);
hipError_t launch_attention_fp16(const AttnArgs& a, const AttnPlan& p, uint32_t head_dim, uint32_t page_tokens,
                                 bool tree, uint32_t lds, hipStream_t s);

template <class E, int D, int T, int MR, bool SHARED, bool TREE>
static hipError_t launch_attend(const AttnArgs& a, uint32_t lds, hipStream_t s) {
    if (lds > kMaxLdsPerBlock) {  // more than 64 KiB has to be asked for
        const hipError_t e =
            hipFuncSetAttribute(reinterpret_cast<const void*>(k_attend<E, D, T, MR, SHARED, TREE>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_attend<E, D, T, MR, SHARED, TREE>), dim3(a.splits * a.work * a.row_tiles),
                       dim3(kWave * kAttnWaves), lds, s, a);
    return hipGetLastError();
}

template <class E, int D, int T>
static hipError_t launch_attention_t(const AttnArgs& a, const AttnPlan& p, bool tree, uint32_t lds, hipStream_t s) {
    hipError_t e;
    constexpr int M2 = D <= 128 ? 2 : 1;  // 32 rows of 256 dims would not leave registers for two waves per SIMD
    if (!tree)
        e = p.mr == 1 ? launch_attend<E, D, T, 1, false, false>(a, lds, s)
                      : launch_attend<E, D, T, M2, false, false>(a, lds, s);
    else if (!p.shared)
        e = p.mr == 1 ? launch_attend<E, D, T, 1, false, true>(a, lds, s)
                      : launch_attend<E, D, T, M2, false, true>(a, lds, s);
    else
        e = p.mr == 1 ? launch_attend<E, D, T, 1, true, true>(a, lds, s)
                      : launch_attend<E, D, T, M2, true, true>(a, lds, s);
    if (e != hipSuccess || a.splits == 1) return e;
    const uint64_t threads = a.n_rows * a.kv_heads * a.group * (D / 4);
    hipLaunchKernelGGL((k_join<E, D>), dim3((uint32_t)((threads + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <class E>
static hipError_t launch_attention_e(const AttnArgs& a, const AttnPlan& p, uint32_t head_dim, uint32_t page_tokens,
                                     bool tree, uint32_t lds, hipStream_t s) {
    if (head_dim == 64 && page_tokens == 16) return launch_attention_t<E, 64, 16>(a, p, tree, lds, s);
    if (head_dim == 64 && page_tokens == 32) return launch_attention_t<E, 64, 32>(a, p, tree, lds, s);
    if (head_dim == 64 && page_tokens == 64) return launch_attention_t<E, 64, 64>(a, p, tree, lds, s);
    if (head_dim == 128 && page_tokens == 16) return launch_attention_t<E, 128, 16>(a, p, tree, lds, s);
    if (head_dim == 128 && page_tokens == 32) return launch_attention_t<E, 128, 32>(a, p, tree, lds, s);
    if (head_dim == 256 && page_tokens == 16) return launch_attention_t<E, 256, 16>(a, p, tree, lds, s);
    return hipErrorInvalidValue;
}

}  // namespace ibp
