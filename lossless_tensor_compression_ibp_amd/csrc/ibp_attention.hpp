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
// Two kernels:
//   k_attend_few, up to 16 MR rows.  Every wave walks pages of its own for all
//     rows, without a barrier, and the waves' results are joined at the end.
//     Bound by the pages' bytes, or by latency when there are few of them (16
//     streams of 4 K and 16 heads of 64 dims, 185 MB: 37 us, 5 TB/s; one of
//     1,000 tokens and 8 heads of 128 dims: 9.1 us and 4.0 to join; 512 rows
//     with 128 of 4,096 pages each, 4.3 GB out of the caches: 284 us, 15 TB/s).
//   k_attend_many.  Four waves with 16 MR rows each share a step's pages,
//     which they load and rebuild between them; two such workgroups on a
//     compute unit overlap one's rebuilding with the other's products.  (Eight
//     waves with two buffers and one barrier per step, measured: the waves
//     that rebuild hold up all others; eight streams of 24 drafted tokens over
//     8 K 140 us instead of 86, two 64 K contexts with 64 drafted tokens,
//     nothing to rebuild, 470 us instead of 420.)  With the join these now
//     take 88 and 379 us in calls queued one after another (405 us each in a
//     kernel trace), the latter 726 TFLOP/s, 0.6 of a large matrix product:
//     LDS (a step's operands, half of them as transposed 8-byte reads), the
//     products and the exponentials each work a quarter of the time, and wait
//     for each other.
// A long context is split over workgroups; k_join adds the parts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ibp_kv_math.hpp"

namespace ibp {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kFewWaves = 4;
constexpr uint32_t kManyWaves = 4;

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

// Sizes of the two kernels.  A token's row in LDS is padded so that the reads
// of 16 tokens (keys) and of four tokens at a time (values) spread over all
// banks.
template <int D, int T>
struct PageShape {
    static constexpr int NV = D * T / 512;                  // vectors per lane of a page
    static constexpr int U = 2;                             // steps of a rebuild taken together
    static constexpr int RK = 2 * D + 16, RV = 2 * D + 32;  // bytes per token row in LDS
    static constexpr uint32_t stage_bytes = 4 * page_stage_words<NV>();
    static_assert(stage_bytes % 16 == 0, "areas are vectors");
};

template <int D, int T>
struct FewShape : PageShape<D, T> {
    using P = PageShape<D, T>;
    static constexpr int STEP = T < 32 ? 32 : T;            // tokens per step of a wave
    static constexpr int PW = STEP / T;                     // pages of each kind
    static constexpr bool ONE = PW * P::NV > 8;             // one register buffer for keys and values in turn
    static constexpr uint32_t wave_bytes = PW * P::stage_bytes + STEP * P::RV;
    static constexpr uint32_t join_bytes = kFewWaves * 16 * (D + 4) * 4;
    static constexpr uint32_t area_bytes = kFewWaves * wave_bytes > join_bytes ? kFewWaves * wave_bytes : join_bytes;
};

template <int D, int T>
struct ManyShape : PageShape<D, T> {
    using P = PageShape<D, T>;
    static constexpr int STEP = 64;                         // tokens per step of the workgroup
    static constexpr int KP = STEP / T;                     // pages of each kind
    static constexpr bool BOTH = KP == kManyWaves;          // every wave has a page of each kind
    static constexpr int JOBS = BOTH ? KP : 2 * KP;         // waves that a step's pages take
    static constexpr int ROUNDS = kManyWaves / JOBS;        // a wave loads for every ROUNDS-th step
    static constexpr uint32_t tile_bytes = STEP * (P::RK + P::RV);
    static constexpr uint32_t area_bytes = tile_bytes + JOBS * P::stage_bytes;
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

// An error of the keys' pages, or of the values': those are latched on both
// handles, so that the keys' one stands for the whole call.
__device__ __forceinline__ void latch_page_error(bool values, uint32_t error) {
    const ArgsPtr c = args_again();
    atomicCAS(c->k.err, 0u, error);
    if (values) atomicCAS(c->v.err, 0u, error);
}

// What a workgroup works on.
struct Work {
    uint32_t split, h, item, rt;           // split, key/value head, sequence (tree) or row, row tile
    uint32_t seq, first_row, n_new, rows;  // rows: query heads of the group times drafted tokens (or one)
    int32_t len;
};

// False when there is nothing to do; what is not valid latches kErrRange.
template <int T, bool TREE>
__device__ __forceinline__ bool find_work(const AttnArgs& a, uint32_t rows_per_wg, Work& w) {
    w.split = blockIdx.x % a.splits;
    const uint32_t wg = (blockIdx.x / a.splits) % a.work;
    w.rt = blockIdx.x / a.splits / a.work;
    w.h = wg % a.kv_heads;
    w.item = wg / a.kv_heads;
    w.seq = w.item;
    w.first_row = TREE ? 0u : w.item;
    w.n_new = TREE ? 0u : 1u;
    w.len = a.lens[w.item];
    bool bad = w.len < 0 || (uint64_t)w.len > a.table_blocks * T;
    if (TREE) {
        const int32_t r0 = a.new_rows[w.item], r1 = a.new_rows[w.item + 1];
        const uint32_t n = (uint32_t)(r1 - r0);
        if (r0 < 0 || r1 < r0 || (uint64_t)r1 > a.n_rows || n > a.max_new || n > 32u * a.mask_words2) {
            bad = true;
        } else {
            w.first_row = (uint32_t)r0;
            w.n_new = n;
        }
    } else if (a.row_seq) {
        const int32_t s = a.row_seq[w.item];
        bad = bad || s < 0 || (uint64_t)s >= a.n_seqs;
        w.seq = (uint32_t)s;
    }
    if (bad) {
        latch_error(a.k.err, kErrRange);
        if (TREE) return false;
        w.seq = 0;
        w.len = 0;
    }
    w.rows = w.n_new * a.group;
    return w.rt * rows_per_wg < w.rows;
}

// The drafted token and query head of row rho of the group.
__device__ __forceinline__ uint32_t row_of_group(const AttnArgs& a, const Work& w, uint32_t rho, uint32_t* head) {
    const uint32_t i = rho / a.group;
    *head = w.h * a.group + (rho - i * a.group);
    return w.first_row + i;
}

// First vector per thread of each pool's tables, on its way while a wave
// finds its pages; and the tables' place in LDS.
struct EarlyTables {
    u32x4 k, v;
    __device__ __forceinline__ void load(const AttnArgs& a) {
        k = v = u32x4{0u, 0u, 0u, 0u};
        if (4 * threadIdx.x < a.tab_words_k) k = page_table_vector(a.k, threadIdx.x);
        if (4 * threadIdx.x < a.tab_words_v) v = page_table_vector(a.v, threadIdx.x);
    }
    __device__ __forceinline__ void put(const AttnArgs& a, uint32_t* smem) const {
        if (4 * threadIdx.x < a.tab_words_k) reinterpret_cast<u32x4*>(smem)[threadIdx.x] = k;
        if (4 * threadIdx.x < a.tab_words_v) reinterpret_cast<u32x4*>(smem + a.tab_words_k)[threadIdx.x] = v;
        if (a.tab_words_k > 4 * blockDim.x) stage_page_tables(a.k, smem, blockDim.x);
        if (a.tab_words_v > 4 * blockDim.x) stage_page_tables(a.v, smem + a.tab_words_k, blockDim.x);
    }
};

__device__ __forceinline__ PageTab kind_tab(const AttnArgs& a, const uint32_t* smem, bool values) {
    return page_tab(values ? a.v : a.k, smem + (values && !a.same_tab ? a.tab_words_k : 0u),
                    values ? a.tab_lds_v : a.tab_lds_k);
}

// One wave: T rows from token j0 of the drafted tokens' keys or values, as
// load_page lays out a page; rows past the last token read the last one.
template <int D, int NV>
__device__ __forceinline__ void load_drafted(u32x4* st, const Work& w, bool values, uint32_t j0) {
    const ArgsPtr c = args_again();
    const uint16_t* base = (values ? c->v_new : c->k_new) + (int64_t)w.h * c->new_head;
    const int64_t row = c->new_row;
#pragma unroll
    for (int r = 0; r < NV; ++r) {
        const uint32_t x = 256u * r + 4u * lane_id(), token = min(j0 + x / (D / 2), w.n_new - 1);
        st[r] = load_eight(base + (int64_t)(w.first_row + token) * row + 2 * (x % (D / 2)));
    }
}

// Words x of a page (four from word at) to its rows of tokens in LDS; tokens
// from n on become zero.
template <int D>
__device__ __forceinline__ void put_words(char* rows, int stride, uint32_t n, uint32_t at, u32x4 x) {
    const uint32_t token = at / (D / 2);
    if (token >= n) x = u32x4{0u, 0u, 0u, 0u};
    *reinterpret_cast<u32x4*>(rows + token * stride + 4 * (at % (D / 2))) = x;
}
template <int D, int T, int NV>
__device__ __forceinline__ void put_raw_page(const u32x4* st, char* rows, int stride, uint32_t n) {
    const uint32_t lane = lane_id();
    if (n == (uint32_t)T) {
#pragma unroll
        for (int r = 0; r < NV; ++r) put_words<D>(rows, stride, T, 256u * r + 4u * lane, st[r]);
    } else {
#pragma unroll
        for (int r = 0; r < NV; ++r) put_words<D>(rows, stride, n, 256u * r + 4u * lane, st[r]);
    }
}

// A wave's 16 MR rows: queries, running maximum, sum and output, and the
// scores of the TILES * 16 tokens at work.
template <class E, int D, int MR, int TILES>
struct Rows {
    using V8 = typename E::V8;
    static constexpr int DK = D / 32, DN = D / 16;
    V8 q[MR][DK];
    float m[MR], l[MR];
    f32x4 o[MR][DN];
    f32x4 s[MR][TILES];
    uint32_t row[MR];  // of this lane's column in q and the mask; kNoPage past the last row

    __device__ __forceinline__ void init(const AttnArgs& a, const Work& w, uint32_t row0) {
        const ArgsPtr c = args_again();
        const uint32_t col = lane_id() & 15u, g = lane_id() >> 4;
#pragma unroll
        for (int t = 0; t < MR; ++t) {
            const uint32_t rho = row0 + 16 * t + col;
            uint32_t head;
            row[t] = row_of_group(a, w, rho, &head);
            if (rho >= w.rows) row[t] = kNoPage;
            const uint16_t* p = c->q + (int64_t)row[t] * c->q_row + (int64_t)head * c->q_head;
#pragma unroll
            for (int kk = 0; kk < DK; ++kk) {
                u32x4 x = {0u, 0u, 0u, 0u};
                if (rho < w.rows) x = load_eight(p + 32 * kk + 8 * g);
                q[t][kk] = bits_as<V8>(x ^ c->q_sign);  // (a negative scale is taken into the queries)
            }
            m[t] = -__builtin_inff();
            l[t] = 0.f;
#pragma unroll
            for (int n = 0; n < DN; ++n) o[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }

    // S^T = K Q^T
    __device__ __forceinline__ void scores(const char* keys, int stride) {
        const uint32_t col = lane_id() & 15u, g = lane_id() >> 4;
#pragma unroll
        for (int kk = 0; kk < DK; ++kk) {
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                const V8 kf = *reinterpret_cast<const V8*>(keys + (16 * u + col) * stride + 64 * kk + 16 * g);
#pragma unroll
                for (int t = 0; t < MR; ++t)
                    s[t][u] = E::mfma(kf, q[t][kk], kk ? s[t][u] : f32x4{0.f, 0.f, 0.f, 0.f});
            }
        }
    }

    // Scores of row tile t, tile u that bit j of `seen` does not have: -infinity.
    __device__ __forceinline__ void mask(int t, int u, uint32_t seen) {
        const uint32_t g = lane_id() >> 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][u][e] = (seen >> (4 * g + e)) & 1u ? s[t][u][e] : -__builtin_inff();
    }

    // Scores in octaves, and their running maximum.  The maximum, less
    // E::kLead, is the exponent m that weights are taken against:
    // exp2(score - m).  It is moved only when a score passes it by more than
    // kLead + 8 (weights then stay below 2^(kLead + 8) and sums far from
    // overflow), so most steps rescale nothing; one branch for all rows leaves
    // the rest of a step in one block, where the compiler can run weights
    // beside products.  Scores are scaled and rounded here, before the maximum
    // is taken off: with both in one multiply-add the highest score would
    // differ from the maximum by up to half a step of 32 bits, which past 2^31
    // octaves is more than a weight can hold.
    //
    // The weights are rounded to the data's type, once, for the matrix product
    // with the values; their sum l takes them unrounded, in 32 bits.  (The
    // matrix cores do a sixteenth of the products in 32 bits, and weights split
    // in two 16-bit parts would take twice as many.)  Each is off by half a
    // step at most, 2^-8 or 2^-11 of its value, which moves a row by that share
    // of its mean |v| at most.  bf16 has the range of 32 bits.  In fp16 numbers
    // below 2^-14 have steps of 2^-24, so with a largest weight of 1 a key 25
    // octaves below it would weigh nothing here but count in l, and a long
    // context of such keys is not nothing (65,535 of them: 0.2 %).  With 2^7
    // to 2^15 for the largest weight a key loses at most 2^-32 of it.
    __device__ __forceinline__ void raise(float scale2) {
        float top[MR];
        bool move = false;
#pragma unroll
        for (int t = 0; t < MR; ++t) {
            float x[TILES];
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                s[t][u] *= scale2;
                x[u] = fmaxf(fmaxf(s[t][u][0], s[t][u][1]), fmaxf(s[t][u][2], s[t][u][3]));
            }
            top[t] = x[0];
#pragma unroll
            for (int u = 1; u < TILES; ++u) top[t] = fmaxf(top[t], x[u]);
            top[t] = max_over_four(top[t]);
            move = move || top[t] - m[t] > E::kLead + 8.f;  // (also the first one, from -infinity)
        }
        if (ballot(move)) {
#pragma unroll
            for (int t = 0; t < MR; ++t) {
                const float m_new = fmaxf(m[t], top[t] - E::kLead);
                const float f = m_new == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(m[t] - m_new);
                m[t] = m_new;
                l[t] *= f;
#pragma unroll
                for (int n = 0; n < DN; ++n) o[t][n] *= f;
            }
        }
    }

    // Weights, their sum, and O^T += V^T P^T, two tiles of tokens at a time.
    __device__ __forceinline__ void values(const char* vals, int stride) {
#pragma clang fp contract(off)  // (scores stay rounded, see above)
        const uint32_t col = lane_id() & 15u, g = lane_id() >> 4;
        float base[MR];
#pragma unroll
        for (int t = 0; t < MR; ++t) base[t] = m[t] == -__builtin_inff() ? 0.f : -m[t];
#pragma unroll
        for (int u = 0; u < TILES; u += 2) {
            V8 p[MR];
#pragma unroll
            for (int t = 0; t < MR; ++t) {
#pragma unroll
                for (int v = u; v < u + 2; ++v) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[t][v][e] = __builtin_amdgcn_exp2f(s[t][v][e] + base[t]);
                    l[t] += (s[t][v][0] + s[t][v][1]) + (s[t][v][2] + s[t][v][3]);
                }
                const u32x4 x = {E::pack(s[t][u][0], s[t][u][1]), E::pack(s[t][u][2], s[t][u][3]),
                                 E::pack(s[t][u + 1][0], s[t][u + 1][1]), E::pack(s[t][u + 1][2], s[t][u + 1][3])};
                p[t] = bits_as<V8>(x);
            }
            const char* at = vals + (16 * u + 4 * g + (col >> 2)) * stride + 8 * (col & 3);
#pragma unroll
            for (int n = 0; n < DN; ++n) {
                const u32x2 x = read_transposed(at + 32 * n), y = read_transposed(at + 16 * stride + 32 * n);
                const V8 vf = bits_as<V8>(u32x4{x[0], x[1], y[0], y[1]});
#pragma unroll
                for (int t = 0; t < MR; ++t) o[t][n] = E::mfma(vf, p[t], o[t][n]);
            }
        }
    }
};

// Whether a row has any weight (or a NaN for one).  Without one it is zeros,
// whatever the values are that weighed nothing.
__device__ __forceinline__ bool has_weight(float l) { return l > 0.f || l != l; }

// Four dims of a row whose weights are l: the quotient in the data's type.
template <class E>
__device__ __forceinline__ u32x2 row_of(f32x4 x, float l) {
    const float inv = 1.f / l;
    const u32x2 y = {E::pack(x[0] * inv, x[1] * inv), E::pack(x[2] * inv, x[3] * inv)};
    return has_weight(l) ? y : u32x2{0u, 0u};
}

// Four dims of a row: the result, or this split's part of it.
template <class E, int D>
__device__ __forceinline__ void put_result(ArgsPtr c, uint32_t split, uint32_t row, uint32_t head, uint32_t d, f32x4 x,
                                           float m, float l) {
    const uint64_t rh = (uint64_t)row * (c->kv_heads * c->group) + head;
    if (c->splits == 1) {
        *reinterpret_cast<u32x2*>(c->out + rh * D + d) = row_of<E>(x, l);
        if (d == 0 && c->lse)
            c->lse[rh] = has_weight(l) ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -__builtin_inff();
    } else {
        *reinterpret_cast<f32x4*>(c->part + (rh * c->splits + split) * D + d) = x;
        if (d == 0) {
            c->part_ml[(rh * c->splits + split) * 2] = m;
            c->part_ml[(rh * c->splits + split) * 2 + 1] = l;
        }
    }
}

// Whole workgroup, after its results are in memory: drafted values j_lo ..
// j_hi - 1 that are infinite or NaN, added to the rows that see them.  (They
// were taken out of the products, where they would have reached every row
// through a weight of zero.)  weighed: of the workgroup's rows, those that have
// a weight; of parts, k_join knows.
template <class E, int D>
__device__ __forceinline__ void add_odd_values(const AttnArgs& a, const Work& w, uint32_t rows_per_wg,
                                               const bool* weighed, uint32_t j_lo, uint32_t j_hi) {
    const ArgsPtr c = args_again();
    const uint32_t n_rows = min(w.rows - w.rt * rows_per_wg, rows_per_wg);
#pragma unroll 1
    for (uint32_t e = threadIdx.x; e < n_rows * D; e += blockDim.x) {
        const uint32_t d = e % D;
        if (c->splits == 1 && !weighed[e / D]) continue;
        uint32_t head;
        const uint32_t row = row_of_group(a, w, w.rt * rows_per_wg + e / D, &head);
        float sum = 0.f;
        bool any = false;
#pragma unroll 1
        for (uint32_t k = j_lo; k < j_hi; ++k) {
            if (!((c->mask[(uint64_t)row * c->mask_words2 + k / 32] >> (k % 32)) & 1u)) continue;
            const uint32_t v = c->v_new[(int64_t)(w.first_row + k) * c->new_row + (int64_t)w.h * c->new_head + d];
            if ((v & E::kExponent) != E::kExponent) continue;
            sum += E::from_bits(v);
            any = true;
        }
        if (!any) continue;
        const uint64_t rh = (uint64_t)row * (c->kv_heads * c->group) + head;
        if (c->splits == 1)
            c->out[rh * D + d] = (uint16_t)E::pack(E::from_bits(c->out[rh * D + d]) + sum, 0.f);
        else
            c->part[(rh * c->splits + w.split) * D + d] += sum;
    }
}

// The step that covers tokens 0 .. n - 1 of 16 TILES from its first: bit j of
// tile u's tokens.
__device__ __forceinline__ uint32_t tile_bits(uint32_t n, int u) {
    const uint32_t k = n > 16u * u ? n - 16u * u : 0u;
    return k >= 16u ? 0xFFFFu : (1u << k) - 1u;
}

// Mask words of drafted tokens 32 word .. for a lane's rows.
template <int MR, int WORDS>
__device__ __forceinline__ void load_sees(uint32_t (&sees)[MR][WORDS], const uint32_t (&row)[MR], uint32_t word) {
    const ArgsPtr c = args_again();
#pragma unroll
    for (int t = 0; t < MR; ++t) {
#pragma unroll
        for (int x = 0; x < WORDS; ++x) {
            sees[t][x] = 0;
            if (row[t] != kNoPage && word + x < c->mask_words2)
                sees[t][x] = c->mask[(uint64_t)row[t] * c->mask_words2 + word + x];
        }
    }
}

template <class E, int D, int T, int MR, bool TREE>
__global__ __launch_bounds__(kWave * kFewWaves, 2) void k_attend_few(AttnArgs a) {
    using S = FewShape<D, T>;
    constexpr int NV = S::NV, STEP = S::STEP, PW = S::PW, TILES = STEP / 16, DN = D / 16;
    constexpr uint32_t kRowsWg = 16u * MR;
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ float join_m[kFewWaves][16], join_l[kFewWaves][16];
    __shared__ uint32_t odd_values;  // an infinity or NaN among the drafted values
    __shared__ bool weighed[kRowsWg];
    const uint32_t lane = lane_id(), wib = uniform(threadIdx.x / kWave);
    const uint32_t col = lane & 15u, g = lane >> 4;

    EarlyTables tables;
    tables.load(a);
    if (TREE && threadIdx.x == 0) odd_values = 0;
    Work w;
    if (!find_work<T, TREE>(a, kRowsWg, w)) return;
    const uint32_t row0 = w.rt * kRowsWg;

    // steps of this split: the context's, then the drafted tokens'
    const uint32_t ctx_pages = TREE ? ((uint32_t)w.len + T - 1) / T : (w.len > 0 ? a.n_list : 0u);
    const uint32_t ctx_steps = (ctx_pages + PW - 1) / PW;
    const uint32_t all_steps = ctx_steps + (TREE ? (w.n_new + STEP - 1) / STEP : 0u);
    const uint32_t per = (all_steps + a.splits - 1) / a.splits;
    const uint32_t s_lo = min(w.split * per, all_steps), s_hi = min(s_lo + per, all_steps);
    const uint32_t s_first = s_lo + wib;
    const uint32_t n_steps = s_first < s_hi ? (s_hi - s_first + kFewWaves - 1) / kFewWaves : 0u;

    char* const area = reinterpret_cast<char*>(smem + a.tab_words_k + a.tab_words_v);
    uint32_t* const stage = reinterpret_cast<uint32_t*>(area + wib * S::wave_bytes);
    char* const tile = reinterpret_cast<char*>(stage) + PW * S::stage_bytes;  // keys, then values

    Rows<E, D, MR, TILES> rows;
    rows.init(a, w, row0);

    // --- the wave's next pages: lane l has page l % PW of its step base + l / PW
    uint32_t id_k = 0, id_v = 0, held = 0, comp = 0;
    auto refill = [&](uint32_t base) __attribute__((always_inline)) {
        const ArgsPtr c = args_again();
        const uint32_t s = s_first + (base + lane / PW) * kFewWaves;
        id_k = id_v = held = comp = 0;
        if (s < s_hi && s < ctx_steps) {
            const uint32_t n = s * PW + lane % PW;
            int32_t block = n < ctx_pages ? (int32_t)n : -1;
            if (!TREE && n < ctx_pages) block = c->blocks[((uint64_t)w.item * a.kv_heads + w.h) * c->n_list + n];
            if (block >= 0 && (int64_t)block * T < w.len) {
                held = (uint32_t)min(T, w.len - block * T);
                const uint64_t at = ((uint64_t)w.seq * a.kv_heads + w.h) * c->table_blocks + (uint32_t)block;
                // both ids, then both bits, each pair in one latency
                const int64_t k64 = c->k_table[at], v64 = c->v_table[at];
                const uint32_t k = page_id(k64, c->k.n_slots), v = page_id(v64, c->v.n_slots);
                id_k = k == kNoPage ? 0u : k;
                id_v = v == kNoPage ? 0u : v;
                const uint32_t k_word = c->k.bitmask[id_k >> 5], v_word = c->v.bitmask[id_v >> 5];
                comp = (k == kNoPage ? 0u : (k_word >> (id_k & 31u)) & 1u) |
                       (v == kNoPage ? 0u : ((v_word >> (id_v & 31u)) & 1u) << 1);
                if (k == kNoPage || v == kNoPage) latch_page_error(v == kNoPage, kErrRange);
            }
        }
    };
    auto load = [&](u32x4* st, uint32_t j, bool values, uint32_t ids) __attribute__((always_inline)) {
        const uint32_t s = s_first + j * kFewWaves;
#pragma unroll
        for (int p = 0; p < PW; ++p) {
            if (!TREE || s < ctx_steps)
                load_page<NV>(st + p * NV, values ? a.v.slots : a.k.slots,
                              lane_value(ids, (int)((j % (64 / PW)) * PW + p)));
            else
                load_drafted<D, NV>(st + p * NV, w, values, (s - ctx_steps) * STEP + p * T);
        }
    };
    // The wave's pages as rows of tokens in LDS.  A record goes through the
    // stage; values behind a page's last token become zero.
    auto put = [&](const u32x4* st, bool values, uint32_t records, const uint32_t* keep) __attribute__((
                   always_inline)) {
        const int stride = values ? S::RV : S::RK;
        lds_order();
#pragma unroll
        for (int p = 0; p < PW; ++p) {
            if ((records >> p) & 1u)
                stage_page<NV>(st + p * NV, stage + p * (S::stage_bytes / 4));
            else
                put_raw_page<D, T, NV>(st + p * NV, tile + p * T * stride, stride, values ? keep[p] : (uint32_t)T);
        }
        for (; records; records &= records - 1) {
            const uint32_t p = PW == 1 ? 0u : (uint32_t)__builtin_ctz(records);
            const uint32_t n = !values ? (uint32_t)T : PW == 1 || p == 0 ? keep[0] : keep[PW - 1];
            if (!rebuild_page<NV, S::U>(values ? a.v : a.k, kind_tab(a, smem, values),
                                        stage + p * (S::stage_bytes / 4),
                                        [&](uint32_t at, u32x4 x) __attribute__((always_inline)) {
                                            put_words<D>(tile + p * T * stride, stride, n, at, x);
                                        }))
                if (lane == 0) latch_page_error(values, kErrCorrupt);
        }
        lds_order();
    };

    u32x4 st_a[PW * NV], st_b[S::ONE ? 1 : PW * NV];
    bool odd = false;
    // of the step at work and of the next: tokens of each page, and the rows'
    // mask words of drafted steps; which pages at work are records (keys, then
    // values); ids of the value pages at work (ONE)
    uint32_t n_held[PW], next_held[PW], records = 0, ids_v = 0;
    uint32_t sees[MR][STEP / 32], next_sees[MR][STEP / 32];
    auto facts = [&](uint32_t j) __attribute__((always_inline)) {
        const uint32_t sn = s_first + j * kFewWaves;
        const bool drafted = TREE && sn >= ctx_steps;
#pragma unroll
        for (int p = 0; p < PW; ++p) {
            next_held[p] = lane_value(held, (int)((j % (64 / PW)) * PW + p));
            if (drafted) {
                const uint32_t j0 = (sn - ctx_steps) * STEP + p * T;
                next_held[p] = w.n_new > j0 ? min(w.n_new - j0, (uint32_t)T) : 0u;
            }
        }
        if (drafted) load_sees(next_sees, rows.row, (sn - ctx_steps) * (STEP / 32));
    };
    // step j becomes the one at work (after its loads have been sent: the
    // records' bits come a latency after the ids)
    auto advance = [&](uint32_t j) __attribute__((always_inline)) {
        records = 0;
        ids_v = id_v;
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
                for (int x = 0; x < STEP / 32; ++x) sees[t][x] = next_sees[t][x];
            }
        }
    };
#pragma unroll
    for (int t = 0; t < MR; ++t) {
#pragma unroll
        for (int x = 0; x < STEP / 32; ++x) sees[t][x] = next_sees[t][x] = 0;
    }
    if (n_steps) {
        refill(0);
        facts(0);
        load(st_a, 0, false, id_k);
        if constexpr (!S::ONE) load(st_b, 0, true, id_v);
    }
    tables.put(a, smem);
    if (n_steps) {
        advance(0);
        take_sees();
    }
    __syncthreads();

    for (uint32_t i = 0; i < n_steps; ++i) {
        const bool more = i + 1 < n_steps;
        const uint32_t s = s_first + i * kFewWaves;
        const bool draft = TREE && s >= ctx_steps;
        put(st_a, false, records & ((1u << PW) - 1), n_held);
        uint32_t tokens[PW];  // of the pages at work, for the masks
        bool whole = !draft;
#pragma unroll
        for (int p = 0; p < PW; ++p) {
            tokens[p] = n_held[p];
            whole = whole && n_held[p] == (uint32_t)T;
        }
        if constexpr (S::ONE) load(st_a, i, true, ids_v);
        if (more) {
            if ((i + 1) % (64 / PW) == 0) refill(i + 1);
            facts(i + 1);
            if constexpr (!S::ONE) load(st_a, i + 1, false, id_k);
        }
        rows.scores(tile, S::RK);
        if (!whole) {
#pragma unroll
            for (int t = 0; t < MR; ++t) {
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
                    uint32_t seen = tile_bits(tokens[16 * u / T], u - 16 * u / T * (T / 16));
                    if (draft) seen &= sees[t][u / 2] >> (16 * (u & 1));
                    rows.mask(t, u, seen);
                }
            }
        }
        rows.raise(a.scale2);
        u32x4* const st_v = S::ONE ? st_a : st_b;
        if (draft) {
#pragma unroll
            for (int r = 0; r < PW * NV; ++r) odd |= clear_odd<E>(st_v[r]);
        }
        put(st_v, true, records >> PW, n_held);
        if (more) {
            if constexpr (S::ONE)
                load(st_a, i + 1, false, id_k);
            else
                load(st_b, i + 1, true, id_v);
            advance(i + 1);
        }
        rows.values(tile, S::RV);
        lds_order();
        if (more) take_sees();
    }

    // --- the waves' rows joined through LDS: [wave][row][D + 4]
    const ArgsPtr c = args_again();
#pragma unroll
    for (int t = 0; t < MR; ++t) {
        const float l = sum_over_four(rows.l[t]);
        float* const buf = reinterpret_cast<float*>(area);
        __syncthreads();
#pragma unroll
        for (int n = 0; n < DN; ++n)
            *reinterpret_cast<f32x4*>(buf + (wib * 16 + col) * (D + 4) + 16 * n + 4 * g) = rows.o[t][n];
        if (g == 0) {
            join_m[wib][col] = rows.m[t];
            join_l[wib][col] = l;
        }
        __syncthreads();
#pragma unroll 1
        for (uint32_t e = threadIdx.x; e < 16 * (D / 4); e += kWave * kFewWaves) {
            const uint32_t r = e / (D / 4), d = 4 * (e % (D / 4));
            const uint32_t rho = row0 + 16 * t + r;
            if (rho >= w.rows) break;
            float mm = -__builtin_inff(), ll = 0.f;
#pragma unroll
            for (uint32_t v = 0; v < kFewWaves; ++v) mm = fmaxf(mm, join_m[v][r]);
            const float base = mm == -__builtin_inff() ? 0.f : mm;
            f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (uint32_t v = 0; v < kFewWaves; ++v) {
                const float f = __builtin_amdgcn_exp2f(join_m[v][r] - base);
                ll += f * join_l[v][r];
                x += f * *reinterpret_cast<const f32x4*>(buf + (v * 16 + r) * (D + 4) + d);
            }
            uint32_t head;
            const uint32_t row = row_of_group(a, w, rho, &head);
            put_result<E, D>(c, w.split, row, head, d, x, mm, ll);
            if (TREE && d == 0) weighed[16 * t + r] = has_weight(ll);
        }
    }
    if constexpr (TREE) {
        if (ballot(odd) && lane == 0) odd_values = 1;
        __syncthreads();
        if (odd_values)
            add_odd_values<E, D>(a, w, kRowsWg, weighed, s_lo > ctx_steps ? (s_lo - ctx_steps) * STEP : 0u,
                                 s_hi > ctx_steps ? min((s_hi - ctx_steps) * STEP, w.n_new) : 0u);
    }
}

template <class E, int D, int T, int MR>
__global__ __launch_bounds__(kWave * kManyWaves, 2) void k_attend_many(AttnArgs a) {
    using S = ManyShape<D, T>;
    constexpr int NV = S::NV, STEP = S::STEP, TILES = STEP / 16, DN = D / 16;
    constexpr uint32_t kRowsWg = 16u * MR * kManyWaves;
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ uint32_t odd_values;  // an infinity or NaN among the drafted values
    __shared__ bool weighed[kRowsWg];
    const uint32_t lane = lane_id(), wib = uniform(threadIdx.x / kWave);
    const uint32_t col = lane & 15u, g = lane >> 4;

    EarlyTables tables;
    tables.load(a);
    if (threadIdx.x == 0) odd_values = 0;
    Work w;
    if (!find_work<T, true>(a, kRowsWg, w)) return;

    const uint32_t ctx_steps = ((uint32_t)w.len + STEP - 1) / STEP;
    const uint32_t all_steps = ctx_steps + (w.n_new + STEP - 1) / STEP;
    const uint32_t per = (all_steps + a.splits - 1) / a.splits;
    const uint32_t s_lo = min(w.split * per, all_steps), s_hi = min(s_lo + per, all_steps);

    // this wave's page of every ROUNDS-th step: of keys and values, or of one
    const uint32_t job = wib % S::JOBS, phase = wib / S::JOBS;
    const bool only_v = !S::BOTH && job >= (uint32_t)S::KP;
    const uint32_t page = only_v ? job - S::KP : job;
    char* const area = reinterpret_cast<char*>(smem + a.tab_words_k + a.tab_words_v);
    uint32_t* const stage = reinterpret_cast<uint32_t*>(area + S::tile_bytes + job * S::stage_bytes);

    // lane l: ids and bits (keys, then values) of the wave's page of its own
    // step base + l
    uint32_t id_k = 0, id_v = 0, comp = 0;
    auto refill = [&](uint32_t base) __attribute__((always_inline)) {
        const ArgsPtr c = args_again();
        const uint32_t s = s_lo + phase + (base + lane) * S::ROUNDS;
        const uint32_t block = s * S::KP + page;
        id_k = id_v = comp = 0;
        if (s < s_hi && s < ctx_steps && block * T < (uint32_t)w.len) {
            const uint64_t at = ((uint64_t)w.seq * a.kv_heads + w.h) * c->table_blocks + block;
            // both ids, then both bits, each pair in one latency
            const int64_t k64 = c->k_table[at], v64 = c->v_table[at];
            const uint32_t k = page_id(k64, c->k.n_slots), v = page_id(v64, c->v.n_slots);
            id_k = k == kNoPage ? 0u : k;
            id_v = v == kNoPage ? 0u : v;
            const uint32_t k_word = c->k.bitmask[id_k >> 5], v_word = c->v.bitmask[id_v >> 5];
            comp = (k == kNoPage ? 0u : (k_word >> (id_k & 31u)) & 1u) |
                   (v == kNoPage ? 0u : ((v_word >> (id_v & 31u)) & 1u) << 1);
            if (k == kNoPage || v == kNoPage) latch_page_error(v == kNoPage, kErrRange);
        }
    };
    u32x4 st_a[NV], st_b[S::BOTH ? NV : 1];
    bool odd = false;
    uint32_t k = 0;  // own steps loaded so far
    auto load = [&]() __attribute__((always_inline)) {
        const uint32_t s = s_lo + phase + k * S::ROUNDS;
        if (s >= s_hi) return;
        if (k % 64 == 0) refill(k);
        if (s < ctx_steps) {
            load_page<NV>(st_a, only_v ? a.v.slots : a.k.slots, lane_value(only_v ? id_v : id_k, (int)(k % 64)));
            if constexpr (S::BOTH) load_page<NV>(st_b, a.v.slots, lane_value(id_v, (int)(k % 64)));
        } else {
            load_drafted<D, NV>(st_a, w, only_v, (s - ctx_steps) * STEP + page * T);
            if constexpr (S::BOTH) load_drafted<D, NV>(st_b, w, true, (s - ctx_steps) * STEP + page * T);
        }
        ++k;
    };
    // a page of step s to its rows of tokens in LDS; values behind the last
    // token become zero
    auto put = [&](u32x4* st, bool values, uint32_t s) __attribute__((always_inline)) {
        const int stride = values ? S::RV : S::RK;
        char* const to = area + (values ? STEP * S::RK : 0) + page * T * stride;
        const bool drafted = s >= ctx_steps;
        const uint32_t first = (drafted ? s - ctx_steps : s) * STEP + page * T;
        const uint32_t end = drafted ? w.n_new : (uint32_t)w.len;
        const uint32_t held = !values ? (uint32_t)T : end > first ? min(end - first, (uint32_t)T) : 0u;
        if (drafted && values) {
#pragma unroll
            for (int r = 0; r < NV; ++r) odd |= clear_odd<E>(st[r]);
        }
        lds_order();
        if (!drafted && ((lane_value(comp, (int)((k - 1) % 64)) >> (values ? 1 : 0)) & 1u)) {
            stage_page<NV>(st, stage);
            if (!rebuild_page<NV, S::U>(values ? a.v : a.k, kind_tab(a, smem, values), stage,
                                        [&](uint32_t at, u32x4 x) __attribute__((always_inline)) {
                                            put_words<D>(to, stride, held, at, x);
                                        }))
                if (lane == 0) latch_page_error(values, kErrCorrupt);
        } else {
            put_raw_page<D, T, NV>(st, to, stride, held);
        }
        lds_order();
    };

    load();
    Rows<E, D, MR, TILES> rows;
    rows.init(a, w, w.rt * kRowsWg + wib * 16u * MR);
    tables.put(a, smem);

    for (uint32_t s = s_lo; s < s_hi; ++s) {
        const bool draft = s >= ctx_steps;
        uint32_t sees[MR][STEP / 32];
        if (draft) load_sees(sees, rows.row, (s - ctx_steps) * (STEP / 32));
        __syncthreads();  // the tiles are free, and the tables there
        if (S::ROUNDS == 1 || (s - s_lo) % S::ROUNDS == phase) {
            if constexpr (S::BOTH) {
                put(st_a, false, s);
                put(st_b, true, s);
            } else {
                if (only_v)
                    put(st_a, true, s);
                else
                    put(st_a, false, s);
            }
            load();
        }
        __syncthreads();
        const uint32_t tokens = draft ? w.n_new - (s - ctx_steps) * STEP : (uint32_t)w.len - s * STEP;
        rows.scores(area, S::RK);
        if (draft || tokens < (uint32_t)STEP) {
#pragma unroll
            for (int t = 0; t < MR; ++t) {
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
                    uint32_t seen = tile_bits(tokens, u);
                    if (draft) seen &= sees[t][u / 2] >> (16 * (u & 1));
                    rows.mask(t, u, seen);
                }
            }
        }
        rows.raise(a.scale2);
        rows.values(area + STEP * S::RK, S::RV);
    }

    const ArgsPtr c = args_again();
#pragma unroll
    for (int t = 0; t < MR; ++t) {
        const float l = sum_over_four(rows.l[t]);
        uint32_t head;
        const uint32_t row = row_of_group(a, w, w.rt * kRowsWg + (wib * MR + t) * 16u + col, &head);
        if (rows.row[t] != kNoPage) {
#pragma unroll
            for (int n = 0; n < DN; ++n)
                put_result<E, D>(c, w.split, row, head, 16 * n + 4 * g, rows.o[t][n], rows.m[t], l);
            if (g == 0) weighed[(wib * MR + t) * 16u + col] = has_weight(l);
        }
    }
    if (ballot(odd) && lane == 0) odd_values = 1;
    __syncthreads();
    if (odd_values)
        add_odd_values<E, D>(a, w, kRowsWg, weighed, s_lo > ctx_steps ? (s_lo - ctx_steps) * STEP : 0u,
                             s_hi > ctx_steps ? min((s_hi - ctx_steps) * STEP, w.n_new) : 0u);
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
    // Lane j of the row's takes the maximum and sum of split j (and j + D / 4,
    // ...), so that they arrive in one latency; then four splits' numbers at a
    // time.
    constexpr int W = D / 4;
    const float* ml = a.part_ml + rh * a.splits * 2;
    const float* part = a.part + rh * a.splits * D + d;
    const uint32_t lane = (uint32_t)(e % W);
    float mm = -__builtin_inff(), ll = 0.f;
    for (uint32_t s = lane; s < a.splits; s += W) mm = fmaxf(mm, ml[2 * s]);
    for (int o = W / 2; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor(mm, o));
    const float base = mm == -__builtin_inff() ? 0.f : mm;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t s0 = 0; s0 < a.splits; s0 += W) {
        float f = 0.f;
        if (s0 + lane < a.splits) {
            f = __builtin_amdgcn_exp2f(ml[2 * (s0 + lane)] - base);
            ll += f * ml[2 * (s0 + lane) + 1];
        }
        const uint32_t n = min(a.splits - s0, (uint32_t)W);
        for (uint32_t s = 0; s < n; s += 4) {
            f32x4 y[4];
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u)
                y[u] = *reinterpret_cast<const f32x4*>(part + (uint64_t)(s0 + min(s + u, n - 1)) * D);
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
                const float g = __shfl(f, (int)(threadIdx.x - lane + s + u) & 63);
                if (s + u < n) x += g * y[u];
            }
        }
    }
    for (int o = W / 2; o > 0; o >>= 1) ll += __shfl_xor(ll, o);
    *reinterpret_cast<u32x2*>(a.out + rh * D + d) = row_of<E>(x, ll);
    if (d == 0 && a.lse) a.lse[rh] = has_weight(ll) ? (mm + __builtin_amdgcn_logf(ll)) * kLn2 : -__builtin_inff();
}

// Shape of a launch, chosen by the host (plan_attention).
struct AttnPlan {
    int mr = 1;              // tiles of 16 rows per wave
    bool many = false;       // k_attend_many
    uint32_t step = 0;       // tokens per step
    uint32_t area_bytes = 0; // LDS besides the tables
    uint32_t row_tiles = 1, splits = 1;
};

hipError_t launch_attention_bf16(const AttnArgs& a, const AttnPlan& p, uint32_t head_dim, uint32_t page_tokens,
                                 bool tree, uint32_t lds, hipStream_t s);
hipError_t launch_attention_fp16(const AttnArgs& a, const AttnPlan& p, uint32_t head_dim, uint32_t page_tokens,
                                 bool tree, uint32_t lds, hipStream_t s);

constexpr uint64_t kLdsLimit = kLdsPerCu - 2048;  // of dynamic LDS: the kernels' static arrays aside

// More than 64 KiB of LDS has to be asked for, once per kernel and device (the
// call costs about as much as a launch).
template <auto kernel>
static hipError_t launch_attend(const AttnArgs& a, uint32_t waves, uint32_t lds, hipStream_t s) {
    static std::atomic<uint64_t> asked{0};
    if (lds > kMaxLdsPerBlock) {
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        const uint64_t bit = 1ull << (dev & 63);
        if (e == hipSuccess && !(asked.load(std::memory_order_relaxed) & bit)) {
            e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kLdsLimit);
            if (e == hipSuccess && dev < 64) asked.fetch_or(bit, std::memory_order_relaxed);
        }
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3(a.splits * a.work * a.row_tiles), dim3(kWave * waves), lds, s, a);
    return hipGetLastError();
}

template <class E, int D, int T>
static hipError_t launch_attention_t(const AttnArgs& a, const AttnPlan& p, bool tree, uint32_t lds, hipStream_t s) {
    hipError_t e;
    constexpr int M2 = D <= 128 ? 2 : 1;  // 32 rows of 256 dims would not leave registers for two waves per SIMD
    if (!tree)
        e = p.mr == 1 ? launch_attend<k_attend_few<E, D, T, 1, false>>(a, kFewWaves, lds, s)
                      : launch_attend<k_attend_few<E, D, T, M2, false>>(a, kFewWaves, lds, s);
    else if (!p.many)
        e = p.mr == 1 ? launch_attend<k_attend_few<E, D, T, 1, true>>(a, kFewWaves, lds, s)
                      : launch_attend<k_attend_few<E, D, T, M2, true>>(a, kFewWaves, lds, s);
    else
        e = p.mr == 1 ? launch_attend<k_attend_many<E, D, T, 1>>(a, kManyWaves, lds, s)
                      : launch_attend<k_attend_many<E, D, T, M2>>(a, kManyWaves, lds, s);
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
