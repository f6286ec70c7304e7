// ibp_kv_device.hpp -- what the page operators (copying, bounds, attention)
// share on the device: a pool of pages, the load of one page by one wave, and
// its rebuild in registers when the slot holds a record.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ibp_device.hpp"
#include "ibp_internal.hpp"

namespace ibp {

constexpr uint32_t kNoPage = 0xFFFFFFFFu;
constexpr uint64_t kMaxPoolSlots = 0xFFFFFFFEull;  // page ids are held in 32 bits
constexpr uint64_t kMaxPageBytes = 4ull * kMaxTileWords;

// A pool of pages as a kernel sees it.  The tables are those of the handle;
// a position of the period holds Mask/Bitval's word and what the rebuild
// needs of it (Tables).
struct Pool {
    const uint8_t* slots;
    const uint32_t* bitmask;
    uint32_t* err;
    Tables t;
    uint32_t n_slots;
    uint32_t Mw;      // period in words; 1 where every position has the same Mask/Bitval word
    uint32_t src_Mw;  // words between the rows of the tables in device memory
    uint32_t runs;    // most runs of kept bits in one word
    uint32_t log2g;   // log2 of the words per chunk
    uint32_t hw;      // header words
    uint32_t valid;   // participation bits of the last header word
};

// Per-position tables as the rebuild reads them: rows kd, b, dx (one per four
// runs past the third), r (one per run), each `stride` words.
struct PageTab {
    const uint32_t* kd;
    const uint32_t* b;
    const uint32_t* dx;
    const uint32_t* r;
    uint32_t stride, runs;
};

__host__ __device__ constexpr uint32_t page_dx_rows(uint32_t runs) { return runs > 3 ? runs / 4u : 0u; }
__host__ __device__ constexpr uint32_t page_tab_stride(uint32_t Mw) { return Mw < 4 ? 4u : Mw; }
// LDS words of a pool's tables: four positions at least, so that a lane's
// four words are always one vector of a row.
__host__ __device__ constexpr uint32_t page_tab_words(uint32_t Mw, uint32_t runs) {
    return (2u + page_dx_rows(runs) + runs) * page_tab_stride(Mw);
}

// Vector i (four words) of the pool's tables as they stand in LDS.
__device__ __forceinline__ u32x4 page_table_vector(const Pool& p, uint32_t i) {
    const uint32_t S = page_tab_stride(p.Mw), dxr = page_dx_rows(p.runs);
    const uint32_t row = (4 * i) >> (31 - __builtin_clz(S)), pos = (4 * i) & (S - 1);  // periods are powers of two
    const uint32_t* src = row == 0 ? p.t.kd
                          : row == 1 ? p.t.b
                          : row < 2 + dxr ? p.t.dx + (row - 2) * p.src_Mw
                                          : p.t.r + (row - 2 - dxr) * p.src_Mw;
    if (p.Mw >= 4) return *reinterpret_cast<const u32x4*>(src + pos);
    const uint32_t x = src[0], y = src[p.Mw - 1];
    return u32x4{x, y, x, y};
}

// Whole workgroup: vectors [from, page_tab_words / 4) of the pool's tables
// into lds, four loads of a thread in flight.  The caller synchronises.
__device__ __forceinline__ void stage_page_tables(const Pool& p, uint32_t* lds, uint32_t from = 0) {
    const uint32_t n = page_tab_words(p.Mw, p.runs) / 4;
    for (uint32_t i = from + threadIdx.x; i < n; i += 4 * blockDim.x) {
        u32x4 v[4];
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u) v[u] = page_table_vector(p, min(i + u * blockDim.x, n - 1));
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u)
            if (i + u * blockDim.x < n) reinterpret_cast<u32x4*>(lds)[i + u * blockDim.x] = v[u];
    }
}

__device__ __forceinline__ PageTab page_tab(const Pool& p, const uint32_t* lds) {
    const uint32_t S = page_tab_stride(p.Mw), dxr = page_dx_rows(p.runs);
    return PageTab{lds, lds + S, lds + 2 * S, lds + (2 + dxr) * S, S, p.runs};
}
// The tables where they lie in device memory (period of at least four words).
__device__ __forceinline__ PageTab page_tab_global(const Pool& p) {
    return PageTab{p.t.kd, p.t.b, p.t.dx, p.t.r, p.Mw, p.runs};
}

// LDS words that one wave needs to rebuild a page of NV vectors per lane: the
// slot, and room for what a corrupt header can make the rebuild read (a
// header and every word verbatim, and the word after).
template <int NV>
__host__ __device__ constexpr uint32_t page_stage_words() {
    return 256u * NV + (256u * NV / 32u) + 8u;
}

// One wave.  st[r] of lane l: words 256 r + 4 l .. + 3 of a slot that holds a
// record; sink(w, x) receives words w .. w + 3 of the page, w = 256 s + 4 l
// for s = 0 .. NV - 1.  stage: page_stage_words<NV> words of this wave's LDS.
// Returns false for a record that is not valid (header padding set, or as
// long as the page).
//
// The rebuild is the codec's: a lane's four words take p ? 32 - k : 32 bits
// each, a wave scan gives their start bits, a funnel shift cuts the field out
// of two words of the record, and the field's runs go to their places.  The
// loop over s is not unrolled: unrolled, its table and record reads were
// hoisted together and the attention kernels spilled registers.
template <int NV, class Sink>
__device__ __forceinline__ bool rebuild_page(const u32x4* st, const Pool& p, const PageTab& tab, uint32_t* stage,
                                             Sink sink) {
    const uint32_t lane = lane_id();
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < NV; ++r) reinterpret_cast<u32x4*>(stage)[r * kWave + lane] = st[r];
    if (lane < 8) stage[256 * NV + lane] = 0;
    __builtin_amdgcn_wave_barrier();
    const uint32_t* pay = stage + p.hw;
    const uint32_t lg = p.log2g;
    const bool ok = p.valid >= 32 || (stage[p.hw - 1] >> p.valid) == 0;
    uint32_t carry = 0;
#pragma unroll 1
    for (int s = 0; s < NV; ++s) {
        const uint32_t w0 = 256u * s + 4u * lane;
        const uint32_t pos = w0 & (tab.stride - 1);
        const u32x4 kd = *reinterpret_cast<const u32x4*>(tab.kd + pos);
        u32x4 x = *reinterpret_cast<const u32x4*>(tab.b + pos);
        const uint32_t c0 = w0 >> lg;
        const uint32_t h = stage[c0 >> 5] >> (c0 & 31u);
        uint32_t part[4], size[4], tot = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            part[j] = (h >> ((uint32_t)j >> lg)) & 1u;
            size[j] = part[j] ? 32u - (kd[j] & 63u) : 32u;
            tot += size[j];
        }
        const uint32_t incl = wave_incl_scan(tot);
        uint32_t off = carry + incl - tot;
        carry += lane_value(incl, kWave - 1);
        uint32_t f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t q = off >> 5;
            f[j] = funnel(pay[q + 1], pay[q], off);
            off += size[j];
        }
#pragma unroll
        for (uint32_t r = 0; r < 3; ++r) {
            if (r < tab.runs) {
                const u32x4 rm = *reinterpret_cast<const u32x4*>(tab.r + r * tab.stride + pos);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] |= (f[j] << ((kd[j] >> (8 * (r + 1))) & 31u)) & rm[j];
            }
        }
        for (uint32_t r = 3; r < tab.runs; ++r) {
            const u32x4 rm = *reinterpret_cast<const u32x4*>(tab.r + r * tab.stride + pos);
            const u32x4 dv = *reinterpret_cast<const u32x4*>(tab.dx + ((r - 3) >> 2) * tab.stride + pos);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] |= (f[j] << ((dv[j] >> (8 * ((r - 3) & 3u))) & 31u)) & rm[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = part[j] ? x[j] : f[j];
        sink(w0, x);
    }
    __builtin_amdgcn_wave_barrier();
    return ok && p.hw + (carry + 31) / 32 < 256u * NV;
}

// One wave: the words of page `id` (kNoPage: zeros) as they lie in its slot.
template <int NV>
__device__ __forceinline__ void load_page(u32x4* st, const uint8_t* slots, uint32_t id) {
    const uint32_t lane = lane_id();
    if (id == kNoPage) {
#pragma unroll
        for (int r = 0; r < NV; ++r) st[r] = u32x4{0u, 0u, 0u, 0u};
        return;
    }
    const u32x4* s4 = reinterpret_cast<const u32x4*>(slots + (uint64_t)id * (1024ull * NV));
#pragma unroll
    for (int r = 0; r < NV; ++r) st[r] = s4[r * kWave + lane];
}

// A table's or list's page id in 32 bits; kNoPage when it is not a slot.
__device__ __forceinline__ uint32_t page_id(int64_t id, uint32_t n_slots) {
    return id >= 0 && (uint64_t)id < n_slots ? (uint32_t)id : kNoPage;
}

__device__ __forceinline__ uint32_t page_bit(const uint32_t* bitmask, uint32_t id) {
    return (bitmask[id >> 5] >> (id & 31u)) & 1u;
}

}  // namespace ibp
