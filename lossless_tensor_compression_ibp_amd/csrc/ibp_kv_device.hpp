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

// A pool of pages as a kernel sees it.  `tab` is row kd of the handle's
// tables: in device memory row b (Bitval) lies one row before it, the dx rows
// from one row and the r rows from five rows behind it, all src_Mw words
// apart.
struct Pool {
    const uint8_t* slots;
    const uint32_t* bitmask;
    uint32_t* err;
    const uint32_t* tab;
    uint32_t n_slots;
    uint32_t Mw;      // period in words; 1 where every position has the same Mask/Bitval word
    uint32_t src_Mw;  // words between the rows of the tables in device memory
    uint32_t runs;    // most runs of kept bits in one word
    uint32_t log2g;   // log2 of the words per chunk
    uint32_t hw;      // header words
    uint32_t valid;   // participation bits of the last header word
};

// Rows of a table as the rebuild reads them, all `stride` words: kd, b, dx
// (one per four runs past the third), r (one per run) in LDS; in device
// memory (in_lds 0) as above.  Pointers to LDS keep their address space: a
// choice between two generic pointers would be read with flat loads.
typedef const __attribute__((address_space(3))) uint32_t* LdsWords;
typedef const __attribute__((address_space(3))) u32x4* LdsVectors;
struct PageTab {
    LdsWords lds;
    const uint32_t* mem;
    uint32_t in_lds, stride, runs;
};

__host__ __device__ constexpr uint32_t page_dx_rows(uint32_t runs) { return runs > 3 ? runs / 4u : 0u; }
__host__ __device__ constexpr uint32_t page_tab_stride(uint32_t Mw) { return Mw < 4 ? 4u : Mw; }
// LDS words of a pool's tables: four positions at least, so that a lane's
// four words are always one vector of a row.
__host__ __device__ constexpr uint32_t page_tab_words(uint32_t Mw, uint32_t runs) {
    return (2u + page_dx_rows(runs) + runs) * page_tab_stride(Mw);
}

__device__ __forceinline__ int32_t page_tab_source_row(uint32_t row, uint32_t dxr) {
    return row == 0 ? 0 : row == 1 ? -1 : row < 2 + dxr ? (int32_t)row - 1 : (int32_t)(row - 2 - dxr) + 5;
}

// Vector i (four words) of the pool's tables as they stand in LDS.
__device__ __forceinline__ u32x4 page_table_vector(const Pool& p, uint32_t i) {
    const uint32_t S = page_tab_stride(p.Mw), dxr = page_dx_rows(p.runs);
    const uint32_t row = (4 * i) >> (31 - __builtin_clz(S)), pos = (4 * i) & (S - 1);  // periods are powers of two
    const uint32_t* src = p.tab + (int64_t)page_tab_source_row(row, dxr) * p.src_Mw;
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

// The tables at `lds`, or where they lie in device memory (in_lds 0; a period
// of at least four words).
__device__ __forceinline__ PageTab page_tab(const Pool& p, const uint32_t* lds, uint32_t in_lds) {
    return PageTab{(LdsWords)lds, p.tab, in_lds, in_lds ? page_tab_stride(p.Mw) : p.src_Mw, p.runs};
}

// Four positions of a row: at `lds_row` in LDS, `mem_row` in device memory.
__device__ __forceinline__ u32x4 tab_vector(const PageTab& t, uint32_t lds_row, int32_t mem_row, uint32_t pos) {
    if (t.in_lds) return *(LdsVectors)(t.lds + lds_row * t.stride + pos);
    return *reinterpret_cast<const u32x4*>(t.mem + (int64_t)mem_row * t.stride + pos);
}

// LDS words that one wave needs to rebuild a page of NV vectors per lane: the
// slot, and room for what a corrupt header can make the rebuild read (a
// header and every word verbatim, and the word after).
template <int NV>
__host__ __device__ constexpr uint32_t page_stage_words() {
    return 256u * NV + (256u * NV / 32u) + 8u;
}

// One wave: a slot from registers (load_page) to its LDS.
template <int NV>
__device__ __forceinline__ void stage_page(const u32x4* st, uint32_t* stage) {
    const uint32_t lane = lane_id();
#pragma unroll
    for (int r = 0; r < NV; ++r) reinterpret_cast<u32x4*>(stage)[r * kWave + lane] = st[r];
    if (lane < 8) stage[256 * NV + lane] = 0;
}

// One wave: the record in stage (page_stage_words<NV> words of this wave's
// LDS) rebuilt; sink(w, x) receives words w .. w + 3 of the page, w = 256 s +
// 4 l for s = 0 .. NV - 1.  Returns false for a record that is not valid
// (header padding set, or as long as the page).
//
// The rebuild is the codec's: a lane's four words take p ? 32 - k : 32 bits
// each, a wave scan gives their start bits, a funnel shift cuts the field out
// of two words of the record, and the field's runs go to their places.  It is
// a chain of latencies (header, scan, record, tables), so U steps of 256 words
// go through it together where the table entries allow: with a period of at
// most 256 words a lane's positions are the same in every step and its
// entries are read once.  (Attention over eight streams, 61 % of the value
// pages records, 16-token pages of 128 dims: 4,500 cycles a page one step at
// a time.)  With longer periods a step's entries fill the registers.
template <int U, class Sink>
__device__ __forceinline__ void rebuild_steps(const Pool& p, const PageTab& tab, const uint32_t* stage, uint32_t s0,
                                              bool read, u32x4& kd, u32x4& bv, u32x4 (&rm)[3], uint32_t& carry,
                                              Sink sink) {
    const uint32_t lane = lane_id(), lg = p.log2g, runs = tab.runs, dxr = page_dx_rows(runs);
    const uint32_t* pay = stage + p.hw;
    const uint32_t pos = (256u * s0 + 4u * lane) & (tab.stride - 1);
    uint32_t h[U], off[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t c0 = (256u * (s0 + u) + 4u * lane) >> lg;
        h[u] = stage[c0 >> 5] >> (c0 & 31u);
    }
    if (read) {
        kd = tab_vector(tab, 0, 0, pos);
        bv = tab_vector(tab, 1, -1, pos);
#pragma unroll
        for (uint32_t r = 0; r < 3; ++r)
            if (r < runs) rm[r] = tab_vector(tab, 2 + dxr + r, 5 + r, pos);
    }
    auto part = [&](int u, int j) __attribute__((always_inline)) { return (h[u] >> ((uint32_t)j >> lg)) & 1u; };
    uint32_t tot[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        tot[u] = 128u;
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[u] -= part(u, j) ? kd[j] & 63u : 0u;
        off[u] = tot[u];
    }
    // U wave scans side by side (wave_incl_scan)
#define IBP_SCAN_STEP(ctrl, rows)                                                                        \
    _Pragma("unroll") for (int u = 0; u < U; ++u)                                                        \
        off[u] += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)off[u], ctrl, rows, 0xf, false);
    IBP_SCAN_STEP(0x111, 0xf)
    IBP_SCAN_STEP(0x112, 0xf)
    IBP_SCAN_STEP(0x114, 0xf)
    IBP_SCAN_STEP(0x118, 0xf)
    IBP_SCAN_STEP(0x142, 0xa)
    IBP_SCAN_STEP(0x143, 0xc)
#undef IBP_SCAN_STEP
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t end = lane_value(off[u], kWave - 1);
        off[u] += carry - tot[u];
        carry += end;
    }
    u32x4 f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t q = off[u] >> 5;
            f[u][j] = funnel(pay[q + 1], pay[q], off[u]);
            off[u] += 32u - (part(u, j) ? kd[j] & 63u : 0u);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        u32x4 x = bv;
#pragma unroll
        for (uint32_t r = 0; r < 3; ++r)  // (rows that are not there stay zero)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] |= (f[u][j] << ((kd[j] >> (8 * (r + 1))) & 31u)) & rm[r][j];
        for (uint32_t r = 3; U == 1 && r < runs; ++r) {
            const u32x4 m = tab_vector(tab, 2 + dxr + r, 5 + r, pos);
            const u32x4 dv = tab_vector(tab, 2 + ((r - 3) >> 2), 1 + ((r - 3) >> 2), pos);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] |= (f[u][j] << ((dv[j] >> (8 * ((r - 3) & 3u))) & 31u)) & m[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = part(u, j) ? x[j] : f[u][j];
        sink(256u * (s0 + u) + 4u * lane, x);
    }
}

template <int NV, int U, class Sink>
__device__ __forceinline__ bool rebuild_page(const Pool& p, const PageTab& tab, const uint32_t* stage, Sink sink) {
    static_assert(NV % U == 0, "whole groups of steps");
    __builtin_amdgcn_wave_barrier();
    const bool ok = p.valid >= 32 || (stage[p.hw - 1] >> p.valid) == 0;
    uint32_t carry = 0;
    u32x4 kd = {0u, 0u, 0u, 0u}, bv = kd, rm[3] = {kd, kd, kd};
    if (U > 1 && tab.stride <= 256u && tab.runs <= 3) {
#pragma unroll 1
        for (int s = 0; s < NV; s += U) rebuild_steps<U>(p, tab, stage, s, s == 0, kd, bv, rm, carry, sink);
    } else {
#pragma unroll 1
        for (int s = 0; s < NV; ++s)
            rebuild_steps<1>(p, tab, stage, s, s == 0 || tab.stride > 256u, kd, bv, rm, carry, sink);
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
