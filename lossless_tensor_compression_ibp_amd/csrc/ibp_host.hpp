// ibp_host.hpp -- host-side pieces that every entry point of libibp shares:
// the metadata handle, the device guard, pointer checks and error mapping.
// Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <map>
#include <mutex>
#include <vector>

#include "../../include/ibp.h"
#include "ibp_internal.hpp"

namespace ibp {

// Look-back scratch of one (handle, stream) pair.  The ticket counter is
// zeroed on the stream before every launch; only the epoch, which keeps a
// launch's status words apart from those of earlier launches, is counted on
// the host.
struct Scratch {
    unsigned long long* status = nullptr;
    uint64_t status_cap = 0;
    uint64_t* totals = nullptr;
    uint64_t totals_cap = 0;
    uint32_t* ticket = nullptr;
    uint32_t epoch = 0;
};

}  // namespace ibp

struct ibp_meta_s {
    int device = 0;
    uint32_t cu_count = 0;
    uint64_t first_read_bytes = 0;  // 0: default policy
    uint64_t typical_item_bytes = 0; // median stored bytes over the metadata sample (0: unknown)
    ibp_params params{};
    uint32_t Mw = 0, Pc = 0, g = 0, log2g = 0, G = 0, Ne = 0;
    std::vector<uint32_t> mask_h, bitval_h;
    void* dmem = nullptr;
    uint32_t* d_mask = nullptr;
    uint32_t* d_bitval = nullptr;
    ibp::Summary* d_summary = nullptr;
    uint32_t* d_err = nullptr;
    ibp::Tables tabs{};
    ibp::Summary sum{};
    std::mutex mu;
    std::map<hipStream_t, ibp::Scratch> scratch;
};

namespace ibp {

struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) {
            ok = false;
            return;
        }
        if (prev != dev && hipSetDevice(dev) != hipSuccess) ok = false;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
    }
};

enum class Kind { Device, Host, Bad };

inline Kind pointer_kind(const void* ptr, int device) {
    if (!ptr) return Kind::Bad;
    hipPointerAttribute_t a;
    memset(&a, 0, sizeof(a));
    if (hipPointerGetAttributes(&a, ptr) != hipSuccess) {
        (void)hipGetLastError();
        return Kind::Bad;
    }
    switch (a.type) {
        case hipMemoryTypeDevice:
            return a.device == device ? Kind::Device : Kind::Bad;
        case hipMemoryTypeManaged:
            return Kind::Device;
        case hipMemoryTypeHost:
            return Kind::Host;
        default:
            return Kind::Bad;
    }
}

inline bool device_or_pinned(const void* p, int dev) { return pointer_kind(p, dev) != Kind::Bad; }
inline bool device_only(const void* p, int dev) { return pointer_kind(p, dev) == Kind::Device; }

inline ibp_status from_hip(hipError_t e) {
    if (e == hipSuccess) return IBP_OK;
    (void)hipGetLastError();
    return e == hipErrorOutOfMemory ? IBP_ERR_NOMEM : IBP_ERR_DEVICE;
}

#define IBP_TRY(expr)                        \
    do {                                     \
        ibp_status st_ = from_hip(expr);     \
        if (st_ != IBP_OK) return st_;       \
    } while (0)

inline bool aligned16(uint64_t L, std::initializer_list<const void*> ptrs) {
    if (L % 16 != 0) return false;
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    return true;
}

inline bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

constexpr uint64_t kLineWords = 64;     // 256-byte first-read granule
constexpr uint64_t kMemLineWords = 32;  // 128-byte line that memory reads move

inline uint32_t bit_length(uint32_t v) {
    uint32_t n = 0;
    while (v) {
        ++n;
        v >>= 1;
    }
    return n;
}

inline uint64_t min_record_bits(const ibp_meta_s* h) {
    const uint64_t L = h->params.tensor_bytes;
    const uint64_t n_chunks = 8 * L / h->params.chunk_bits;
    const uint64_t H = 32 * ((n_chunks + 31) / 32);
    const uint64_t periods = 8 * L / h->params.period_bits;
    return H + 8 * L - periods * h->sum.invariant_bits;
}

inline Geo make_geo(const ibp_meta_s* h, bool aligned16, uint32_t long_tile_words) {
    Geo g{};
    const uint64_t L = h->params.tensor_bytes;
    g.L = L;
    g.n_words = L / 4;
    g.n_chunks = 8 * L / h->params.chunk_bits;
    g.hdr_words = (g.n_chunks + 31) / 32;
    g.Mw = h->Mw;
    g.Pc = h->Pc;
    g.log2g = h->log2g;
    g.G = h->G;
    g.np = bit_length(h->sum.max_chunk_k);
    if (g.np > (uint32_t)kPlanes) g.np = kPlanes;
    g.k1 = g.Pc == 1 ? h->sum.max_chunk_k : 0;
    g.aligned16 = aligned16 ? 1u : 0u;
    if (g.n_words <= kMaxTileWords) {
        g.tile_words = (uint32_t)g.n_words;
        g.tiles_per_tensor = 1;
    } else {
        g.tile_words = long_tile_words;
        g.tiles_per_tensor = (g.n_words + long_tile_words - 1) / long_tile_words;
    }
    // First read of a single-tile record: every record is at least min_words
    // long, so the read is cut at the last 256-byte boundary inside that
    // prefix, and is never shorter than 256 bytes (the second read then starts
    // on a 256-byte boundary; zero-copy reads of pinned host memory measured
    // fastest with this split).  Memory moves whole 128-byte lines, so when
    // the shortest record already covers all but 1/16 of the slot's lines,
    // the whole slot is read at once instead of paying a second round trip.
    const uint64_t min_words = (min_record_bits(h) + 31) / 32;
    const uint64_t slot_lines = (g.n_words + kMemLineWords - 1) / kMemLineWords;
    const uint64_t min_lines = (min_words + kMemLineWords - 1) / kMemLineWords;
    uint64_t spec;
    if (h->first_read_bytes) {
        spec = (h->first_read_bytes + 3) / 4;
        if (spec < g.hdr_words) spec = g.hdr_words;
    } else if (min_lines >= slot_lines || (slot_lines - min_lines) * 16 <= slot_lines) {
        spec = g.n_words;
    } else {
        spec = (min_words / kLineWords) * kLineWords;
        if (spec < kLineWords) spec = kLineWords;
        // records of the sample mostly shorter than that: one 128-byte line
        // (rounded up to whole lines) covers the usual record in one read
        if (h->typical_item_bytes) {
            const uint64_t usual = (h->typical_item_bytes + 4 * kMemLineWords - 1) / (4 * kMemLineWords) * kMemLineWords;
            if (usual < spec) spec = usual;
        }
        if (spec < g.hdr_words) spec = g.hdr_words;
    }
    if (aligned16) spec = (spec + 3) & ~3ull;
    if (spec > g.n_words) spec = g.n_words;
    g.spec_words = (uint32_t)spec;
    return g;
}

}  // namespace ibp
