// ibp_pages.hip -- pages of a cache moved and counted without decoding them:
// copying, allocating, forking, freeing and compacting slots.
//
// A page is one slot of the codec's fixed-slot layout; its item is the
// record when its bitmask bit is 1 (4*ceil(R/32) bytes, R from the header),
// else all L bytes.  Copying moves the item and its bit, so a compressed page
// costs its stored bytes only, and pages go to and from pinned host memory at
// their compressed size.  Reference counts (one int32 per slot, 0 = free) and
// block tables (int64 slot ids, -1 = none) live in device memory, and every
// call is a fixed sequence of launches that the host plans without reading
// them, so each may be captured in a graph.
//
// Nothing here depends on the order in which workgroups run: free slots are
// ranked by a prefix sum (the lowest first), counts change by integer
// atomics, and bitmask bits by atomic AND / OR of single bits.
//
// Short calls are bound by launches: 263 pages of 4 KiB are copied in 4.5 us
// on the GPU and 7.3 us of host time per call.  Compacting 65,536 slots of
// 4 KiB, 55 % of them live, moves 134 MB in 35 us, 3.8 TB/s (a large copy
// 4.8); counting, planning and remapping take 12 us more.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/ibp.h"
#include "ibp_device.hpp"
#include "ibp_host.hpp"
#include "ibp_internal.hpp"
#include "ibp_kv_device.hpp"

namespace ibp {

constexpr uint32_t kPageWaves = 4;        // waves (items) per workgroup of the copies
constexpr uint32_t kCountBlock = 256;     // threads of the counting kernels
constexpr uint32_t kCountPer = 4;         // slots per thread
constexpr uint32_t kCountSlots = kCountBlock * kCountPer;
// The free slots that a fork may take are counted and listed in one launch in
// pools of up to kListSlots slots: its workgroups (of kListBlock threads) each
// read all counts, at most 16 loads of 16 bytes per thread.  With 32,768 slots
// that is 6.7 us on the GPU against 5.4 in two launches, but forks are bound by
// the host, for which a launch is 4 to 5 us (fork and free 28.8 us, 34.3 with
// the second launch).  The plan of a compaction does so in pools of up to
// kPlanSlots (pools of a few thousand slots, bound by the host: 27 us a call,
// 30 with the second launch); with 65,536 slots, where the GPU is the bound, it
// took 10.4 us this way and 6.8 in two launches.
constexpr uint32_t kListBlock = 1024;
constexpr uint64_t kListSlots = 65536;
constexpr uint64_t kPlanSlots = 32768;

// Removed bits of the item's header, summed over the wave.  st[0] of lane l
// holds words 4 l .. 4 l + 3 of the slot, which include every header word
// (at most 64: 2,048 words of one word per chunk).
__device__ __forceinline__ uint32_t item_removed_bits(const Tables& t, const Geo& g, const u32x4& head, bool* bad) {
    const uint32_t lane = lane_id();
    uint32_t rem = 0;
    bool b = false;
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) {
        const uint32_t j = 4 * lane + c;
        if (j < g.hdr_words) {
            uint32_t h = head[c];
            if (j == g.hdr_words - 1) {
                const uint32_t valid = (uint32_t)(g.n_chunks - 32ull * j);
                if (valid < 32) {
                    b = (h >> valid) != 0;
                    h &= (1u << valid) - 1u;
                }
            }
            rem += removed_bits_pl(t.planes, g, j, h);
        }
    }
    *bad = ballot(b) != 0;
    return wave_sum(rem);
}

__device__ __forceinline__ void set_bit(uint32_t* bitmask, uint64_t i, uint32_t bit) {
    const uint32_t m = 1u << (i & 31);
    if (bit)
        atomicOr(bitmask + (i >> 5), m);
    else
        atomicAnd(bitmask + (i >> 5), ~m);
}

// One wave: the item of slot `from` to slot `to`, and its bit.  The first
// spec_words of the slot are read at once; the rest of a record follows when
// its header has told its length.  Bytes of the destination past the item
// stay as they were.  A record that is not valid is copied as a whole slot
// and latches kErrCorrupt.
template <int NV>
__device__ __forceinline__ void copy_item(const Tables& t, const Geo& g, const uint8_t* src_slots,
                                          const uint32_t* src_bitmask, uint64_t from, uint8_t* dst_slots,
                                          uint32_t* dst_bitmask, uint64_t to, uint32_t* err) {
    const uint32_t lane = lane_id();
    const u32x4* s4 = reinterpret_cast<const u32x4*>(src_slots + from * g.L);
    uint32_t* dw = reinterpret_cast<uint32_t*>(dst_slots + to * g.L);
    u32x4* d4 = reinterpret_cast<u32x4*>(dw);
    const uint32_t n4 = (uint32_t)(g.n_words >> 2);
    const uint32_t first = min(g.spec_words >> 2, n4);
    u32x4 st[NV];
#pragma unroll
    for (int r = 0; r < NV; ++r) {
        const uint32_t i = lane + (uint32_t)r * kWave;
        st[r] = u32x4{0u, 0u, 0u, 0u};
        if (i < first) st[r] = __builtin_nontemporal_load(s4 + i);
    }
    const uint32_t bit = uniform((src_bitmask[from >> 5] >> (from & 31)) & 1u);
    uint32_t words = (uint32_t)g.n_words;
    if (bit) {
        bool bad;
        const uint32_t rem = item_removed_bits(t, g, st[0], &bad);
        const uint64_t R = 32ull * g.hdr_words + 32ull * g.n_words - rem;
        const uint64_t w = (R + 31) / 32;
        if (bad || w >= g.n_words)
            latch_error(err, kErrCorrupt);
        else
            words = (uint32_t)w;
    }
    if (4 * first < words) {
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const uint32_t i = lane + (uint32_t)r * kWave;
            if (i >= first && 4 * i < words) st[r] = __builtin_nontemporal_load(s4 + i);
        }
    }
#pragma unroll
    for (int r = 0; r < NV; ++r) {
        const uint32_t i = lane + (uint32_t)r * kWave;
        if (4 * i + 3 < words) {
            __builtin_nontemporal_store(st[r], d4 + i);
        } else {
#pragma unroll
            for (uint32_t c = 0; c < 3; ++c)
                if (4 * i + c < words) dw[4 * i + c] = st[r][c];
        }
    }
    if (lane == 0) set_bit(dst_bitmask, to, bit);
}

template <int NV>
__global__ __launch_bounds__(kWave * kPageWaves) void k_pages_copy(Tables t, Geo g, const uint8_t* src, uint64_t n_src,
                                                                   const uint32_t* src_bm, const int64_t* src_ids,
                                                                   uint8_t* dst, uint64_t n_dst, uint32_t* dst_bm,
                                                                   const int64_t* dst_ids, uint64_t n,
                                                                   uint32_t* err) {
    const uint64_t stride = (uint64_t)gridDim.x * kPageWaves;
    for (uint64_t i = (uint64_t)blockIdx.x * kPageWaves + uniform(threadIdx.x / kWave); i < n; i += stride) {
        const int64_t a = (int64_t)uniform64((uint64_t)src_ids[i]), b = (int64_t)uniform64((uint64_t)dst_ids[i]);
        if (a == -1 || b == -1) continue;
        if (a < 0 || (uint64_t)a >= n_src || b < 0 || (uint64_t)b >= n_dst) {
            latch_error(err, kErrRange);
            continue;
        }
        copy_item<NV>(t, g, src, src_bm, (uint64_t)a, dst, dst_bm, (uint64_t)b, err);
    }
}

// ---------------------------------------------------------------------------
// Free slots.  counts[b]: free slots (refs <= 0) among the kCountSlots slots
// of block b.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* sh) {
    const uint32_t w = threadIdx.x / kWave;
    v = wave_sum(v);
    __syncthreads();
    if (lane_id() == 0) sh[w] = v;
    __syncthreads();
    uint32_t s = 0;
    for (uint32_t i = 0; i < blockDim.x / kWave; ++i) s += sh[i];
    return s;
}

// Bit c of the result: slot base + c of this thread is free.
__device__ __forceinline__ uint32_t free_flags(const int32_t* refs, uint64_t n_slots, uint64_t base) {
    uint32_t f = 0;
#pragma unroll
    for (uint32_t c = 0; c < kCountPer; ++c)
        if (base + c < n_slots && refs[base + c] <= 0) f |= 1u << c;
    return f;
}

__global__ __launch_bounds__(kCountBlock) void k_count_free(const int32_t* refs, uint64_t n_slots, uint32_t* counts) {
    __shared__ uint32_t sh[kCountBlock / kWave];
    const uint64_t base = (uint64_t)blockIdx.x * kCountSlots + threadIdx.x * kCountPer;
    const uint32_t s = block_sum((uint32_t)__builtin_popcount(free_flags(refs, n_slots, base)), sh);
    if (threadIdx.x == 0) counts[blockIdx.x] = s;
}

// Free slots before this thread's first one; *all: in the whole pool.  SCAN:
// from `refs` themselves, which nobody may be writing, instead of `counts`.
template <bool SCAN>
__device__ __forceinline__ uint64_t free_before(const int32_t* refs, uint64_t n_slots, const uint32_t* counts,
                                                uint32_t mine, uint64_t* all) {
    constexpr uint32_t kBlock = SCAN ? kListBlock : kCountBlock;
    __shared__ uint64_t before_sh[kBlock / kWave], all_sh[kBlock / kWave];
    __shared__ uint32_t sh[kBlock / kWave];
    uint64_t before = 0, total = 0;
    if (SCAN) {
        typedef int32_t Four __attribute__((ext_vector_type(4), aligned(4)));
        const uint32_t n = (uint32_t)n_slots, full = n & ~3u, first = blockIdx.x * (kBlock * kCountPer);
#pragma unroll 4
        for (uint32_t i = 4 * threadIdx.x; i < full; i += 4 * kBlock) {
            const Four v = *reinterpret_cast<const Four*>(refs + i);
            const uint32_t c = (uint32_t)(v.x <= 0) + (v.y <= 0) + (v.z <= 0) + (v.w <= 0);
            total += c;
            if (i < first) before += c;
        }
        if (threadIdx.x < n - full) total += refs[full + threadIdx.x] <= 0;  // behind every block's first
    } else {
        for (uint32_t b = threadIdx.x; b < gridDim.x; b += kBlock) {
            const uint32_t c = counts[b];
            total += c;
            if (b < blockIdx.x) before += c;
        }
    }
    before = wave_sum64(before);
    total = wave_sum64(total);
    const uint32_t w = threadIdx.x / kWave;
    const uint32_t incl = wave_incl_scan(mine);
    if (lane_id() == kWave - 1) sh[w] = incl;
    if (lane_id() == 0) {
        before_sh[w] = before;
        all_sh[w] = total;
    }
    __syncthreads();
    uint64_t r = incl - mine;
    *all = 0;
    for (uint32_t i = 0; i < kBlock / kWave; ++i) {
        r += before_sh[i];
        *all += all_sh[i];
        if (i < w) r += sh[i];
    }
    return r;
}

// ids[r] <- the r-th free slot, r < n.  TAKE: the slots' counts become 1 (and
// their bits in bitmask, if given, 0), ids without a slot -1, and too few free
// slots latch kErrFull.
template <bool TAKE, bool SCAN>
__global__ __launch_bounds__(SCAN ? kListBlock : kCountBlock) void k_list_free(int32_t* refs, uint64_t n_slots,
                                                                              const uint32_t* counts, int64_t* ids,
                                                                              uint64_t n, uint32_t* bitmask,
                                                                              uint32_t* err) {
    static_assert(!(TAKE && SCAN), "other workgroups would read counts while this one writes its own");
    const uint64_t base = ((uint64_t)blockIdx.x * blockDim.x + threadIdx.x) * kCountPer;
    uint32_t f = free_flags(refs, n_slots, base);
    uint64_t all;
    uint64_t r = free_before<SCAN>(refs, n_slots, counts, (uint32_t)__builtin_popcount(f), &all);
    while (f && r < n) {
        const uint64_t slot = base + (uint32_t)__builtin_ctz(f);
        f &= f - 1;
        ids[r++] = (int64_t)slot;
        if (TAKE) {
            refs[slot] = 1;
            if (bitmask) set_bit(bitmask, slot, 0);
        }
    }
    if (blockIdx.x == gridDim.x - 1 && all < n) {
        for (uint64_t i = all + threadIdx.x; i < n; i += blockDim.x) ids[i] = -1;
        if (TAKE) latch_error(err, kErrFull);
    }
}

// ---------------------------------------------------------------------------
// Forking.  One workgroup per (fork, head): the parent's full pages are
// shared (counts + 1), a page that is still being filled is copied into a
// free slot of its own -- the r-th of `fresh`, r counting the forks and heads
// before this one that need a slot.
// ---------------------------------------------------------------------------
struct ForkArgs {
    const uint8_t* slots;
    uint8_t* dst;
    uint32_t* bitmask;
    int32_t* refs;
    int64_t* table;
    const int32_t* lens;
    const int64_t* parents;
    const int64_t* children;
    const int64_t* fresh;
    uint64_t n_slots, n_seqs, blocks, n;
    uint32_t heads, page_tokens;
};

// Context tokens of the parent of fork i; -1 when the fork is not valid.
__device__ __forceinline__ int64_t fork_len(const ForkArgs& a, uint64_t i) {
    const int64_t p = a.parents[i], c = a.children[i];
    if (p < 0 || (uint64_t)p >= a.n_seqs || c < 0 || (uint64_t)c >= a.n_seqs || p == c) return -1;
    const int64_t len = a.lens[p];
    return len < 0 || (uint64_t)len > a.blocks * a.page_tokens ? -1 : len;
}

template <int NV>
__global__ __launch_bounds__(256) void k_pages_fork(Tables t, Geo g, ForkArgs a, uint32_t* err) {
    __shared__ uint32_t sh[4];
    const uint64_t i = blockIdx.x / a.heads;
    const uint32_t h = blockIdx.x % a.heads;
    const int64_t len = fork_len(a, i);
    if (len < 0) {
        latch_error(err, kErrRange);
        return;
    }
    uint32_t before = 0;
    for (uint64_t j = threadIdx.x; j < i; j += blockDim.x) {
        const int64_t l = fork_len(a, j);
        before += l > 0 && l % a.page_tokens != 0;
    }
    before = block_sum(before, sh);
    const uint64_t full = (uint64_t)len / a.page_tokens;
    const bool tail = (uint64_t)len % a.page_tokens != 0;
    const int64_t* from = a.table + ((uint64_t)a.parents[i] * a.heads + h) * a.blocks;
    int64_t* to = a.table + ((uint64_t)a.children[i] * a.heads + h) * a.blocks;
    bool bad = false;
    for (uint64_t b = threadIdx.x; b < a.blocks; b += blockDim.x) {
        int64_t id = -1;
        if (b < full) {
            id = from[b];
            if (id < 0 || (uint64_t)id >= a.n_slots) {
                bad = true;
                id = -1;
            } else {
                atomicAdd(a.refs + id, 1);
            }
        }
        if (!(tail && b == full)) to[b] = id;
    }
    if (ballot(bad)) latch_error(err, kErrRange);
    if (tail && threadIdx.x < kWave) {
        const int64_t old = (int64_t)uniform64((uint64_t)from[full]);
        const int64_t neu = (int64_t)uniform64((uint64_t)a.fresh[(uint64_t)before * a.heads + h]);
        const bool bad_old = old < 0 || (uint64_t)old >= a.n_slots;
        if (bad_old || neu < 0) {
            latch_error(err, bad_old ? kErrRange : kErrFull);
            if (lane_id() == 0) to[full] = -1;
            return;
        }
        copy_item<NV>(t, g, a.slots, a.bitmask, (uint64_t)old, a.dst, a.bitmask, (uint64_t)neu, err);
        if (lane_id() == 0) {
            to[full] = neu;
            a.refs[neu] = 1;
        }
    }
}

// A table entry of the sequences given after another: the entry becomes -1 and
// its page's count falls by one.  The exchange makes a sequence that is given
// twice count once.
__global__ __launch_bounds__(256) void k_pages_free(int32_t* refs, uint64_t n_slots, int64_t* table, uint64_t n_seqs,
                                                    uint64_t row, const int64_t* seqs, uint64_t n, uint32_t* err) {
    const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
    bool range = false, below = false;
    for (uint64_t e = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n * row; e += stride) {
        const int64_t s = seqs[e / row];
        if (s < 0 || (uint64_t)s >= n_seqs) {
            range = true;
            continue;
        }
        unsigned long long* p = reinterpret_cast<unsigned long long*>(table + (uint64_t)s * row + e % row);
        const int64_t id = (int64_t)atomicExch(p, ~0ull);
        if (id >= 0 && (uint64_t)id < n_slots) {
            if (atomicSub(refs + id, 1) <= 0) {
                atomicAdd(refs + id, 1);
                below = true;
            }
        } else if (id != -1) {
            range = true;
        }
    }
    if (range) atomicCAS(err, 0u, (uint32_t)kErrRange);
    if (below) atomicCAS(err, 0u, (uint32_t)kErrCorrupt);
}

// ---------------------------------------------------------------------------
// Compaction.  With n_live live pages, hole j (the j-th free slot, counted
// from the front, if it lies before n_live) takes mover j (the j-th live slot
// counted from the back): as many movers as holes, and a mover lies behind
// every hole, so no move reads a slot that another one writes.
// ---------------------------------------------------------------------------
template <bool SCAN>
__global__ __launch_bounds__(SCAN ? kListBlock : kCountBlock) void k_compact_plan(
    const int32_t* refs, uint64_t n_slots, const uint32_t* counts, int64_t* map, int64_t* n_live, uint64_t* n_moves,
    uint32_t* holes, uint32_t* movers) {
    const uint64_t base = ((uint64_t)blockIdx.x * blockDim.x + threadIdx.x) * kCountPer;
    const uint32_t f = free_flags(refs, n_slots, base);
    uint64_t all;
    uint64_t r = free_before<SCAN>(refs, n_slots, counts, (uint32_t)__builtin_popcount(f), &all);
    const uint64_t live = n_slots - all;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *n_live = (int64_t)live;
        if (live == n_slots) *n_moves = 0;
    }
#pragma unroll
    for (uint32_t c = 0; c < kCountPer; ++c) {
        const uint64_t i = base + c;
        if (i >= n_slots) break;
        if (i == live) *n_moves = r;
        if ((f >> c) & 1u) {
            if (i < live) holes[r] = (uint32_t)i;
            map[i] = -1;
            ++r;
        } else if (i < live) {
            map[i] = (int64_t)i;
        } else {
            movers[live - 1 - (i - r)] = (uint32_t)i;
        }
    }
}

template <int NV>
__global__ __launch_bounds__(kWave * kPageWaves) void k_compact_move(Tables t, Geo g, uint8_t* slots,
                                                                     uint32_t* bitmask, int32_t* refs, int64_t* map,
                                                                     const uint64_t* n_moves, const uint32_t* holes,
                                                                     const uint32_t* movers, uint32_t* err) {
    const uint64_t n = uniform64(*n_moves);
    const uint64_t stride = (uint64_t)gridDim.x * kPageWaves;
    for (uint64_t j = (uint64_t)blockIdx.x * kPageWaves + uniform(threadIdx.x / kWave); j < n; j += stride) {
        const uint32_t to = uniform(holes[j]), from = uniform(movers[j]);
        if (lane_id() == 0) {
            map[from] = (int64_t)to;
            refs[to] = refs[from];
            refs[from] = 0;
        }
        copy_item<NV>(t, g, slots, bitmask, from, slots, bitmask, to, err);
    }
}

__global__ __launch_bounds__(256) void k_remap(const int64_t* map, uint64_t n_slots, int64_t* table, uint64_t n,
                                               uint32_t* err) {
    const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t e = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += stride) {
        const int64_t id = table[e];
        if (id == -1) continue;
        if (id >= 0 && (uint64_t)id < n_slots)
            table[e] = map[id];
        else
            atomicCAS(err, 0u, (uint32_t)kErrRange);
    }
}

// Workgroups of the kernels that stride over their items: one per `per` of
// them, and fewer only where one launch does not hold as many.
constexpr uint64_t kMaxStriding = 1u << 22;
static dim3 striding_grid(uint64_t items, uint64_t per) {
    return dim3((uint32_t)std::min<uint64_t>((items + per - 1) / per, kMaxStriding));
}

// f.template operator()<NV>() for the vectors per lane that a page of L bytes takes.
template <class F>
static hipError_t by_vectors(uint64_t L, F f) {
    if (L <= 1024) return f(std::integral_constant<int, 1>{});
    if (L <= 2048) return f(std::integral_constant<int, 2>{});
    if (L <= 4096) return f(std::integral_constant<int, 4>{});
    return f(std::integral_constant<int, 8>{});
}

static uint64_t count_blocks(uint64_t n_slots) { return (n_slots + kCountSlots - 1) / kCountSlots; }

// Workspace of the calls below, in 8-byte words: block counts, then either
// the list of free slots (n words) or the move count and the two move lists.
static uint64_t count_words(uint64_t n_slots) { return (count_blocks(n_slots) + 1) / 2 + 1; }

}  // namespace ibp

using namespace ibp;

// What every call that copies items needs of the handle's format.
static ibp_status check_page_format(ibp_meta_t h, std::initializer_list<const void*> slots) {
    const uint64_t L = h->params.tensor_bytes;
    if (L > kMaxPageBytes || !aligned16(L, slots)) return IBP_ERR_UNSUPPORTED;
    return IBP_OK;
}

// Threads and workgroups of a kernel that lists without counts.
static dim3 scan_grid(uint64_t n_slots) {
    return dim3((uint32_t)((n_slots + kListBlock * kCountPer - 1) / (kListBlock * kCountPer)));
}

static hipError_t launch_count_free(const int32_t* refs, uint64_t n_slots, uint32_t* counts, hipStream_t s) {
    hipLaunchKernelGGL(k_count_free, dim3((uint32_t)count_blocks(n_slots)), dim3(kCountBlock), 0, s, refs, n_slots,
                       counts);
    return hipGetLastError();
}

extern "C" {

ibp_status ibp_pages_copy(ibp_meta_t h, const void* src_slots, uint64_t n_src, const uint32_t* src_bitmask,
                          const int64_t* src_ids, void* dst_slots, uint64_t n_dst, uint32_t* dst_bitmask,
                          const int64_t* dst_ids, uint64_t n, hipStream_t stream) {
    if (!h) return IBP_ERR_INVALID_ARG;
    if (n == 0) return IBP_OK;
    DeviceGuard guard(h->device);
    if (!guard.ok) return IBP_ERR_DEVICE;
    const uint64_t L = h->params.tensor_bytes;
    if (n_src > kMaxPoolSlots || n_dst > kMaxPoolSlots || n > kMaxPoolSlots) return IBP_ERR_INVALID_ARG;
    const Kind kind = pointer_kind(src_slots, h->device);
    if (kind == Kind::Bad || !device_or_pinned(dst_slots, h->device)) return IBP_ERR_INVALID_ARG;
    if (!device_only(src_bitmask, h->device) || !device_only(dst_bitmask, h->device) ||
        !device_only(src_ids, h->device) || !device_only(dst_ids, h->device))
        return IBP_ERR_INVALID_ARG;
    // one pool copied within itself, or two that do not touch
    if (src_slots != dst_slots && overlaps(src_slots, n_src * L, dst_slots, n_dst * L)) return IBP_ERR_INVALID_ARG;
    ibp_status st = check_page_format(h, {src_slots, dst_slots});
    if (st != IBP_OK) return st;
    const Geo geo = make_geo(h, true, kLongTileWordsDecode);
    return from_hip(by_vectors(L, [&](auto nv) {
        hipLaunchKernelGGL((k_pages_copy<decltype(nv)::value>), striding_grid(n, kPageWaves),
                           dim3(kWave * kPageWaves), 0, stream, h->tabs, geo, static_cast<const uint8_t*>(src_slots),
                           n_src, src_bitmask, src_ids, static_cast<uint8_t*>(dst_slots), n_dst, dst_bitmask, dst_ids,
                           n, h->d_err);
        return hipGetLastError();
    }));
}

uint64_t ibp_pages_workspace(uint64_t n_slots, uint64_t n) {
    // the two move lists of a compaction (uint32 each), or n slot ids
    return 8 * (count_words(n_slots) + 1 + std::max(n_slots, n));
}

static ibp_status check_workspace(ibp_meta_t h, const void* ws, uint64_t bytes, uint64_t need) {
    if (bytes < need || !device_only(ws, h->device) || reinterpret_cast<uintptr_t>(ws) % 16) return IBP_ERR_INVALID_ARG;
    return IBP_OK;
}

// bitmask: NULL, or where the bits of the slots taken become 0.
static ibp_status take_slots(ibp_meta_t h, int32_t* refs, uint64_t n_slots, uint32_t* bitmask, int64_t* ids, uint64_t n,
                             void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
    if (n_slots == 0 || n_slots > kMaxPoolSlots || n > kMaxPoolSlots) return IBP_ERR_INVALID_ARG;
    if (!device_only(refs, h->device) || !device_only(ids, h->device)) return IBP_ERR_INVALID_ARG;
    if (bitmask && !device_only(bitmask, h->device)) return IBP_ERR_INVALID_ARG;
    ibp_status st = check_workspace(h, workspace, workspace_bytes, ibp_pages_workspace(n_slots, 0));
    if (st != IBP_OK) return st;
    uint32_t* counts = static_cast<uint32_t*>(workspace);
    IBP_TRY(launch_count_free(refs, n_slots, counts, stream));
    hipLaunchKernelGGL((k_list_free<true, false>), dim3((uint32_t)count_blocks(n_slots)), dim3(kCountBlock), 0, stream, refs,
                       n_slots, counts, ids, n, bitmask, h->d_err);
    return from_hip(hipGetLastError());
}

ibp_status ibp_pages_alloc(ibp_meta_t h, int32_t* refs, uint64_t n_slots, int64_t* ids, uint64_t n, void* workspace,
                           uint64_t workspace_bytes, hipStream_t stream) {
    if (!h) return IBP_ERR_INVALID_ARG;
    if (n == 0) return IBP_OK;
    DeviceGuard guard(h->device);
    if (!guard.ok) return IBP_ERR_DEVICE;
    return take_slots(h, refs, n_slots, nullptr, ids, n, workspace, workspace_bytes, stream);
}

ibp_status ibp_pages_alloc_raw(ibp_meta_t h, int32_t* refs, uint64_t n_slots, uint32_t* bitmask, int64_t* ids,
                               uint64_t n, void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
    if (!h) return IBP_ERR_INVALID_ARG;
    if (n == 0) return IBP_OK;
    DeviceGuard guard(h->device);
    if (!guard.ok) return IBP_ERR_DEVICE;
    if (!bitmask) return IBP_ERR_INVALID_ARG;
    return take_slots(h, refs, n_slots, bitmask, ids, n, workspace, workspace_bytes, stream);
}

ibp_status ibp_pages_fork(ibp_meta_t h, void* slots, uint64_t n_slots, uint32_t* bitmask, int32_t* refs,
                          int64_t* table, uint64_t n_seqs, uint32_t n_heads, uint64_t table_blocks,
                          const int32_t* lens, uint32_t page_tokens, const int64_t* parents, const int64_t* children,
                          uint64_t n, void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
    if (!h) return IBP_ERR_INVALID_ARG;
    if (n == 0) return IBP_OK;
    DeviceGuard guard(h->device);
    if (!guard.ok) return IBP_ERR_DEVICE;
    if (n_slots == 0 || n_slots > kMaxPoolSlots || n_heads == 0 || page_tokens == 0 || table_blocks == 0 ||
        table_blocks > (1ull << 31) / page_tokens || n_seqs > kMaxPoolSlots)
        return IBP_ERR_INVALID_ARG;
    if (n > max_workgroups(256) / n_heads) return IBP_ERR_UNSUPPORTED;
    if (!device_or_pinned(slots, h->device)) return IBP_ERR_INVALID_ARG;
    for (const void* p : {(const void*)bitmask, (const void*)refs, (const void*)table, (const void*)lens,
                          (const void*)parents, (const void*)children})
        if (!device_only(p, h->device)) return IBP_ERR_INVALID_ARG;
    ibp_status st = check_page_format(h, {slots});
    if (st != IBP_OK) return st;
    st = check_workspace(h, workspace, workspace_bytes, ibp_pages_workspace(n_slots, n * n_heads));
    if (st != IBP_OK) return st;
    uint32_t* counts = static_cast<uint32_t*>(workspace);
    int64_t* fresh = static_cast<int64_t*>(workspace) + count_words(n_slots);
    if (n_slots <= kListSlots) {
        hipLaunchKernelGGL((k_list_free<false, true>), scan_grid(n_slots), dim3(kListBlock), 0, stream, refs, n_slots,
                           nullptr, fresh, n * n_heads, nullptr, h->d_err);
    } else {
        IBP_TRY(launch_count_free(refs, n_slots, counts, stream));
        hipLaunchKernelGGL((k_list_free<false, false>), dim3((uint32_t)count_blocks(n_slots)), dim3(kCountBlock), 0,
                           stream, refs, n_slots, counts, fresh, n * n_heads, nullptr, h->d_err);
    }
    IBP_TRY(hipGetLastError());
    const Geo geo = make_geo(h, true, kLongTileWordsDecode);
    const ForkArgs a{static_cast<const uint8_t*>(slots), static_cast<uint8_t*>(slots), bitmask, refs, table, lens,
                     parents, children, fresh, n_slots, n_seqs, table_blocks, n, n_heads, page_tokens};
    return from_hip(by_vectors(h->params.tensor_bytes, [&](auto nv) {
        hipLaunchKernelGGL((k_pages_fork<decltype(nv)::value>), dim3((uint32_t)(n * n_heads)), dim3(256), 0, stream,
                           h->tabs, geo, a, h->d_err);
        return hipGetLastError();
    }));
}

ibp_status ibp_pages_free(ibp_meta_t h, int32_t* refs, uint64_t n_slots, int64_t* table, uint64_t n_seqs,
                          uint32_t n_heads, uint64_t table_blocks, const int64_t* seqs, uint64_t n,
                          hipStream_t stream) {
    if (!h) return IBP_ERR_INVALID_ARG;
    if (n == 0) return IBP_OK;
    DeviceGuard guard(h->device);
    if (!guard.ok) return IBP_ERR_DEVICE;
    if (n_slots == 0 || n_slots > kMaxPoolSlots || n_heads == 0 || table_blocks == 0 || table_blocks > (1ull << 31))
        return IBP_ERR_INVALID_ARG;
    const uint64_t row = n_heads * table_blocks;
    if (n > (1ull << 62) / row) return IBP_ERR_INVALID_ARG;
    for (const void* p : {(const void*)refs, (const void*)table, (const void*)seqs})
        if (!device_only(p, h->device)) return IBP_ERR_INVALID_ARG;
    hipLaunchKernelGGL(k_pages_free, striding_grid(n * row, 256), dim3(256), 0, stream, refs, n_slots,
                       table, n_seqs, row, seqs, n, h->d_err);
    return from_hip(hipGetLastError());
}

ibp_status ibp_pages_compact(ibp_meta_t h, void* slots, uint64_t n_slots, uint32_t* bitmask, int32_t* refs,
                             int64_t* map, int64_t* n_live, int64_t* table, uint64_t n_entries, void* workspace,
                             uint64_t workspace_bytes, hipStream_t stream) {
    if (!h) return IBP_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (!guard.ok) return IBP_ERR_DEVICE;
    if (n_slots == 0 || n_slots > kMaxPoolSlots || n_entries > 1ull << 62) return IBP_ERR_INVALID_ARG;
    if (!device_or_pinned(slots, h->device)) return IBP_ERR_INVALID_ARG;
    for (const void* p : {(const void*)bitmask, (const void*)refs, (const void*)map, (const void*)n_live})
        if (!device_only(p, h->device)) return IBP_ERR_INVALID_ARG;
    if (n_entries && !device_only(table, h->device)) return IBP_ERR_INVALID_ARG;
    ibp_status st = check_page_format(h, {slots});
    if (st != IBP_OK) return st;
    st = check_workspace(h, workspace, workspace_bytes, ibp_pages_workspace(n_slots, 0));
    if (st != IBP_OK) return st;
    uint32_t* counts = static_cast<uint32_t*>(workspace);
    uint64_t* n_moves = static_cast<uint64_t*>(workspace) + count_words(n_slots);
    uint32_t* holes = reinterpret_cast<uint32_t*>(n_moves + 1);
    uint32_t* movers = holes + n_slots;
    if (n_slots <= kPlanSlots) {
        hipLaunchKernelGGL(k_compact_plan<true>, scan_grid(n_slots), dim3(kListBlock), 0, stream, refs, n_slots,
                           nullptr, map, n_live, n_moves, holes, movers);
    } else {
        IBP_TRY(launch_count_free(refs, n_slots, counts, stream));
        hipLaunchKernelGGL(k_compact_plan<false>, dim3((uint32_t)count_blocks(n_slots)), dim3(kCountBlock), 0, stream,
                           refs, n_slots, counts, map, n_live, n_moves, holes, movers);
    }
    IBP_TRY(hipGetLastError());
    const Geo geo = make_geo(h, true, kLongTileWordsDecode);
    // at most half of the pool moves
    const uint64_t most = (n_slots / 2 + kPageWaves) / kPageWaves;
    const uint32_t grid = (uint32_t)std::min<uint64_t>(most, 16ull * h->cu_count);
    IBP_TRY(by_vectors(h->params.tensor_bytes, [&](auto nv) {
        hipLaunchKernelGGL((k_compact_move<decltype(nv)::value>), dim3(grid), dim3(kWave * kPageWaves), 0, stream,
                           h->tabs, geo, static_cast<uint8_t*>(slots), bitmask, refs, map, n_moves, holes, movers,
                           h->d_err);
        return hipGetLastError();
    }));
    if (n_entries) {
        hipLaunchKernelGGL(k_remap, striding_grid(n_entries, 256), dim3(256), 0, stream, map, n_slots,
                           table, n_entries, h->d_err);
        IBP_TRY(hipGetLastError());
    }
    return IBP_OK;
}

}  // extern "C"
