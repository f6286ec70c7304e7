// ibp_kv_math.hpp -- number types and matrix-core forms of the page operators,
// and the argument checks that their entry points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ibp_host.hpp"
#include "ibp_kv_device.hpp"

namespace ibp {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

template <class To, class From>
__device__ __forceinline__ To bits_as(const From& x) {
    static_assert(sizeof(To) == sizeof(From), "same size");
    return __builtin_bit_cast(To, x);
}

// D = A B + C on 16 x 16 with 32 products per number: lane l holds row (A) or
// column (B) l % 16 and k = 8 (l / 16) .. + 7; of D, column l % 16 and rows
// 4 (l / 16) .. + 3.
struct Bf16 {
    using V8 = bf16x8;
    static __device__ __forceinline__ float from_bits(uint32_t b) { return __uint_as_float(b << 16); }
    // two floats to nearest even, the first in the low half
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        typedef __bf16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, v2{(__bf16)a, (__bf16)b});
    }
    static __device__ __forceinline__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // all exponent bits set in either half: an infinity or a NaN
    static constexpr uint32_t kExponent = 0x7F80u;
    // octaves above 1 at which the largest softmax weight is kept (see raise)
    static constexpr float kLead = 0.f;
};

struct Fp16 {
    using V8 = f16x8;
    static __device__ __forceinline__ float from_bits(uint32_t b) {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        typedef _Float16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, v2{(_Float16)a, (_Float16)b});
    }
    static __device__ __forceinline__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static constexpr uint32_t kExponent = 0x7C00u;
    static constexpr float kLead = 7.f;
};

// Eight numbers of a dense row, which need not start on more than two bytes
// (the memory of this GPU takes 16-byte reads at any address).
__device__ __forceinline__ u32x4 load_eight(const uint16_t* p) {
    typedef u32x4 u32x4_any __attribute__((aligned(2)));
    return *reinterpret_cast<const u32x4_any*>(p);
}

// The pool of k as the kernels see it.
inline ibp_status make_pool(const ibp_pages* k, int device, Pool* out) {
    if (!k || !k->meta || k->meta->device != device) return IBP_ERR_INVALID_ARG;
    const ibp_meta_s* h = k->meta;
    if (k->n_slots == 0 || k->n_slots > kMaxPoolSlots) return IBP_ERR_INVALID_ARG;
    if (!device_or_pinned(k->slots, device) || !device_only(k->bitmask, device)) return IBP_ERR_INVALID_ARG;
    if (!aligned16(h->params.tensor_bytes, {k->slots})) return IBP_ERR_UNSUPPORTED;
    // the tables' rows as Pool describes them
    if (h->tabs.b != h->tabs.kd - h->Mw || h->tabs.dx != h->tabs.kd + h->Mw || h->tabs.r != h->tabs.kd + 5ull * h->Mw)
        return IBP_ERR_UNSUPPORTED;
    const uint64_t chunks = 8 * h->params.tensor_bytes / h->params.chunk_bits;
    out->slots = static_cast<const uint8_t*>(k->slots);
    out->bitmask = k->bitmask;
    out->err = h->d_err;
    out->tab = h->tabs.kd;
    out->n_slots = (uint32_t)k->n_slots;
    out->Mw = h->sum.uniform ? 1u : h->Mw;
    out->src_Mw = h->Mw;
    out->runs = h->sum.max_runs;
    out->log2g = h->log2g;
    out->hw = (uint32_t)((chunks + 31) / 32);
    out->valid = (uint32_t)(chunks - 32ull * (out->hw - 1));
    return IBP_OK;
}

// What every operator with queries asks of its shape.
inline ibp_status check_attention(const ibp_attention* a) {
    if (a->dtype > IBP_FP16 || a->n_kv_heads == 0 || a->n_q_heads == 0 || a->n_q_heads % a->n_kv_heads != 0)
        return IBP_ERR_INVALID_ARG;
    if (a->n_q_heads > 65535) return IBP_ERR_UNSUPPORTED;
    if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256) return IBP_ERR_UNSUPPORTED;
    if (a->page_tokens != 16 && a->page_tokens != 32 && a->page_tokens != 64) return IBP_ERR_UNSUPPORTED;
    if ((uint64_t)a->head_dim * a->page_tokens * 2 > kMaxPageBytes) return IBP_ERR_UNSUPPORTED;
    if (a->n_rows && (a->n_seqs == 0 || a->table_blocks == 0)) return IBP_ERR_INVALID_ARG;
    if (a->table_blocks > (1ull << 31) / a->page_tokens || a->n_seqs > (1ull << 31) || a->n_rows > (1ull << 31))
        return IBP_ERR_INVALID_ARG;
    if (a->q_row_stride < 0 || a->q_head_stride < 0) return IBP_ERR_INVALID_ARG;
    return IBP_OK;
}

}  // namespace ibp
