// ibp_attention.hip -- entry points of attention over pages: argument checks
// and the shape of the launch.  The kernels are in ibp_attention.hpp.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <limits>

#include "../../include/ibp.h"
#include "ibp_attention.hpp"

using namespace ibp;

namespace {

// Waves that a launch should have: eight per compute unit of an MI355X.
constexpr uint64_t kTargetWaves = 2048;
constexpr uint64_t kMaxSplits = 256;

// Rows per workgroup, split of the context, LDS.  `rows`: most rows of one
// (sequence or row, key/value head).
AttnPlan plan_attention(const ibp_attention* a, bool tree, uint64_t items, uint64_t rows, uint64_t tokens,
                        uint64_t new_tokens) {
    AttnPlan p;
    const uint32_t D = a->head_dim, T = a->page_tokens;
    const uint32_t m2 = D <= 128 ? 2 : 1;
    p.many = tree && rows > 16 * m2;
    const uint32_t waves = p.many ? kManyWaves : kFewWaves;
    p.mr = rows <= (p.many ? 16u * kManyWaves : 16u) ? 1 : 2;
    const uint64_t per_wg = 16ull * (p.mr == 1 ? 1 : m2) * (p.many ? kManyWaves : 1);
    p.row_tiles = (uint32_t)((rows + per_wg - 1) / per_wg);
#define IBP_SHAPE(DD, TT)                                                                      \
    if (D == DD && T == TT) {                                                                  \
        p.step = p.many ? ManyShape<DD, TT>::STEP : FewShape<DD, TT>::STEP;                    \
        p.area_bytes = p.many ? ManyShape<DD, TT>::area_bytes : FewShape<DD, TT>::area_bytes;  \
    }
    IBP_SHAPE(64, 16)
    IBP_SHAPE(64, 32)
    IBP_SHAPE(64, 64)
    IBP_SHAPE(128, 16)
    IBP_SHAPE(128, 32)
    IBP_SHAPE(256, 16)
#undef IBP_SHAPE
    const uint64_t steps = (tokens + p.step - 1) / p.step + (new_tokens + p.step - 1) / p.step;
    const uint64_t groups = items * a->n_kv_heads * p.row_tiles;
    const uint64_t target = kTargetWaves / waves;
    const uint64_t least = p.many ? 2 : kFewWaves;  // steps that make a split worth joining
    const uint64_t most = std::max<uint64_t>(1, (steps + least - 1) / least);
    p.splits = (uint32_t)std::min({most, (target + groups - 1) / groups, kMaxSplits});
    return p;
}

uint64_t part_floats(const ibp_attention* a, uint32_t splits) {
    return splits == 1 ? 0 : a->n_rows * a->n_q_heads * splits * (a->head_dim + 2ull);
}

uint64_t context_hint(const ibp_attention* a) {
    const uint64_t held = a->table_blocks * a->page_tokens;
    return a->max_len && a->max_len < held ? a->max_len : held;
}

AttnPlan plan_tree(const ibp_attention* a) {
    return plan_attention(a, true, a->n_seqs, (uint64_t)a->max_new * (a->n_q_heads / a->n_kv_heads),
                          context_hint(a), a->max_new);
}

AttnPlan plan_sparse(const ibp_attention* a, uint32_t n_blocks) {
    return plan_attention(a, false, a->n_rows, a->n_q_heads / a->n_kv_heads, (uint64_t)n_blocks * a->page_tokens, 0);
}

// The parts of AttnArgs that both operators fill alike, and the LDS.
ibp_status fill_args(const ibp_pages* k, const ibp_pages* v, const ibp_attention* a, const void* q,
                     const int64_t* k_table, const int64_t* v_table, const int32_t* lens, void* out, float* lse,
                     void* workspace, uint64_t workspace_bytes, const AttnPlan& p, uint64_t items, AttnArgs* x,
                     uint32_t* lds) {
    const int dev = k->meta->device;
    ibp_status st = make_pool(k, dev, &x->k);
    if (st == IBP_OK) st = make_pool(v, dev, &x->v);
    if (st != IBP_OK) return st;
    const uint64_t L = (uint64_t)a->head_dim * a->page_tokens * 2;
    if (k->meta->params.tensor_bytes != L || v->meta->params.tensor_bytes != L) return IBP_ERR_INVALID_ARG;
    for (const void* ptr : {q, (const void*)k_table, (const void*)v_table, (const void*)lens, (const void*)out})
        if (!device_only(ptr, dev)) return IBP_ERR_INVALID_ARG;
    if (lse && !device_only(lse, dev)) return IBP_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(out) % 8 || reinterpret_cast<uintptr_t>(q) % 2) return IBP_ERR_INVALID_ARG;
    const uint64_t need = 4 * part_floats(a, p.splits);
    if (need) {
        if (workspace_bytes < need || !device_only(workspace, dev) || reinterpret_cast<uintptr_t>(workspace) % 16)
            return IBP_ERR_INVALID_ARG;
    }
    const uint64_t groups = items * a->n_kv_heads * p.row_tiles * p.splits;
    if (groups > max_workgroups(kWave * std::max(kFewWaves, kManyWaves)) ||
        (p.splits > 1 && a->n_rows * a->n_q_heads * (a->head_dim / 4) > kMaxLaunchThreads - 255))
        return IBP_ERR_UNSUPPORTED;
    x->q = static_cast<const uint16_t*>(q);
    x->k_table = k_table;
    x->v_table = v_table;
    x->lens = lens;
    x->out = static_cast<uint16_t*>(out);
    x->lse = lse;
    x->part = static_cast<float*>(workspace);
    x->part_ml = x->part + a->n_rows * a->n_q_heads * p.splits * a->head_dim;
    x->n_rows = a->n_rows;
    x->n_seqs = a->n_seqs;
    x->table_blocks = a->table_blocks;
    x->q_row = a->q_row_stride;
    x->q_head = a->q_head_stride;
    x->kv_heads = a->n_kv_heads;
    x->group = a->n_q_heads / a->n_kv_heads;
    x->splits = p.splits;
    x->row_tiles = p.row_tiles;
    x->work = (uint32_t)(items * a->n_kv_heads);
    // a scale of zero weighs all keys alike: the smallest number of 32 bits
    // leaves scores below 1e-6, and masked ones -infinity
    x->scale2 = std::max(std::fabs(a->scale) * kLog2e, std::numeric_limits<float>::denorm_min());
    x->q_sign = a->scale < 0.f ? 0x80008000u : 0u;
    // Tables in LDS where they fit; large ones otherwise stay in device memory
    // (small ones, of fewer than four positions, always fit).
    x->same_tab = k->meta == v->meta;
    const uint64_t wk = page_tab_words(x->k.Mw, x->k.runs);
    const uint64_t wv = x->same_tab ? 0 : page_tab_words(x->v.Mw, x->v.runs);
    uint64_t room = kLdsLimit - p.area_bytes;
    x->tab_lds_k = 4 * wk <= room;
    if (x->tab_lds_k) room -= 4 * wk;
    x->tab_lds_v = x->same_tab ? x->tab_lds_k : 4 * wv <= room;
    x->tab_words_k = x->tab_lds_k ? (uint32_t)wk : 0;
    x->tab_words_v = x->tab_lds_v ? (uint32_t)wv : 0;
    *lds = p.area_bytes + 4 * (x->tab_words_k + x->tab_words_v);
    return IBP_OK;
}

ibp_status launch(const AttnArgs& x, const AttnPlan& p, const ibp_attention* a, bool tree, uint32_t lds,
                  hipStream_t stream) {
    return from_hip(a->dtype == IBP_BF16
                        ? launch_attention_bf16(x, p, a->head_dim, a->page_tokens, tree, lds, stream)
                        : launch_attention_fp16(x, p, a->head_dim, a->page_tokens, tree, lds, stream));
}

}  // namespace

extern "C" {

uint64_t ibp_tree_attention_workspace(const ibp_attention* a) {
    if (!a || check_attention(a) != IBP_OK || a->max_new == 0 || a->n_rows == 0) return 0;
    return 4 * part_floats(a, plan_tree(a).splits);
}

ibp_status ibp_tree_attention(const ibp_pages* k, const ibp_pages* v, const ibp_attention* a, const void* q,
                              const int64_t* k_table, const int64_t* v_table, const int32_t* lens,
                              const int32_t* new_rows, const void* k_new, const void* v_new, const uint64_t* mask,
                              uint32_t mask_words, void* out, float* lse, void* workspace, uint64_t workspace_bytes,
                              hipStream_t stream) {
    if (!k || !v || !a || !k->meta || !v->meta) return IBP_ERR_INVALID_ARG;
    const int dev = k->meta->device;
    DeviceGuard guard(dev);
    if (!guard.ok) return IBP_ERR_DEVICE;
    ibp_status st = check_attention(a);
    if (st != IBP_OK) return st;
    if (a->n_rows == 0) return IBP_OK;
    if (a->max_new == 0 || mask_words == 0 || mask_words > (1u << 20) || a->max_new > (1u << 20) ||
        a->new_row_stride < 0 || a->new_head_stride < 0 || a->new_row_stride >= (1ll << 30))
        return IBP_ERR_INVALID_ARG;
    for (const void* p : {(const void*)new_rows, k_new, v_new, (const void*)mask})
        if (!device_only(p, dev)) return IBP_ERR_INVALID_ARG;
    if ((uint64_t)a->max_new * (a->n_q_heads / a->n_kv_heads) > 0x7FFFFFFFull) return IBP_ERR_UNSUPPORTED;
    const AttnPlan p = plan_tree(a);
    AttnArgs x{};
    uint32_t lds = 0;
    st = fill_args(k, v, a, q, k_table, v_table, lens, out, lse, workspace, workspace_bytes, p, a->n_seqs, &x, &lds);
    if (st != IBP_OK) return st;
    x.new_rows = new_rows;
    x.k_new = static_cast<const uint16_t*>(k_new);
    x.v_new = static_cast<const uint16_t*>(v_new);
    x.mask = reinterpret_cast<const uint32_t*>(mask);
    x.mask_words2 = 2 * mask_words;
    x.max_new = a->max_new;
    x.new_row = a->new_row_stride;
    x.new_head = a->new_head_stride;
    return launch(x, p, a, true, lds, stream);
}

uint64_t ibp_sparse_attention_workspace(const ibp_attention* a, uint32_t n_blocks) {
    if (!a || check_attention(a) != IBP_OK || n_blocks == 0 || a->n_rows == 0) return 0;
    return 4 * part_floats(a, plan_sparse(a, n_blocks).splits);
}

ibp_status ibp_sparse_attention(const ibp_pages* k, const ibp_pages* v, const ibp_attention* a, const void* q,
                                const int64_t* k_table, const int64_t* v_table, const int32_t* lens,
                                const int32_t* row_seq, const int32_t* blocks, uint32_t n_blocks, void* out,
                                float* lse, void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
    if (!k || !v || !a || !k->meta || !v->meta) return IBP_ERR_INVALID_ARG;
    const int dev = k->meta->device;
    DeviceGuard guard(dev);
    if (!guard.ok) return IBP_ERR_DEVICE;
    ibp_status st = check_attention(a);
    if (st != IBP_OK) return st;
    if (a->n_rows == 0) return IBP_OK;
    if (n_blocks == 0 || n_blocks > (1u << 26)) return IBP_ERR_INVALID_ARG;
    if (!row_seq && a->n_rows > a->n_seqs) return IBP_ERR_INVALID_ARG;
    if (!device_only(blocks, dev) || (row_seq && !device_only(row_seq, dev))) return IBP_ERR_INVALID_ARG;
    const AttnPlan p = plan_sparse(a, n_blocks);
    AttnArgs x{};
    uint32_t lds = 0;
    st = fill_args(k, v, a, q, k_table, v_table, lens, out, lse, workspace, workspace_bytes, p, a->n_rows, &x, &lds);
    if (st != IBP_OK) return st;
    x.row_seq = row_seq;
    x.blocks = blocks;
    x.n_list = n_blocks;
    return launch(x, p, a, false, lds, stream);
}

}  // extern "C"
