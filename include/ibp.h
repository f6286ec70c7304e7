/*
 * ibp.h -- C ABI of libibp, an MI355X (gfx950) implementation of Invariant
 * Bit Packing (IBP), a lossless codec for ML tensors.
 *
 * Sources cited below:
 *   FR summary = gist.science French technical summary of arXiv 2605.30728,
 *     "Résumé Technique : Réduire le goulot d'étranglement de la mémoire GPU
 *     par la compression sans perte pour le ML";
 *   KO summary = its Korean counterpart, "Reducing the GPU Memory
 *     Bottleneck with Lossless Compression for ML -- Extended".
 * Both describe the method in section "Algorithme central" / "핵심 알고리즘"
 * (1 preprocessing, 2 compression, 3 decompression) and its use in section
 * "Intégration au système" / "시스템 통합" (fixed-size slots, GPU bitmask).
 *
 * Format (the pages fix no bit layout; this is the layout every call uses):
 *   - a tensor of L bytes is a bit string, bit i = bit (i mod 32) of
 *     little-endian 32-bit word i/32; chunk c = bits [c*W, c*W + W);
 *   - Mask/Bitval are M-bit strings (M/32 words, same bit order); chunk c
 *     is tested against their bits (c*W .. c*W+W-1) mod M;
 *   - a record = n = 8L/W participation bits (1 = the chunk matched and lost
 *     its masked bits), zero padded to H = 32*ceil(n/32) bits, then each
 *     chunk's kept bits in chunk order and ascending bit position, then zero
 *     bits up to a multiple of 32 (R bits before padding);
 *   - slot t (L bytes at slots + t*L) holds the record when
 *     4*ceil(R/32) < L and bitmask bit t is 1; otherwise the slot holds the
 *     tensor unchanged and the bit is 0.  Bitmask bit t is bit t%32 of word
 *     t/32.  Slot bytes after a record are unspecified.
 *
 * Memory kinds.  "device" = hipMalloc'd memory of the handle's GPU.
 * "device or pinned" = device memory or page-locked host memory
 * (hipHostMalloc / torch pin_memory), which kernels read or write directly
 * over the host link (zero copy).  Pageable host memory is rejected with
 * IBP_ERR_INVALID_ARG.  The caller owns and frees every buffer passed in;
 * the library owns only what an ibp_meta_t holds.
 *
 * Calls are asynchronous on `stream` unless stated; argument checks happen
 * on the host before any launch and leave outputs untouched on error.  Errors
 * found by kernels (an id out of range, a corrupt record) are latched in the
 * handle and reported by ibp_check().  Calls on one handle may run on
 * different streams at once; calls on the same stream run in order, also
 * when several host threads issue them.
 *
 * Tensors longer than one tile (more than 8 KiB) are cut into tiles whose
 * start bits need per-stream scratch of the handle: an encode of a source in
 * pinned host memory, and a decode of records read over the host link, find
 * them by a decoupled look-back; an encode of a 16-byte aligned source in
 * device memory computes them first from the source (a pass over it and a
 * scan per tensor), and a decode of records in device memory from the header
 * words (likewise).  ibp_compress,
 * ibp_decompress and ibp_gather_decompress of such tensors, and
 * ibp_packed_offsets, return IBP_ERR_UNSUPPORTED while `stream` is capturing
 * a HIP graph; single-tile calls may be captured.
 */
#ifndef IBP_H
#define IBP_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ibp_status {
    IBP_OK = 0,
    IBP_ERR_INVALID_ARG = -1, /* bad size, pointer kind or parameter */
    IBP_ERR_UNSUPPORTED = -2, /* valid format this GPU path does not implement */
    IBP_ERR_DEVICE = -3,      /* a HIP call failed */
    IBP_ERR_NOMEM = -4,       /* device or host allocation failed */
    IBP_ERR_CORRUPT = -5,     /* a compressed slot holds no valid record */
    IBP_ERR_RANGE = -6,       /* a gather id lies outside [0, n_slots) */
    IBP_ERR_TOO_LARGE = -7    /* more tiles than ibp_decompress_noalloc's static scratch holds */
} ibp_status;

typedef struct ibp_meta_s* ibp_meta_t; /* opaque, owned by the library */

typedef struct ibp_params {
    uint64_t tensor_bytes; /* L: multiple of 4; multiple of W/8 and of M/8        */
    uint32_t chunk_bits;   /* W: 32, 64, 128, 256, 512 or 1024                    */
    uint32_t period_bits;  /* M: multiple of W that divides 8L, at most 2^20      */
    double threshold;      /* T in (0.5, 1]; read by ibp_build_metadata only      */
} ibp_params;

/* Derived facts about a handle's metadata. */
typedef struct ibp_meta_info {
    uint64_t invariant_bits;    /* popcount(Mask) over the M-bit period            */
    uint64_t min_record_bytes;  /* record bytes when every chunk matches           */
    uint32_t max_runs;          /* most runs of kept (unmasked) bits in one word   */
    uint32_t uniform;           /* 1 when every 32-bit Mask/Bitval word is equal   */
} ibp_meta_info;

/* Step 1, preprocessing (FR/KO summary, "Algorithme central" step 1).
 * sample: n_sample tensors of L bytes, contiguous, device or pinned.  Every
 * M-bit block of the sample is one observation; bit position j (0 <= j < M)
 * is invariant when at least K = ceil(T * n_obs) observations agree on it
 * (product rounded to nearest in IEEE double, then ceiling), and Bitval
 * keeps the agreed value there (0 elsewhere).  The histogram runs on the GPU;
 * the call then waits for `stream` and keeps a host copy of Mask/Bitval, so
 * it is synchronous.  n_sample * 8L / M must lie in [1, 2^32).  *out
 * receives a new handle bound to the current HIP device. */
ibp_status ibp_build_metadata(const ibp_params* params, const void* sample, uint64_t n_sample,
                              ibp_meta_t* out, hipStream_t stream);

/* A handle from Mask/Bitval given in host memory (M/32 words each; Bitval
 * bits outside Mask must be 0).  Lets metadata be saved and reused for a
 * whole dataset (FR/KO summary, step 1, last bullet).  Synchronous. */
ibp_status ibp_meta_create(const ibp_params* params, const uint32_t* mask, const uint32_t* bitval,
                           ibp_meta_t* out, hipStream_t stream);

/* Copies the parameters and Mask/Bitval (M/32 words each) to host memory;
 * any output pointer may be NULL. */
ibp_status ibp_meta_get(ibp_meta_t meta, ibp_params* params, uint32_t* mask, uint32_t* bitval);

ibp_status ibp_meta_get_info(ibp_meta_t meta, ibp_meta_info* info);

/* Tuning: bytes of a compressed slot that decode reads before it has seen
 * the record header (a record's length is known only from its header, so a
 * second read fetches the rest).  0 restores the default: the largest
 * 256-byte-aligned prefix no record can be shorter than, but at least 256
 * bytes -- or fewer whole 128-byte lines when the median record of the
 * metadata sample fits in them -- or the whole slot when the shortest
 * possible record spans all but at most 1/16 of the slot's 128-byte lines.
 * Rounded up to a multiple of 16 bytes and to at least the header; capped at
 * the slot.  Affects later decode calls on any stream, except decodes of
 * tensors of at most 1 KiB from slots in GPU memory in launches of at most
 * 128 rows per compute unit, which read each slot whole in one pass. */
ibp_status ibp_meta_set_first_read(ibp_meta_t meta, uint64_t bytes);

/* Waits for all work on the handle's GPU, then frees the handle. */
ibp_status ibp_meta_destroy(ibp_meta_t meta);

/* Step 2, compression (FR/KO summary, "Algorithme central" step 2, and
 * "Intégration au système": fixed slots and a bitmask in GPU memory).
 * src: n_tensors tensors of L bytes (device or pinned).  dst_slots:
 * n_tensors slots of L bytes (device or pinned), must not overlap src.
 * bitmask: device, ceil(n_tensors/32) words; bits 0..n_tensors-1 are
 * written, later bits of the last word are left as they were.
 * stored_bytes: device or NULL; entry t = 4*ceil(R/32) for a compressed
 * slot, L for a raw one. */
ibp_status ibp_compress(ibp_meta_t meta, const void* src, uint64_t n_tensors, void* dst_slots,
                        uint32_t* bitmask, uint64_t* stored_bytes, hipStream_t stream);

/* Step 3, decompression (FR/KO summary, "Algorithme central" step 3):
 * tensor t of dst (device, n_tensors * L bytes) <- slot t of slots (device
 * or pinned).  Only the record prefix of a compressed slot is read.  A
 * compressed slot whose header has non-zero padding bits or implies
 * 4*ceil(R/32) >= L latches IBP_ERR_CORRUPT; its output bytes are then
 * unspecified. */
ibp_status ibp_decompress(ibp_meta_t meta, const void* slots, const uint32_t* bitmask,
                          uint64_t n_tensors, void* dst, hipStream_t stream);

/* Gather on decode: row i of dst (device, n_ids * L bytes) <- slot ids[i]
 * of slots (n_slots slots, device or pinned).  ids: device int64, repeats
 * allowed.  An id outside [0, n_slots) latches IBP_ERR_RANGE and leaves that
 * row unspecified; corrupt records as for ibp_decompress. */
ibp_status ibp_gather_decompress(ibp_meta_t meta, const void* slots, uint64_t n_slots,
                                 const uint32_t* bitmask, const int64_t* ids, uint64_t n_ids,
                                 void* dst, hipStream_t stream);

/* ibp_decompress for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, contract and output as ibp_decompress.  It calls no
 * hipMalloc/hipFree: the start-bit scratch of tensors longer than one tile
 * (L > 8 KiB) lives in one static device array of IBP_NOALLOC_SCRATCH_BYTES
 * per GPU, part of the library's code object and held until the process
 * ends (its address is looked up with hipGetSymbolAddress on the first call
 * on each device).  Each call zeroes the part it uses with fill kernels on
 * `stream` (no memset), so a call may be captured and replayed.  At most
 * IBP_NOALLOC_MAX_TILES tiles per call, a tile being 8 KiB of one tensor
 * (n_tensors * ceil(L / 8192) when L > 8192); beyond that the call returns
 * IBP_ERR_TOO_LARGE before anything is queued.  Every call on a GPU shares
 * its array: calls that overlap in time on one GPU (other streams, other
 * handles, other host threads) race on it and their outputs are then
 * unspecified; calls queued on one stream run one after the other. */
#define IBP_NOALLOC_SCRATCH_BYTES (1u << 20)
#define IBP_NOALLOC_MAX_TILES (IBP_NOALLOC_SCRATCH_BYTES / 8u - 32u)
ibp_status ibp_decompress_noalloc(ibp_meta_t meta, const void* slots, const uint32_t* bitmask,
                                  uint64_t n_tensors, void* dst, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Packed cache (FR/KO summary, "Intégration au système": in the GPU software
 * cache of GNN frameworks, compressing the cached tensors raises how many of
 * them fit).  Instead of fixed L-byte slots, the items -- what slot t would
 * hold: the record when 4*ceil(R/32) < L, else the raw tensor -- are stored
 * back to back.  Item t spans bytes [offsets[t], offsets[t+1]) of the buffer;
 * offsets[0] = 0 and offsets[t+1] = offsets[t] + the item's bytes rounded up
 * to a multiple of 16 (the bytes after an item up to the next offset are
 * zero).  offsets: device memory, n + 1 uint64 entries, 8-byte aligned.  The
 * bitmask is the same as for slots.
 *
 * These calls need L to be a multiple of 16 and at most 8 KiB, 16-byte
 * aligned data pointers, and per-position tables that fit the kernels' LDS
 * (every workload shape of the benchmark does); otherwise they return
 * IBP_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------- */

/* offsets <- the item offsets of the n_tensors tensors at src (device or
 * pinned); offsets[n_tensors] is the buffer size ibp_compress_packed needs.
 * Reads src once (the record lengths only).  Asynchronous. */
ibp_status ibp_packed_offsets(ibp_meta_t meta, const void* src, uint64_t n_tensors, uint64_t* offsets,
                              hipStream_t stream);

/* Writes item t of src at dst + offsets[t] (dst: device or pinned, capacity
 * bytes, must not overlap src) and bitmask bits 0..n_tensors-1.  offsets
 * must come from ibp_packed_offsets for the same src and handle: an item
 * whose offsets disagree with its length is not written and latches
 * IBP_ERR_CORRUPT, one that would end past capacity latches IBP_ERR_RANGE. */
ibp_status ibp_compress_packed(ibp_meta_t meta, const void* src, uint64_t n_tensors, const uint64_t* offsets,
                               void* dst, uint64_t capacity, uint32_t* bitmask, hipStream_t stream);

/* Tensor t of dst (device, n_items * L bytes) <- item t of the packed
 * buffer buf (device or pinned, buf_bytes bytes).  Each item is read whole
 * in one pass, its length being known from the offsets.  An item whose
 * offsets are not 16-byte multiples, pass buf_bytes, exceed L rounded up to
 * 16, or do not hold its record (or, raw, the whole tensor) latches
 * IBP_ERR_CORRUPT; no byte outside [offsets[t], offsets[t+1]) is read. */
ibp_status ibp_decompress_packed(ibp_meta_t meta, const void* buf, uint64_t buf_bytes, const uint64_t* offsets,
                                 const uint32_t* bitmask, uint64_t n_items, void* dst, hipStream_t stream);

/* Gather on decode from a packed buffer: row i of dst <- item ids[i]
 * (device int64, repeats allowed; an id outside [0, n_items) latches
 * IBP_ERR_RANGE). */
ibp_status ibp_gather_decompress_packed(ibp_meta_t meta, const void* buf, uint64_t buf_bytes,
                                        const uint64_t* offsets, uint64_t n_items, const uint32_t* bitmask,
                                        const int64_t* ids, uint64_t n_ids, void* dst, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Headers in GPU memory ("Intégration au système" keeps the bitmask of
 * compressed slots in GPU memory; this layout keeps each compressed tensor's
 * header words there too).  Zero-copy reads of pinned host memory move whole
 * 128-byte lines, so a record of 4 + 128*j bytes costs j + 1 lines while its
 * payload alone costs j; with the header in GPU memory the decoder also knows
 * the payload length before it reads the slot, and reads it in one pass.
 *
 * Same compressed/raw decision as ibp_compress.  headers: device memory,
 * n * hw uint32 (hw = ceil(n_chunks/32), at most 4, i.e. at most 128 chunks
 * per tensor), 4-byte aligned; entry t*hw .. t*hw+hw-1 holds tensor t's
 * header words, zero for a raw tensor.  Slot t holds the record's payload
 * words (the record minus its header) when compressed, else the tensor; slot
 * bytes after the payload are unspecified.  stored_bytes (device or NULL):
 * payload bytes, or L when raw.  Needs L a multiple of 16 and at most 8 KiB,
 * 16-byte aligned data pointers and tables that fit the kernels' LDS;
 * otherwise IBP_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------- */
ibp_status ibp_compress_split(ibp_meta_t meta, const void* src, uint64_t n_tensors, void* dst_slots,
                              uint32_t* headers, uint32_t* bitmask, uint64_t* stored_bytes, hipStream_t stream);

/* Tensor t of dst (device) <- slot t (device or pinned) with its header
 * words from headers.  A compressed tensor whose header padding bits are set
 * or whose header implies 4*ceil(R/32) >= L latches IBP_ERR_CORRUPT. */
ibp_status ibp_decompress_split(ibp_meta_t meta, const void* slots, const uint32_t* headers,
                                const uint32_t* bitmask, uint64_t n_tensors, void* dst, hipStream_t stream);

/* Gather on decode in that layout: row i of dst <- tensor ids[i] (device
 * int64; an id outside [0, n_slots) latches IBP_ERR_RANGE). */
ibp_status ibp_gather_decompress_split(ibp_meta_t meta, const void* slots, uint64_t n_slots,
                                       const uint32_t* headers, const uint32_t* bitmask, const int64_t* ids,
                                       uint64_t n_ids, void* dst, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Pages of a key/value cache.  A pool is fixed slots with their bitmask, as
 * ibp_compress leaves them: a closed page may be a record (bit 1), the page
 * that is still being filled is a raw slot (bit 0, see ibp_pages_alloc_raw)
 * that the caller writes in place.  A block table (device int64, row-major) holds the slot ids of a
 * sequence's pages in order, -1 where there is none; refs (device int32, one
 * per slot) counts who holds a page, 0 = free.
 *
 * The calls below need pages of at most 8 KiB that are a multiple of 16
 * bytes, 16-byte aligned slots and at most 2^32 - 2 of them; otherwise they
 * return IBP_ERR_UNSUPPORTED or IBP_ERR_INVALID_ARG.  None allocates memory
 * or reads results on the host, so every one may be captured in a HIP graph;
 * scratch comes from the caller (`workspace`, device, 16-byte aligned), and
 * two calls that may overlap in time must not share it.  Ids that are neither
 * -1 nor a slot latch IBP_ERR_RANGE.  A call forks at most 2^24 - 1 rows of
 * the table (forks times heads); more return IBP_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------- */

/* The item of slot src_ids[i] (its record, or the whole raw page) and its
 * bitmask bit -> slot dst_ids[i], without decoding; entries whose source or
 * destination is -1 are skipped.  Only a record's bytes move, so pages go to
 * and from pinned host memory at their compressed size; destination bytes
 * past the item stay as they were.  The pools may be one (no destination may
 * then be the source of another entry) or must not overlap; destinations
 * must be distinct.  A record that is not valid is copied as a whole slot
 * and latches IBP_ERR_CORRUPT. */
ibp_status ibp_pages_copy(ibp_meta_t meta, const void* src_slots, uint64_t n_src, const uint32_t* src_bitmask,
                          const int64_t* src_ids, void* dst_slots, uint64_t n_dst, uint32_t* dst_bitmask,
                          const int64_t* dst_ids, uint64_t n, hipStream_t stream);

/* Workspace bytes of the next calls: n = 0 for ibp_pages_alloc,
 * ibp_pages_alloc_raw and ibp_pages_compact, forks * heads for
 * ibp_pages_fork. */
uint64_t ibp_pages_workspace(uint64_t n_slots, uint64_t n);

/* ids[0..n) <- the n lowest free slots in ascending order, whose counts
 * become 1.  With fewer free slots the rest of ids is -1 and IBP_ERR_NOMEM
 * is latched.  The slots' bitmask bits stay as they were, 1 where a record was
 * freed: for slots that ibp_pages_copy or an encode will fill. */
ibp_status ibp_pages_alloc(ibp_meta_t meta, int32_t* refs, uint64_t n_slots, int64_t* ids, uint64_t n,
                           void* workspace, uint64_t workspace_bytes, hipStream_t stream);

/* The same for pages that the caller writes in place: the bits of the slots
 * handed out become 0 (raw). */
ibp_status ibp_pages_alloc_raw(ibp_meta_t meta, int32_t* refs, uint64_t n_slots, uint32_t* bitmask, int64_t* ids,
                               uint64_t n, void* workspace, uint64_t workspace_bytes, hipStream_t stream);

/* Sequence children[i] becomes a fork of sequence parents[i] (device int64,
 * rows of table: n_seqs x n_heads x table_blocks ids): the lens[parent] /
 * page_tokens full pages are shared (their counts grow by one), a partly
 * filled page after them is copied into the lowest free slots, in the order
 * of i and then of heads, and the rest of the child's row becomes -1.  The
 * child's former row is overwritten, not released; lens is only read.
 * Children must be distinct and no child a parent in the same call; a pair
 * that is not valid latches IBP_ERR_RANGE and is left out, and a page for
 * which no slot is free becomes -1 and latches IBP_ERR_NOMEM. */
ibp_status ibp_pages_fork(ibp_meta_t meta, void* slots, uint64_t n_slots, uint32_t* bitmask, int32_t* refs,
                          int64_t* table, uint64_t n_seqs, uint32_t n_heads, uint64_t table_blocks,
                          const int32_t* lens, uint32_t page_tokens, const int64_t* parents, const int64_t* children,
                          uint64_t n, void* workspace, uint64_t workspace_bytes, hipStream_t stream);

/* Every page in the rows of the given sequences is released (its count falls
 * by one) and its entry becomes -1.  A count that is 0 already stays 0 and
 * latches IBP_ERR_CORRUPT. */
ibp_status ibp_pages_free(ibp_meta_t meta, int32_t* refs, uint64_t n_slots, int64_t* table, uint64_t n_seqs,
                          uint32_t n_heads, uint64_t table_blocks, const int64_t* seqs, uint64_t n,
                          hipStream_t stream);

/* Moves the live pages (refs > 0) into slots [0, *n_live): the j-th free
 * slot in front of n_live takes the j-th live page counted from the back,
 * with its bit and count; the count it leaves is 0.  map (device int64,
 * n_slots) receives each slot's new id (-1: it was free), n_live (device
 * int64) the number of live pages, and the n_entries ids at table (may be
 * NULL with 0) are rewritten through map. */
ibp_status ibp_pages_compact(ibp_meta_t meta, void* slots, uint64_t n_slots, uint32_t* bitmask, int32_t* refs,
                             int64_t* map, int64_t* n_live, int64_t* table, uint64_t n_entries, void* workspace,
                             uint64_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Attention over the pages, read where they lie: a page of page_tokens x
 * head_dim numbers (bf16 or fp16, row-major) of one key/value head is one
 * slot, raw or a record, which the kernels rebuild on the way to the matrix
 * cores.  head_dim 64, 128 or 256; page_tokens 16, 32 or 64 with pages of at
 * most 8 KiB; anything else returns IBP_ERR_UNSUPPORTED.  Keys and values
 * have a pool each (two handles, or one), a slot id each, in device or
 * pinned memory.  n_q_heads is a multiple of n_kv_heads; query head h reads
 * key/value head h / (n_q_heads / n_kv_heads).  All other data is device
 * memory; strides are in numbers.
 *
 * Scores are scale * q.k in 32 bits, the softmax's maximum and sum are held
 * in 32 bits, its weights are rounded to the data's type for the product
 * with the values, which is summed in 32 bits.  A row that sees no key, or
 * only keys whose score is -infinity, gives zeros and lse -infinity.  What
 * lies in a page behind a sequence's last token, and keys and values that a
 * row does not see, never reach its result, infinities and NaN included.
 *
 * Errors are latched on the keys' handle; those of the values' pages and of
 * the ids in their table on the values' handle as well.
 *
 * A call is one launch of at most 2^24 - 1 workgroups, one or more for each
 * (row, or sequence of drafted tokens; key/value head); larger ones return
 * IBP_ERR_UNSUPPORTED before anything is queued and are given in parts.
 * ------------------------------------------------------------------------- */
typedef enum ibp_dtype { IBP_BF16 = 0, IBP_FP16 = 1 } ibp_dtype;

typedef struct ibp_pages {
    ibp_meta_t meta;         /* L = page_tokens * head_dim * 2 */
    const void* slots;       /* device or pinned, 16-byte aligned */
    uint64_t n_slots;
    const uint32_t* bitmask; /* device */
} ibp_pages;

typedef struct ibp_attention {
    uint32_t dtype;          /* ibp_dtype of q, pages, k_new, v_new and out */
    uint32_t head_dim;
    uint32_t page_tokens;
    uint32_t n_q_heads;
    uint32_t n_kv_heads;
    float scale;
    uint64_t n_rows;         /* rows of q, out and lse; without any a call does nothing */
    uint64_t n_seqs;         /* rows of the block tables: n_seqs x n_kv_heads x table_blocks, */
    uint64_t table_blocks;   /* at least 1 each where there are rows */
    uint64_t max_len;        /* about the longest context: a hint, read to plan the split only */
    uint32_t max_new;        /* most drafted tokens of a sequence (tree attention) */
    int64_t q_row_stride, q_head_stride;
    int64_t new_row_stride, new_head_stride; /* of k_new and v_new */
} ibp_attention;

/* Attention of a tree of drafted tokens.  Sequence s has lens[s] tokens in
 * its pages and new_rows[s + 1] - new_rows[s] drafted ones (device int32,
 * n_seqs + 1, ascending), whose queries, keys and values are those rows of
 * q (n_q_heads x head_dim), k_new and v_new (n_kv_heads x head_dim).  A
 * drafted token sees all of the context and drafted token j of its sequence
 * where bit j % 64 of word j / 64 of its mask row (device uint64, n_rows x
 * mask_words) is set: itself and its ancestors in a tree, any other pattern
 * just as well.  Decoding one token is the tree of one node.
 * out: n_rows x n_q_heads x head_dim; lse (may be NULL): n_rows x n_q_heads
 * floats, the log of the softmax's sum.  Rows behind the last sequence's stay
 * as they were.  A sequence with more than max_new or 64 * mask_words drafted
 * tokens, or more context than its table row holds, latches IBP_ERR_RANGE
 * and its rows are unspecified, as are those of corrupt pages
 * (IBP_ERR_CORRUPT) and of table entries that are no slot (IBP_ERR_RANGE). */
uint64_t ibp_tree_attention_workspace(const ibp_attention* a);
ibp_status ibp_tree_attention(const ibp_pages* k, const ibp_pages* v, const ibp_attention* a, const void* q,
                              const int64_t* k_table, const int64_t* v_table, const int32_t* lens,
                              const int32_t* new_rows, const void* k_new, const void* v_new, const uint64_t* mask,
                              uint32_t mask_words, void* out, float* lse, void* workspace, uint64_t workspace_bytes,
                              hipStream_t stream);

/* Bounds of pages: for i < n, bounds[ids[i]] (2 x head_dim numbers of the
 * data's type) <- the smallest, then the largest, of each number over the
 * first tokens[i] tokens (NULL: all) of page ids[i]; an id of -1 or no token
 * at all is skipped, and a NaN is passed on.  An id may be listed twice with
 * the same tokens only.  With q these bound the score of
 * every key in the page: sum over d of max(q_d lo_d, q_d hi_d). */
ibp_status ibp_page_bounds(const ibp_pages* k, uint32_t dtype, uint32_t head_dim, const int64_t* ids,
                           const int32_t* tokens, uint64_t n, void* bounds, hipStream_t stream);

/* The pages that each query reads: row r of q belongs to sequence row_seq[r]
 * (device int32; NULL: r) and sees its first lens[r] tokens, in nb =
 * ceil(lens[r] / page_tokens) pages.  blocks (device int32, n_rows x n_kv_heads
 * x n_blocks) receives block numbers in ascending order, -1 behind them: the
 * first keep_first and the last keep_last of the nb, then those with the
 * highest score until there are n_blocks.  A block's score is the highest of
 * its bound over the query heads of the group, summed in 64 bits and rounded to
 * 32; equal scores go to the lower block, and a NaN counts as the lowest (an
 * infinite bound is one like any other: only 0 times infinity and sums of both
 * infinities are NaN).  bounds: pool-wide, as ibp_page_bounds leaves them,
 * indexed by the ids of the keys' table.
 *
 * At most 2^17 blocks per row and 2^22 - 1 rows times key/value heads.  Rows
 * four times as many as the sequences, in groups of up to 16 query heads: at
 * most 262,140; others in tables of more than 1,024 blocks: 65,535.  More may
 * return IBP_ERR_UNSUPPORTED, before anything is queued, and are given in
 * parts; so are batches whose scratch, about 4 bytes for each row, head and
 * block, is more than a caller can spare.  Of a, max_len, max_new, scale and
 * the new_ strides are not read. */
uint64_t ibp_select_pages_workspace(const ibp_attention* a);
ibp_status ibp_select_pages(ibp_meta_t meta, const ibp_attention* a, const void* q, const void* bounds,
                            uint64_t n_slots, const int64_t* k_table, const int32_t* lens, const int32_t* row_seq,
                            uint32_t keep_first, uint32_t keep_last, int32_t* blocks, uint32_t n_blocks,
                            void* workspace, uint64_t workspace_bytes, hipStream_t stream);

/* Attention of each row over the blocks listed for it and its key/value head
 * (blocks as ibp_select_pages writes them; -1 is skipped anywhere, a block
 * listed twice counts twice), of which it sees tokens below lens[r]. */
uint64_t ibp_sparse_attention_workspace(const ibp_attention* a, uint32_t n_blocks);
ibp_status ibp_sparse_attention(const ibp_pages* k, const ibp_pages* v, const ibp_attention* a, const void* q,
                                const int64_t* k_table, const int64_t* v_table, const int32_t* lens,
                                const int32_t* row_seq, const int32_t* blocks, uint32_t n_blocks, void* out,
                                float* lse, void* workspace, uint64_t workspace_bytes, hipStream_t stream);

/* Waits for `stream`, returns the first error latched by a kernel of this
 * handle since the last ibp_check (IBP_OK if none) and clears it:
 * IBP_ERR_RANGE, IBP_ERR_CORRUPT, IBP_ERR_NOMEM when a page found no free
 * slot, or IBP_ERR_DEVICE when a tile gave up waiting for its predecessor in
 * the look-back (its tensor's output is then unspecified). */
ibp_status ibp_check(ibp_meta_t meta, hipStream_t stream);

const char* ibp_status_string(ibp_status status);

#ifdef __cplusplus
}
#endif
#endif
