/*
 * mla_cache.h -- C ABI of libmla_decode.so: the operators around the latent
 * cache that mla_decode.h decodes over.  They write it (norms, position
 * rotation and storage format in one pass), read it back as bf16, and manage
 * its pages (growing, truncating, forking, freeing, copying, compacting).
 *
 * Conventions are those of mla_decode.h: every entry point returns an
 * mla_status, allocates nothing, never synchronises, and enqueues on `stream`
 * (a cudaStream_t; NULL = the legacy default stream) of the current device.
 * "device" pointers are device memory.  Host-checked arguments come back as
 * MLA_ERR_INVALID_ARG / MLA_ERR_UNSUPPORTED / MLA_ERR_WORKSPACE_TOO_SMALL with
 * nothing launched.  What only the device can see (a row, page or table entry
 * out of range, too few free pages) sets an error word instead -- the first
 * word of the workspace, or *device_error -- which stays set until
 * mla_decode_poll_error(word, stream) reads and clears it; the bad entry is
 * skipped, never followed.  device_error may be NULL (nothing is recorded).
 *
 * A row is 576 columns: 512 latent ones (the values of the decode are these),
 * then 64 position ones ("pe" below).  A row's number in the cache ("slot") is
 * page * page_size + its place in the page.
 */
#ifndef MLA_CACHE_H
#define MLA_CACHE_H

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_PE_DIM 64
#define MLA_PE_PAIRS 32
#define MLA_MAX_AXES 8

/*
 * A paged cache: num_layers times num_pages pages of page_size rows in the
 * storage format of kv_dtype (mla_decode.h), one page table for all layers.
 * A contiguous cache of R rows is num_pages = R pages of one row.
 */
typedef struct {
  void* kv;                  /* device, 16-byte aligned; rows of 1152 / 576 / 288 / (fp8_row) 576 bytes */
  void* kv_scale;            /* bf16: NULL; fp8: fp32 (per layer, or one for all); mxfp4: uint8
                                e8m0 [rows, scale_stride] per layer, 16-byte aligned; fp8_row: fp32
                                [rows] per layer, scale_stride bytes apart, 16-byte aligned */
  int64_t kv_layer_bytes;    /* bytes from a layer's rows to the next layer's: a multiple of 16, at
                                least the rows of one layer (ignored with one layer) */
  int64_t scale_layer_bytes; /* the same for kv_scale: fp8 a multiple of 4 (0: one scale for all
                                layers); mxfp4 at least one layer's scales; fp8_row the same and a
                                multiple of 4 */
  int32_t kv_dtype;          /* mla_kv_dtype */
  int32_t page_size;         /* rows per page: a power of two */
  int32_t num_pages;         /* num_pages * page_size must fit in int32 */
  int32_t num_layers;        /* >= 1 */
  int32_t scale_stride;      /* mxfp4: bytes between scale rows, >= 18; fp8_row: between the rows' scales,
                                a multiple of 4, >= 4; otherwise 0 */
  int32_t reserved;          /* 0 */
  int32_t scale_width;       /* mxfp4: bytes of each scale row that are this cache's, 18..scale_stride (0: all
                                of them); the others are neither read nor written; fp8_row: 4 (0: all of
                                them move with a row); otherwise 0 */
  int32_t reserved2;         /* 0 */
} mla_cache;

/*
 * The rotation of the 64 position columns: pair i (of 32) of a token whose
 * position on axis a is pos[a] turns by the angle pos[axis[i]] * inv_freq[i],
 *   (a, b) -> scale * (a cos - b sin, a sin + b cos).
 * Filled by mla_rope_plan; must not be edited.
 */
typedef struct {
  uint64_t turn[MLA_PE_PAIRS]; /* inv_freq / 2 pi mod 1, in units of 2^-64 turns */
  uint8_t axis[MLA_PE_PAIRS];  /* the axis whose position turns the pair */
  int32_t num_axes;
  int32_t interleaved;         /* 1: pair i = columns (2i, 2i + 1); 0: columns (i, i + 32) */
  float scale;
  int32_t reserved;
} mla_rope;

/*
 * mla_rope_plan -- host only.  inv_freq[32]: angle per position step of each
 * pair, finite.  axis_of_pair[32] (NULL: all 0): each in [0, num_axes).
 * num_axes: 1..MLA_MAX_AXES (time, height, width, ...).  scale: a factor on
 * the rotated columns (1 for none), finite.
 */
MLA_API int mla_rope_plan(const double* inv_freq, const int32_t* axis_of_pair, int32_t num_axes,
                          int32_t interleaved, double scale, mla_rope* rope);

/* The parts of a token's key row and query heads that a norm applies to. */
enum { MLA_PART_KV_LAT = 0, MLA_PART_KV_PE = 1, MLA_PART_Q_LAT = 2, MLA_PART_Q_PE = 3 };

/*
 * Root-mean-square norms, y = x / sqrt(mean(x^2) + eps) * weight, of the parts
 * in `apply`; queries are normed head by head.  The squares are summed in fp32
 * (columns above about 1e18 overflow the sum).
 */
typedef struct {
  const void* weight[4]; /* device, per part: bf16 or fp32 [512] / [64], 16-byte aligned; NULL: 1 */
  int32_t apply;         /* bit 1 << part: the part is normed */
  int32_t weight_fp32;   /* 1: the weights are fp32; 0: bf16 */
  float eps;             /* finite, >= 0 */
  int32_t reserved;
} mla_norm;

/* One call's tokens.  Strides are in elements. */
typedef struct {
  const void* kv_lat;        /* device bf16 [num_tokens, 512], 16-byte aligned rows; NULL: no key rows */
  const void* kv_pe;         /* device bf16 [num_tokens, 64], 4-byte aligned rows */
  const int32_t* slots;      /* device [num_tokens]: the row each key is stored in; -1: not stored */
  const int32_t* positions;  /* device [num_tokens, num_axes] */
  const void* q_lat;         /* device bf16 [num_tokens, 16, 512], 16-byte aligned rows; NULL: the latent
                                columns of q_out are left as they are */
  const void* q_pe;          /* device bf16 [num_tokens, 16, 64], 4-byte aligned rows; NULL: no queries */
  void* q_out;               /* device bf16 [num_tokens, 16, 576], contiguous, 16-byte aligned */
  int64_t kv_lat_stride;     /* between tokens */
  int64_t kv_pe_stride;
  int64_t position_stride;   /* between tokens; a token's axes are consecutive */
  int64_t q_lat_token_stride, q_lat_head_stride;
  int64_t q_pe_token_stride, q_pe_head_stride;
  int32_t num_tokens;
  int32_t layer;             /* the cache layer the keys go to */
} mla_append_args;

/*
 * mla_cache_append -- norms, rotates and stores the tokens' key rows, and norms
 * and rotates their query heads into the layout the decode reads.
 *
 * Everything is computed in fp32 and rounded once: queries and bf16 rows to
 * bf16; fp8 rows to e4m3(y / kv_scale) (the quotient rounded to fp32 first),
 * saturating at 448 (NaN stays NaN, a zero keeps its sign); mxfp4 rows to e2m1
 * under the smallest power of two 2^e with max|y| <= 6 * 2^e per block of 32
 * (scale byte e + 127; 127 for a block of zeros; a block with an infinity or a
 * NaN gets scale byte 255 = NaN and codes 0); fp8_row rows to e4m3(y / s) (the
 * quotient rounded to fp32 first) with s = max(fp32(max|y| / 448), 2^-64) stored
 * as the row's scale, a zero keeping its sign (a row with an infinity or a NaN
 * gets scale NaN and codes 0).
 *
 * Angles are taken modulo one turn by an integer product: at any int32 position
 * off by at most 2^-23 radians (their conversion to fp32) and 2^-52 of
 * |position * inv_freq| (the plan's fp64 quotient, 2^-21 at the far end for a
 * frequency of 1).
 *
 * rope NULL: no rotation (positions is not read).  norm NULL: no norms.
 * q_lat / q_pe may be the very columns of q_out they go to (in place); no
 * other overlap of inputs and outputs.  The slots of one call are distinct
 * (-1 aside): two tokens with the same slot leave that row undefined.  A slot
 * outside [-1, rows) is skipped and sets MLA_ERR_DEVICE_INDEX.  The bytes of
 * a scale row past its first 18 are left as they are.
 */
MLA_API int mla_cache_append(const mla_cache* cache, const mla_rope* rope, const mla_norm* norm,
                             const mla_append_args* args, int32_t* device_error, void* stream);

/*
 * mla_cache_gather -- rows of one layer as bf16: out[t, :] = bf16(the value of
 * row slots[t]; fp8 and fp8_row: the code times the scale in fp32).  out: device bf16 [num_rows, 576], rows out_stride elements
 * apart (a multiple of 8, >= 576), 16-byte aligned.  Rows of out with slot -1
 * are left as they were; so are those with a slot outside the cache, which
 * set MLA_ERR_DEVICE_INDEX.  Slots may repeat.
 */
MLA_API int mla_cache_gather(const mla_cache* cache, int32_t layer, const int32_t* slots, int32_t num_rows,
                             void* out, int64_t out_stride, int32_t* device_error, void* stream);

/*
 * The page table of a batch, as mla_decode_fwd_paged reads it: sequence b owns
 * the pages kv_indices[page_indptr[b] .. page_indptr[b + 1]), of which the last
 * holds last_page_len[b] (1..page_size) rows; a sequence with no pages is empty
 * (its last_page_len is not read, and written as 0).
 */
typedef struct {
  int32_t* page_indptr;   /* device [batch + 1] */
  int32_t* kv_indices;    /* device [num_indices] */
  int32_t* last_page_len; /* device [batch] */
  int32_t batch;          /* 0..MLA_MAX_BATCH */
  int32_t num_indices;    /* room in kv_indices */
} mla_page_table;

/*
 * mla_cache_slots -- the rows of each sequence's newest tokens: with
 * n_b = qo_indptr[b + 1] - qo_indptr[b] and L_b the sequence's length, token
 * qo_indptr[b] + i is row L_b - n_b + i of sequence b (the tokens' own entries
 * of mla_decode_plan_multi; n_b = L_b: the whole sequence).
 *   slots[t]             its row in the cache
 *   rows[t * row_stride] its place in the sequence (a position for the rotation)
 * (rows may be NULL).  qo_indptr[0] must be 0.  Tokens from qo_indptr[batch] on
 * (a padded batch) get slot -1 and row 0.  A token before its sequence's first
 * row gets slot -1 (and that negative row), and so does one whose table entry is
 * out of range; both set MLA_ERR_DEVICE_INDEX.
 */
MLA_API int mla_cache_slots(const mla_cache* cache, const mla_page_table* table, const int32_t* qo_indptr,
                            int32_t num_tokens, int32_t* slots, int32_t* rows, int64_t row_stride,
                            int32_t* device_error, void* stream);

/*
 * mla_cache_copy_pages -- page dst[i] = page src[i] in every layer (rows and
 * scale rows), i < n.  A page may be the source of several copies; the dst are
 * distinct and none is another copy's src (dst[i] == src[i] is no copy).
 * Pages outside [0, num_pages) are skipped and set MLA_ERR_DEVICE_INDEX.
 */
MLA_API int mla_cache_copy_pages(const mla_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                                 int32_t* device_error, void* stream);

/*
 * Page ownership.  page_refs: device int32 [num_pages], 16-byte aligned, how many
 * sequences hold a page; 0 = free.  Fresh pages are always the free pages of lowest number, in
 * order of sequence and place, so every result is the same from run to run.
 * Part-filled pages belong to one sequence: fork and resize copy a shared one
 * before it can be written.
 *
 * Both take a table `from` and write a table `to` (other buffers).  If the
 * call cannot be met (fewer free pages than it needs: MLA_ERR_OUT_OF_PAGES;
 * `to` has too little room, page_indptr or last_page_len of `from`
 * inconsistent, a bad parent or length: MLA_ERR_DEVICE_INDEX), the error word
 * is set, `to` is left with every sequence empty, and neither the counts nor
 * the cache change.  A page number within `from` that is out of range, or a
 * page that is free as the call begins (its count 0: nobody holds it, and it
 * may be handed out), becomes -1 in `to`, sets MLA_ERR_DEVICE_INDEX and is
 * neither counted nor given back.
 *
 * The workspace is mla_cache_workspace_bytes(cache, batch of `to`) bytes,
 * 256-byte aligned, zeroed before its first use; calls that share it must be
 * ordered on the GPU.
 *
 * mla_cache_fork -- sequence n of `to` is a copy of sequence parents[n] of
 * `from` (repeats allowed): it holds the parent's full pages too (their counts
 * rise by 1) and a fresh copy of the rows of a part-filled last page.  The
 * sequences of `from` live on.
 */
MLA_API int mla_cache_fork(const mla_cache* cache, int32_t* page_refs, const mla_page_table* from,
                           const int32_t* parents, const mla_page_table* to, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * mla_cache_resize -- sequence b gets lengths[b] >= 0 rows (device [batch]);
 * `to` replaces `from` (the same batch).  Rows up to the smaller length are
 * kept; a longer sequence gets fresh pages, whose rows are to be written by
 * the caller; a shorter one gives its last pages back (counts fall by 1).  If a
 * sequence's length changes and the first row that changes lies inside a kept
 * page that others hold too, the sequence gets its own copy of that page's rows
 * before it.
 */
MLA_API int mla_cache_resize(const mla_cache* cache, int32_t* page_refs, const mla_page_table* from,
                             const int32_t* lengths, const mla_page_table* to, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * mla_cache_free -- page_refs[pages[i]] -= 1, i < n: a sequence's hold on its
 * pages ends (pages: e.g. the entries of a table that are in use; a page may
 * occur several times; where only the device knows how many are in use, resize
 * to lengths of 0 ends them).  -1 entries are skipped.  A page out of range, or one given back more
 * often than it is held (its count stays 0), sets MLA_ERR_DEVICE_INDEX.
 */
MLA_API int mla_cache_free(const mla_cache* cache, int32_t* page_refs, const int32_t* pages, int32_t n,
                           int32_t* device_error, void* stream);

/*
 * mla_cache_compact -- moves the L pages in use (page_refs > 0) to the pages
 * [0, L): the k-th page in use at or above L goes to the k-th free page below
 * L, both in rising order; pages below L stay.  Writes
 *   kv_indices_out[i] = the new number of page kv_indices[i], i < num_indices
 *     (-1 stays -1; a page that is free or out of range becomes -1 and sets
 *     MLA_ERR_DEVICE_INDEX),
 *   page_refs_out  the counts by new number (0 from L on),
 *   *live          L (device; may be NULL).
 * page_refs_out may be page_refs, and kv_indices_out may be kv_indices; no
 * other overlap.  The pages moved from keep their rows.  Workspace as above,
 * mla_cache_workspace_bytes(cache, 0).
 */
MLA_API int mla_cache_compact(const mla_cache* cache, const int32_t* page_refs, int32_t* page_refs_out,
                              const int32_t* kv_indices, int32_t* kv_indices_out, int32_t num_indices,
                              int32_t* live, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace for fork / resize of `batch` sequences and for
 * compact on this cache (0 on a null or invalid cache or batch). */
MLA_API size_t mla_cache_workspace_bytes(const mla_cache* cache, int32_t batch);

#ifdef __cplusplus
}
#endif

#endif /* MLA_CACHE_H */
