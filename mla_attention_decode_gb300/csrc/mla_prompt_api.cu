// mla_prompt_api.cu -- entry points of the prompt attention: argument validation,
// tensor maps and launches (include/mla_prompt.h).
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "mla_prompt.h"
#include "mla_prompt_internal.h"

namespace {

constexpr int32_t kMaxRows = 1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 38;  // elements: a tensor map's strides are below 2^40 bytes

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_sizes(const mla_prompt_args* a) {
  if (!a) return MLA_ERR_INVALID_ARG;
  if (a->num_q < 0 || a->num_q >= kMaxRows || a->num_kv < 0 || a->num_kv >= kMaxRows) return MLA_ERR_INVALID_ARG;
  if (a->batch < 0 || a->batch > MLA_MAX_BATCH) return MLA_ERR_INVALID_ARG;
  if (a->heads < 1 || a->heads > MLA_PROMPT_MAX_HEADS) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

constexpr size_t kPartBytes = (MLA_PROMPT_V + 1) * sizeof(float);  // a row's partial result

// How many CTAs share the keys of a tile.  Few rows leave SMs without a CTA, and a
// tile's time is its key tiles one after the other: the keys are dealt to as many CTAs
// as there are SMs, each with at least kSplitTiles key tiles of an average document.
// 16 heads: 17 tokens after 8000 keys 99 -> 21 us, 200 each after 4000 in two documents
// 69 -> 35; one token after 12,000 145 -> 26.  At least 2 tiles instead of 3: 100
// tokens after 700 keys 13.9 us instead of 15.4, but a prompt of 500 tokens 19.9
// instead of 15.0, which has more to join; at least 4: 16.9 and 15.0.
constexpr int64_t kSplitTiles = 3;
int32_t splits_of(const mla_prompt_args* a, int64_t slots, size_t workspace_bytes) {
  // the tiles of documents of equal length (slots counts one more for most of them)
  const int64_t each = (a->num_q + a->batch - 1) / a->batch, full = (each + mla::kPromptQ - 1) / mla::kPromptQ * a->batch;
  const int64_t ctas = (full < slots ? full : slots) * a->heads, sms = mla::kPromptSplitCtas / 2;
  const int64_t tiles = (int64_t)a->num_kv / a->batch / mla::kPromptTile + 1;
  int64_t s = sms / ctas;
  if (s > tiles / kSplitTiles) s = tiles / kSplitTiles;
  if (s > mla::kPromptMaxSplits) s = mla::kPromptMaxSplits;
  const int64_t room = (int64_t)((workspace_bytes - 256) / kPartBytes) / ((int64_t)a->num_q * a->heads);
  if (s > room) s = room;  // (a workspace made for fewer rows)
  return s < 1 ? 1 : static_cast<int32_t>(s);
}

// The 256-token tiles of the batch, at most (mla_prompt.cu says how they are counted).
int64_t slots_of(const mla_prompt_args* a) { return a->num_q / mla::kPromptQ + (int64_t)a->batch; }

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

struct Rows {
  const void* base;
  int32_t columns, tokens;
  int64_t token_stride, head_stride;
};

// (columns, heads, tokens), or (columns, tokens) with heads 0.
bool encode(CUtensorMap* m, const Rows& r, int32_t heads) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  // a dimension of size 1 has no stride that means anything
  const cuuint64_t head = heads > 1 ? (cuuint64_t)r.head_stride * 2 : (cuuint64_t)r.columns * 2;
  const cuuint64_t token = r.tokens > 1 ? (cuuint64_t)r.token_stride * 2 : (cuuint64_t)r.columns * 2;
  const cuuint64_t dims3[3] = {(cuuint64_t)r.columns, (cuuint64_t)heads, (cuuint64_t)r.tokens};
  const cuuint64_t strides3[2] = {head, token};
  const cuuint32_t box3[3] = {64, 1, mla::kPromptTile};
  const cuuint64_t dims2[2] = {(cuuint64_t)r.columns, (cuuint64_t)r.tokens};
  const cuuint64_t strides2[1] = {token};
  const cuuint32_t box2[2] = {64, mla::kPromptTile};
  const cuuint32_t ones[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, heads ? 3 : 2, const_cast<void*>(r.base), heads ? dims3 : dims2,
             heads ? strides3 : strides2, heads ? box3 : box2, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool stride_ok(int64_t s, int64_t n) { return n <= 1 || (s > 0 && s % 8 == 0 && s < kMaxStride); }
bool rows_ok(const Rows& r, int32_t heads) {
  return r.base && aligned(r.base, 16) && stride_ok(r.token_stride, r.tokens) && stride_ok(r.head_stride, heads);
}

}  // namespace

extern "C" {

size_t mla_prompt_workspace_bytes(const mla_prompt_args* args) {
  if (check_sizes(args) != MLA_OK) return 0;
  // partial results of as many rows as any split has, of a call of at most these sizes
  const int64_t rows = (int64_t)args->num_q * args->heads * mla::kPromptMaxSplits;
  const int64_t most = (int64_t)mla::kPromptSplitCtas * mla::kPromptQ;
  return 256 + (size_t)(rows < most ? rows : most) * kPartBytes;
}

int mla_prompt_fwd(const mla_prompt_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_sizes(args);
  if (rc != MLA_OK) return rc;
  const mla_prompt_args& a = *args;
  if (a.causal != 0 && a.causal != 1) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(a.sm_scale) || a.sm_scale <= 0) return MLA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < mla_prompt_workspace_bytes(args)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (a.batch == 0 || a.num_q == 0) return MLA_OK;
  if (!a.qo_indptr || !a.kv_indptr || !aligned(a.qo_indptr, 4) || !aligned(a.kv_indptr, 4) || !aligned(a.prefix, 4))
    return MLA_ERR_INVALID_ARG;
  if (!a.out || !aligned(a.out, 16) || !aligned(a.lse, 4)) return MLA_ERR_INVALID_ARG;
  if (!stride_ok(a.out_token_stride, a.num_q) || !stride_ok(a.out_head_stride, a.heads)) return MLA_ERR_INVALID_ARG;
  Rows rows[5] = {{a.q_nope, MLA_PROMPT_NOPE, a.num_q, a.q_nope_token_stride, a.q_nope_head_stride},
                  {a.q_pe, MLA_PROMPT_PE, a.num_q, a.q_pe_token_stride, a.q_pe_head_stride},
                  {a.k_nope, MLA_PROMPT_NOPE, a.num_kv, a.k_nope_token_stride, a.k_nope_head_stride},
                  {a.k_pe, MLA_PROMPT_PE, a.num_kv, a.k_pe_token_stride, 0},
                  {a.v, MLA_PROMPT_V, a.num_kv, a.v_token_stride, a.v_head_stride}};
  mla::PromptParams p;
  std::memset(&p, 0, sizeof p);
  CUtensorMap* maps[5] = {&p.q_nope, &p.q_pe, &p.k_nope, &p.k_pe, &p.v};
  for (int i = 0; i < 5; ++i) {
    if (i >= 2 && a.num_kv == 0) continue;  // no keys: never read
    const int32_t heads = i == 3 ? 0 : a.heads;
    if (!rows_ok(rows[i], heads)) return MLA_ERR_INVALID_ARG;
    if (!encode(maps[i], rows[i], heads)) return MLA_ERR_CUDA;
  }
  const int64_t slots = slots_of(args);
  if (slots * a.heads > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  p.splits = splits_of(args, slots, workspace_bytes);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
  p.part_lse = p.part_o + (int64_t)p.splits * a.num_q * a.heads * MLA_PROMPT_V;
  p.qo_indptr = a.qo_indptr;
  p.kv_indptr = a.kv_indptr;
  p.prefix = a.prefix;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.out_token_stride = a.num_q > 1 ? a.out_token_stride : 0;
  p.out_head_stride = a.heads > 1 ? a.out_head_stride : 0;
  p.num_q = a.num_q;
  p.num_kv = a.num_kv;
  p.batch = a.batch;
  p.heads = a.heads;
  p.causal = a.causal;
  p.slots = static_cast<int32_t>(slots);
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.ws_err = static_cast<int32_t*>(workspace);
  if (mla::launch_prompt(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

}  // extern "C"
