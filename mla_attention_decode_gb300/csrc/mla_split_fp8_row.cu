// mla_split_fp8_row.cu -- e4m3 KV with a scale per row: the tcgen05 split kernel
// over a contiguous cache or pages of 64 rows and more, over smaller pages, and
// with two query tokens per work unit.
#include "mla_tc.cuh"

namespace mla {
cudaError_t launch_stage1_fp8_row(const Stage1Params& p, cudaStream_t s) {
  if (p.tok == 2) return launch_split_tc<false, 2, tcfp8::kPathRowScales>(p, s);
  if (p.paged && p.page_shift < 6) return launch_split_tc<false, 1, tcfp8::kPathRowScalesSmall>(p, s);
  return launch_split_tc<false, 1, tcfp8::kPathRowScales>(p, s);
}
}  // namespace mla
