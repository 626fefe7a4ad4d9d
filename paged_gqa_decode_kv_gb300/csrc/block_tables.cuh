// block_tables.cuh -- parameters of the kernels that grow and cut block tables
// (block_tables.cu).
#pragma once

#include "pgd_device.cuh"

namespace pgd {

struct GrowParams {
  int32_t *tables;               // [B][MB]
  int32_t *ctx;                  // [B]
  const int32_t *new_tokens;     // [B]
  int32_t *refs;                 // [NB]
  uint32_t *free_bits;           // [(NB + 31) / 32]
  int32_t *positions;            // [B]
  int32_t *starts;               // [B + 1]
  int64_t *slots;                // [N]
  int32_t *token_positions;      // [N]
  int32_t *copy_src, *copy_dst;  // [B]
  int32_t *result;               // [4]
  int B, N, bs, MB, NB;
  // the launch's: log2(bs), or -1; room for the rows' last blocks
  int lg_bs, keep_lasts;
  int32_t *err;
};
constexpr int kMaxGrowRows = 16384;  // three int32 a row in shared memory
cudaError_t grow_tables_launch(const GrowParams &p, cudaStream_t stream);

struct TrimParams {
  int32_t *tables;      // [B][MB]
  int32_t *ctx;         // [B]
  const int32_t *keep;  // [B]
  int32_t *refs;        // [NB]
  uint32_t *free_bits;  // [(NB + 31) / 32]
  int B, bs, MB, NB;
  int lg_bs;            // set by the launch
  int32_t *err;
};
cudaError_t trim_tables_launch(const TrimParams &p, cudaStream_t stream);

}  // namespace pgd
