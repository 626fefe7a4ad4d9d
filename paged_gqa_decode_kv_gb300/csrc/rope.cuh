// rope.cuh -- parameters of the rotary kernels (rope.cu).
#pragma once

#include "pgd_device.cuh"

namespace pgd {

struct RopeParams {
  const __nv_bfloat16 *q, *k, *v;      // rows; v only where K and V are appended
  __nv_bfloat16 *q_out, *k_out;        // rows (k_out null where K is appended)
  unsigned char *k_cache, *v_cache;    // bf16 pools, or null
  const int64_t *slots;                // [T] block * bs + slot, negative: no token
  const int32_t *positions;            // [T]
  const int64_t *freq;                 // [rotary / 2] turns a position, in units of 2^-64
  // distances in elements between tokens and between heads
  long long q_row, q_head, k_row, k_head, v_row, v_head, qo_row, qo_head, ko_row, ko_head;
  int T, n_q, n_kv, d, first, rotary, interleaved;
  int bs, NB;
  float factor;                        // of cosine and sine
  int32_t *err;
};
// sms: the device's.
cudaError_t rope_launch(const RopeParams &p, int sms, cudaStream_t stream);

}  // namespace pgd
