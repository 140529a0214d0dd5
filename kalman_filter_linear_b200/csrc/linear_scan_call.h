// A checked call of the gated linear recurrence, forward or backward, and its
// streaming form (linear_scan_stream.cuh).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kdn.h"

namespace kdn {

struct LsCall {
  const void *a, *b, *x;      // b or null; x is not read by a backward without b
  const void *y, *dy;         // backward
  kdn_dtype gate_dtype, in_dtype;
  const float* h0;            // or null
  const float* end_in;        // backward: dh_T or null
  void* y_out;                // forward
  void *da, *db, *dx;         // backward
  float* end_out;             // h_T, or dh0
  const int32_t* cu;          // packed: N + 1 offsets; then B is 1
  int N, B, T, D;
  void* workspace;
  cudaStream_t stream;
  int64_t skip;               // streaming form, for tests: the first block's copy that is left out, or -1
};

// Runs a call in its streaming form, EIGHT for a D that is a multiple of 8; or
// returns false for a call that is better not run so.
template <bool BWD, bool EIGHT>
bool ls_stream_call(const LsCall& k, kdn_status* st);
extern template bool ls_stream_call<false, false>(const LsCall&, kdn_status*);
extern template bool ls_stream_call<false, true>(const LsCall&, kdn_status*);
extern template bool ls_stream_call<true, false>(const LsCall&, kdn_status*);
extern template bool ls_stream_call<true, true>(const LsCall&, kdn_status*);

}  // namespace kdn
