// The streamed backward kernels for rows of a multiple of 8 channels.
#include "linear_scan_stream.cuh"

namespace kdn {
template bool ls_stream_call<true, true>(const LsCall&, kdn_status*);
}  // namespace kdn
