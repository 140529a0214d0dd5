// The streamed backward kernels for rows of any length.
#include "linear_scan_stream.cuh"

namespace kdn {
template bool ls_stream_call<true, false>(const LsCall&, kdn_status*);
}  // namespace kdn
