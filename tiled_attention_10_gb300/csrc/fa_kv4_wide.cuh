/* fa_kv4_wide.cuh -- launch of the many-rows kernel (fa_kv4_wide.cu). */
#pragma once
#include "fa_kv4_units.cuh"

namespace fa {
namespace kv4 {
constexpr int kWideRows = 128;     // rows of a tile, and of a partial's slot

// The kernel (one block on each of `sms`) and the merge.  err: the device error
// word of bounded waits, limit_ns their limit.
cudaError_t launch_wide(const AttnParams& p, int D, bool f16, int sms, uint32_t* err,
                        uint64_t limit_ns, cudaStream_t stream);
}  // namespace kv4
}  // namespace fa
