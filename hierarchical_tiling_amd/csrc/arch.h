// arch.h -- the device check of calls that are made every step.  Apart from gemm_internal.h, whose
// text is part of the digest that ties stored counters to the kernels they were taken on.
#pragma once

namespace htk {

// Whether the current device is a gfx950, as a status code; remembered for each device.
int arch_status();

}  // namespace htk
