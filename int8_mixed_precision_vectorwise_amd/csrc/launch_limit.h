// Where calls are cut into launches.
#pragma once

#include <cstdint>

// Workgroups of 256 that a launch of the cache's moves and of the microscaled quantization has at most, times two at
// most where queries turn beside: 2^22 (api.hip), for a grid holds fewer than 2^32 lanes.  Larger calls are cut into
// launches.  No part of the interface and not const only so that tests can cut small calls.
extern "C" int64_t i8mp_launch_blocks;
