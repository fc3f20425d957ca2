// router_rows.h -- the grouped router's form for many rows, four a warp.
#pragma once

#include "router_choice.cuh"

namespace et {

// Whether it serves E experts in G groups.
inline bool rows4_serves(int E, int G) { return E % 32 == 0 && !(G & (G - 1)); }

cudaError_t launch_router_rows4(const GroupArgs& a, bool sigmoid, int rows, int dev, void* stream);

}  // namespace et
