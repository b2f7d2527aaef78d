// Internals shared by the MXFP4 product and layer translation units.
#pragma once

#include "moe_mx4.cuh"

// Argument checks of the product and layer calls (sizes; pool).
int mx4_ffn_check(int T, int H, int F, int E, int k);
int mx4_pool_check(int H, int F, int n_slots, const void *pool, size_t slot_bytes);
