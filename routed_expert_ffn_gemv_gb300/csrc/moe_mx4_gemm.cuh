// Internals shared by the MXFP4 product and layer translation units.
#pragma once

#include "moe_mx4.cuh"

// Argument checks of the product and layer calls (sizes; pool).
int mx4_ffn_check(int T, int H, int F, int E, int k);
int mx4_pool_check(int H, int F, int n_slots, const void *pool, size_t slot_bytes);

int mx4_simple_gateup_plain(const void *x, int xtype, int T, int H, int F, int E, int k, const int32_t *ids,
                            const int32_t *table, int n_slots, const void *pool, size_t slot_bytes, float *h,
                            cudaStream_t s);
int mx4_simple_down_plain(const float *h, int T, int H, int F, int E, int k, const int32_t *ids, const float *weights,
                          const int32_t *table, int n_slots, const void *pool, size_t slot_bytes, float *partial,
                          cudaStream_t s);
