// The sliced router product (router.hip), shared with the gate (not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dwdp {

// Tile shape and K slices for a batch.
struct RouterPlan {
    int bm, bn, slices;
};
RouterPlan plan_router(int64_t T, int H, int E, int dtype);

// Whether one launch holds the plan's tiles.
bool router_fits(int64_t T, int E, const RouterPlan& p);

// logits (one slice) or part[slice][T][E] (more) = x w^T; arguments are checked, T >= 1,
// and the plan fits.
int router_split(const void* x, const void* w, int dtype, const float* bias, int64_t T, int H, int E, const RouterPlan& p,
                 float* logits, float* part, hipStream_t st);

}  // namespace dwdp
