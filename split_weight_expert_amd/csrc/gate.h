// Checks of a gate's numbers, shared by the calls that take one (not part of the ABI).
#pragma once

#include "../../include/dwdp_layer.h"

namespace dwdp {

// DWDP_OK, or the error that names the function fn; E is the number of experts.
int check_gate(const char* fn, const dwdp_gate* gate, int E);

}  // namespace dwdp
