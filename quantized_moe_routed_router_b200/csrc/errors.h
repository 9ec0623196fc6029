// The calling thread's last failure outside a handle (ts_moe_last_error(NULL)).
#pragma once
#include "../../include/ts_moe.h"

namespace tsm {
// Keeps `msg` (cut where memory for it runs out) and returns `st`.
ts_moe_status set_last_error(ts_moe_status st, const char* msg) noexcept;
}  // namespace tsm
