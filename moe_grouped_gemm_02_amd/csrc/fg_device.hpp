// fg_device.hpp -- host helpers shared by the entry points: the current
// device's architecture check and pointer alignment.
#pragma once

#include <stdint.h>

namespace fg {

// Checks that the current device is gfx950 (FG_OK, FG_EUNSUPPORTED or
// FG_EDEVICE) and gives its compute units (cus may be null). Defined in
// fg_host.hip.
int current_device(int* cus);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace fg
