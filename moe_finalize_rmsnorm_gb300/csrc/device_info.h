// Per-device facts the C entry points share: filled on a device's first call.
#pragma once

#include <stdint.h>

#include "moe_finalize.h"

namespace mf {

struct DeviceInfo {
    bool ready = false;
    int num_sms = 0;
    int smem_optin = 0;
    int smem_per_sm = 0;
    int bulk_per_sm = 0;       // resident CTAs per SM of the staged hidden-4096 kernel
    int token_cta_per_sm = 0;  // and of the register kernel
    unsigned *status = nullptr;  // device address of the status word
};

// The current device's facts, set up on first use (MF_ERR_CUDA on failure).
mf_status device_info(const DeviceInfo **out);

// Whether launches carry the programmatic stream serialisation attribute.
bool programmatic_launch();

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s bound on every device wait

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

}  // namespace mf
