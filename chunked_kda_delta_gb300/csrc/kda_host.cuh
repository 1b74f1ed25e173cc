// kda_host.cuh -- host-side helpers shared by the translation units of the C ABI: errors,
// the device cache, workspaces and pointer checks.  Defined in kda_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {
namespace host {

void clear_error();
kda_status fail(kda_status st, const char* fmt, ...);
kda_status cuda_fail(cudaError_t e, const char* what);

struct DeviceInfo {
    bool ready = false;
    int cc_major = 0, cc_minor = 0, sm_count = 0;
    int resident_clusters = 0;  // co-resident 2-CTA clusters of the fused kernel
    int32_t* status = nullptr;
};
kda_status device_info(int dev, DeviceInfo** out);
// The current device and its cached properties.
kda_status current_device(int* dev, DeviceInfo** out);

// Scratch of the cache, page and beam calls (kWsServing) is one buffer per (device, stream)
// that those calls share in stream order.  Grown buffers are kept until the release.
enum WorkspaceKind { kWsSegment = 0, kWsHostArena = 1, kWsServing = 2 };
kda_status get_workspace(int dev, cudaStream_t stream, int kind, size_t bytes, void** out);

struct Range {
    const void* p;
    size_t bytes;
};
inline bool overlaps(Range a, Range b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace host
}  // namespace kda
