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

// Scratch of one cache, page or beam call, from the thread's allocator or the library's pool: taken in
// the order of the stream, and given back in it when the object goes, after the call's last launch.
class Scratch {
public:
    Scratch() = default;
    Scratch(const Scratch&) = delete;
    Scratch& operator=(const Scratch&) = delete;
    ~Scratch();
    kda_status take(int dev, void* stream, size_t bytes);
    char* base = nullptr;

private:
    kda_scratch_allocator from_ = {};
    void* stream_ = nullptr;
    size_t bytes_ = 0;
};

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
