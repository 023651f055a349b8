// api_checks.cuh -- the argument checks that the layers' C entry points share
// (layer_api.cu, recurrent_api.cu).
#pragma once

#include <stdint.h>

#include "osdn_device.cuh"

namespace osdn {
namespace api {

constexpr size_t kStatusBytes = 256;
constexpr int kMaxTokens = 1073741760;   // chunk starts stay 32-bit TMA coordinates

inline bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline bool io_ok(int io) { return io == OSDN_F32 || io == OSDN_BF16; }
inline size_t io_bytes(int io) { return io == OSDN_BF16 ? 2 : 4; }

inline int check_device() {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return OSDN_ERR_CUDA;
    return major == 10 && minor == 3 ? OSDN_OK : OSDN_ERR_ARCH;
}

// A buffer of a call: its address, its bytes and whether the call writes it.
struct Buf {
    const void *p;
    size_t n;
    bool out;
};
// OSDN_ERR_ALIGN or OSDN_ERR_ALIAS if a buffer is not 16-byte aligned or a
// written one overlaps another, else OSDN_OK.
template <int N>
int check_bufs(const Buf (&b)[N]) {
    for (int i = 0; i < N; ++i)
        if (misaligned(b[i].p)) return OSDN_ERR_ALIGN;
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < i; ++j) {
            if (!(b[i].out || b[j].out) || !b[i].p || !b[j].p || !b[i].n || !b[j].n) continue;
            const uintptr_t x = reinterpret_cast<uintptr_t>(b[i].p), y = reinterpret_cast<uintptr_t>(b[j].p);
            if (x < y + b[j].n && y < x + b[i].n) return OSDN_ERR_ALIAS;
        }
    return OSDN_OK;
}

inline int done(cudaError_t e) { return e == cudaSuccess ? OSDN_OK : OSDN_ERR_CUDA; }

}  // namespace api
}  // namespace osdn
