// Argument checks shared by the C ABI's translation units (host only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "../../include/w4a16.h"
#include "device_common.h"

namespace w4a16 {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxK = int64_t(1) << 20;   // kernels index rows and columns with 32-bit integers
constexpr int64_t kMaxN = int64_t(1) << 28;
constexpr int64_t kMaxKN = int64_t(1) << 37;  // packed codes index in 32-bit 16-byte units
constexpr int64_t kMaxMK = int64_t(1) << 32;  // activations index in 32-bit elements

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Resolved group size, or 0 if (K, N, group_size) is outside the tile layout.
inline w4a16_status check_shape(int64_t K, int64_t N, int64_t group_size, int64_t* G_out) {
    if (K <= 0 || N <= 0 || K % 128 != 0 || N % 8 != 0) return W4A16_ERR_SHAPE;
    if (K > kMaxK || N > kMaxN || K * N > kMaxKN) return W4A16_ERR_SHAPE;
    const int64_t G = group_size == -1 ? K : group_size;
    if (G <= 0 || K % G != 0 || (G % 128 != 0 && G != 32 && G != 64)) return W4A16_ERR_GROUP;
    *G_out = G;
    return W4A16_OK;
}

// K x Np codes (Np = N rounded up to 16 columns) + one 32-bit word per column per
// unit of min(G, 128) rows, the unit count rounded up to 4 (G resolved)
inline size_t packed_size(int64_t K, int64_t N, int64_t G) {
    const size_t uw = (size_t)padded_units(K, G);
    const size_t np = (size_t)padded_cols(N);
    return (size_t)K * np / 2 + (size_t)4 * uw * np;
}

// 0 = unknown, 1 = gfx950, 2 = other; cached per device ordinal.
inline std::atomic<int> g_device_kind[kMaxDevices];

inline w4a16_status check_device() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return W4A16_ERR_DEVICE;
    if (dev < 0 || dev >= kMaxDevices) return W4A16_ERR_DEVICE;
    int kind = g_device_kind[dev].load(std::memory_order_relaxed);
    if (kind == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return W4A16_ERR_DEVICE;
        kind = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_device_kind[dev].store(kind, std::memory_order_relaxed);
    }
    return kind == 1 ? W4A16_OK : W4A16_ERR_DEVICE;
}

}  // namespace w4a16
