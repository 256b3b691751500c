// hg_check.cuh -- range checks of the checked build.
//
// Built with -DHASHGRID_CHECKED (libhashgrid_checked.so), every global-memory access of the
// kernels is tested against the extent of the buffer it belongs to. Before each launch the
// host records, per buffer role, the byte range the call may touch; an access outside its
// role's range sets that role's bit in a device status word and is skipped (a load reads
// zeros), so a wrong index becomes an error code instead of a fault. After the kernel the
// host reads the word back on the call's stream, clears it and returns
// HASHGRID_ERR_DEVICE_CHECK naming the roles. The checked build is synchronous (each call
// waits for its kernel) and slower; it exists to run the parity tests under it. In the
// regular build in_bounds() is the constant true and every check compiles away.
#pragma once

#include <stdint.h>

namespace hg {

enum CheckRole {
    kChkX = 0,      // point coordinates (read)
    kChkTable = 1,  // feature table (read; Adam also writes it)
    kChkOut = 2,    // encoding, dL/dx, MLP output or index export (written)
    kChkDout = 3,   // upstream gradient rows (read)
    kChkGrad = 4,   // table gradient (reduced into; Adam reads and may clear it)
    kChkM = 5,      // Adam first moment
    kChkV = 6,      // Adam second moment
    kChkWeights = 7,   // layer weights (read)
    kChkBias = 8,      // bias (read) or its gradient (written)
    kChkResidual = 9,  // residual rows (read)
    kChkZ = 10,        // pre-activation rows (written, or read by the backward pass)
    kChkWork = 11,     // workspace
    kChkAdamw = 12,    // any array of an AdamW list (held against its own length)
    kChkRoles = 13
};

struct CheckRanges {
    uint64_t lo[kChkRoles];
    uint64_t hi[kChkRoles];  // one past the last byte; lo == hi: the role is not used
};

#ifdef HASHGRID_CHECKED
__device__ CheckRanges g_check_ranges;
__device__ unsigned int g_check_flags;

template <int R>
__device__ __forceinline__ bool in_bounds(const void* p, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)p;
    if (a >= g_check_ranges.lo[R] && a + bytes <= g_check_ranges.hi[R]) return true;
    atomicOr(&g_check_flags, 1u << R);
    return false;
}
__device__ __forceinline__ bool in_bounds_role(int role, const void* p, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)p;
    if (a >= g_check_ranges.lo[role] && a + bytes <= g_check_ranges.hi[role]) return true;
    atomicOr(&g_check_flags, 1u << role);
    return false;
}
#else
__device__ __forceinline__ constexpr bool in_bounds_role(int, const void*, uint32_t) { return true; }
template <int R>
__device__ __forceinline__ constexpr bool in_bounds(const void*, uint32_t) {
    return true;
}
#endif

// Launched with programmatic stream serialization, a kernel may start while the one before it in the
// stream still runs: it sets itself up and touches no global memory before this, which waits until
// everything before it has finished and can be seen. The kernel after it may then do the same.
__device__ __forceinline__ void after_previous_kernel() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace hg
