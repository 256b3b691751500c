// hashgrid.cu -- C ABI of libhashgrid.so (declared in include/hashgrid.h): handle, host-side
// validation and kernel launches for the multiresolution hash-grid encoding on sm_100a.
//
// Every argument is checked on the host before anything is launched: ranges, NULLs,
// 16-byte alignment, that each pointer is device-accessible memory of the current device,
// and (for cudaMalloc'd memory) that the whole extent the call will touch lies inside the
// pointer's allocation. A call either launches its kernels or returns an error having
// written nothing.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <new>
#include <string>
#include <type_traits>
#include <vector>

#include "hashgrid.h"
#include "hg_adamw.cuh"
#include "hg_device.cuh"
#include "hg_linear.cuh"
#include "hg_mlp.cuh"
#include "hg_nd.cuh"
#include "hg_probe.cuh"
#include "hashgrid_probe.h"

#ifdef HASHGRID_CHECKED
#define HASHGRID_VERSION_STRING "hashgrid-b200 0.2 (sm_100a, checked)"
#else
#define HASHGRID_VERSION_STRING "hashgrid-b200 0.2 (sm_100a)"
#endif

struct hashgrid_s {
    int D;  // input dimensions (3 for hashgrid_create)
    int L, F, log2T, N_min, N_max, dtype;
    int res[HASHGRID_MAX_LEVELS];
    int forward_gather;   // HASHGRID_GATHER_*
    int backward_mode;    // HASHGRID_BACKWARD_*
    int schedule;         // HASHGRID_SCHEDULE_*
    hg::LevelParams lp;
};

struct hashgrid_linear_s {
    int in, out, dtype, act;
};

struct hashgrid_adamw_s {
    int device;
    std::vector<hg::adamw::Tensor> tensors;
    std::vector<uint32_t> first;  // the tensors' first blocks within their launches
    struct Launch {
        int begin, count;  // tensors
        uint32_t blocks;   // of 256 elements
        hg::adamw::Buckets where;
    };
    std::vector<Launch> launches;
};

namespace {

thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return code;
}

int ok() { return HASHGRID_OK; }

// Resolution schedule, [NeRFace-HG] section 2: b = exp((ln N_max - ln N_min)/(L - 1)),
// N_l = floor(N_min * b^l) of the exact-math value. In double, N_min * b^l can fall a few
// ulp short of an integer it equals exactly (16 * b^15 = 4095.99999... for N_max = 4096);
// a value within 1e-9 (relative) of an integer is taken as that integer, any other value
// is floored.
bool compute_resolutions(int L, int N_min, int N_max, int* res) {
    if (L == 1) {
        if (N_min != N_max) return false;
        res[0] = N_min;
        return true;
    }
    const double b = std::exp((std::log((double)N_max) - std::log((double)N_min)) / (double)(L - 1));
    for (int l = 0; l < L; ++l) {
        const double v = (double)N_min * std::pow(b, (double)l);
        const double r = std::nearbyint(v);
        res[l] = (int)((std::fabs(v - r) <= 1e-9 * v) ? r : std::floor(v));
    }
    return true;
}

// cuMemGetAddressRange through the runtime's driver entry-point query, so the library
// needs no link-time dependency on libcuda.
typedef CUresult (*PFN_memGetAddressRange)(CUdeviceptr*, size_t*, CUdeviceptr);

PFN_memGetAddressRange address_range_fn() {
    static PFN_memGetAddressRange fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuMemGetAddressRange", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<PFN_memGetAddressRange>(p);
    }();
    return fn;
}

// Checks one buffer argument that the call will access over [p, p + bytes): not NULL,
// 16-byte aligned, device memory of the current device or managed memory, and (where the
// driver reports the allocation's range) the whole extent inside the allocation.
int check_buffer(const void* p, size_t bytes, const char* name, size_t align = 16) {
    if (p == nullptr) return fail(HASHGRID_ERR_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align != 0)
        return fail(HASHGRID_ERR_ALIGN, "%s (%p) is not %zu-byte aligned", name, p, align);
    cudaPointerAttributes a;
    cudaError_t e = cudaPointerGetAttributes(&a, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(HASHGRID_ERR_ARG, "%s (%p): cudaPointerGetAttributes failed: %s", name, p,
                    cudaGetErrorString(e));
    }
    if (a.type == cudaMemoryTypeUnregistered || a.devicePointer == nullptr)
        return fail(HASHGRID_ERR_ARG, "%s (%p) is not device-accessible memory", name, p);
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return fail(HASHGRID_ERR_CUDA, "cudaGetDevice failed");
    }
    // Host memory (pinned or registered) is device-accessible but its extent cannot be
    // checked here, and the kernels would read it across the host link: not accepted.
    if (a.type == cudaMemoryTypeHost)
        return fail(HASHGRID_ERR_ARG, "%s (%p) is host memory; the library takes device memory", name, p);
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)
        return fail(HASHGRID_ERR_ARG, "%s (%p) has unknown memory type %d", name, p, (int)a.type);
    if (a.type == cudaMemoryTypeDevice && a.device != dev)
        return fail(HASHGRID_ERR_ARG, "%s lives on device %d but device %d is current", name, a.device, dev);
    // The extent the call touches must lie inside the pointer's allocation. Device memory
    // whose range the driver cannot report (none is known) is accepted as before; managed
    // memory is accepted only when its range is known.
    PFN_memGetAddressRange range = address_range_fn();
    CUdeviceptr base = 0;
    size_t size = 0;
    const bool known = range != nullptr && range(&base, &size, (CUdeviceptr)(uintptr_t)p) == CUDA_SUCCESS;
    if (known) {
        const uintptr_t end = (uintptr_t)base + size;
        if ((uintptr_t)p + bytes > end || (uintptr_t)p + bytes < (uintptr_t)p)
            return fail(HASHGRID_ERR_ARG,
                        "%s: the call touches %zu bytes from %p but its allocation ends %zu bytes after it", name,
                        bytes, p, (size_t)(end - (uintptr_t)p));
    } else if (a.type == cudaMemoryTypeManaged) {
        return fail(HASHGRID_ERR_ARG, "%s (%p): the extent of this managed allocation cannot be checked", name, p);
    }
    return ok();
}

int check_handle(const hashgrid_s* h) {
    if (h == nullptr) return fail(HASHGRID_ERR_ARG, "handle is NULL");
    return ok();
}

int check_N(int64_t N, int BP) {
    if (N < 0) return fail(HASHGRID_ERR_ARG, "N = %lld is negative", (long long)N);
    if ((N + BP - 1) / BP > 0x7fffffffLL)
        return fail(HASHGRID_ERR_ARG, "N = %lld exceeds the largest launchable batch", (long long)N);
    return ok();
}

int launch_status(const char* what) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(HASHGRID_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
    return ok();
}

constexpr int kTile = 64;      // points per block tile
constexpr int kMaxThreads = 512;

int tile_threads(int L) {
    const int items = (kTile / 32) * L;
    return items * 32 < kMaxThreads ? items * 32 : kMaxThreads;
}

template <typename K>
int prepare_smem(K kernel, size_t smem) {
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return fail(HASHGRID_ERR_CUDA, "cudaFuncSetAttribute(smem=%zu) failed: %s", smem,
                        cudaGetErrorString(e));
        }
    }
    return ok();
}

template <int F, typename TT>
int launch_forward(const hashgrid_s* h, const float* x, int64_t N, const void* table, float* out,
                   int gather, cudaStream_t s) {
    const size_t smem = hg::tile_smem_bytes(kTile, h->L, F);
    const unsigned blocks = (unsigned)((N + kTile - 1) / kTile);
    if (gather == hg::kGatherLanes) {
        auto k = hg::forward_kernel_lanes<F, TT, kTile>;
        if (int rc = prepare_smem(k, smem)) return rc;
        // a warp item is 16 points at one level: (kTile / 16) * L items per tile
        const int items = (kTile / 16) * h->L;
        const int threads = items * 32 < kMaxThreads ? items * 32 : kMaxThreads;
        k<<<blocks, threads, smem, s>>>(h->lp, x, N, static_cast<const TT*>(table), out);
        return launch_status("forward");
    }
    auto k = gather == hg::kGatherSector ? hg::forward_kernel<F, TT, kTile, hg::kGatherSector>
           : gather == hg::kGatherPair   ? hg::forward_kernel<F, TT, kTile, hg::kGatherPair>
                                         : hg::forward_kernel<F, TT, kTile, hg::kGatherCorner>;
    if (int rc = prepare_smem(k, smem)) return rc;
    k<<<blocks, tile_threads(h->L), smem, s>>>(h->lp, x, N, static_cast<const TT*>(table), out);
    return launch_status("forward");
}

template <int F, int kMode, typename GT = float>
int launch_backward_mode(const hashgrid_s* h, const float* x, const float* dout, int64_t N,
                         GT* dtable, cudaStream_t s) {
    const int cap = hg::backward_threads(kMode);
    const int threads = tile_threads(h->L) < cap ? tile_threads(h->L) : cap;
    const size_t smem = hg::tile_smem_bytes(kTile, h->L, F) +
                        (kMode == hg::kAtomicOnly ? 0 : hg::group_smem_bytes(threads / 32, F));
    const unsigned blocks = (unsigned)((N + kTile - 1) / kTile);
    if constexpr (kMode == hg::kAtomicOnly) {
        auto k = hg::backward_kernel_atomic<F, kTile, GT>;
        if (int rc = prepare_smem(k, smem)) return rc;
        k<<<blocks, threads, smem, s>>>(h->lp, x, dout, N, dtable);
    } else {
        auto k = hg::backward_kernel_grouped<F, kTile, kMode>;
        if (int rc = prepare_smem(k, smem)) return rc;
        k<<<blocks, threads, smem, s>>>(h->lp, x, dout, N, dtable);
    }
    return launch_status("backward");
}

// The forward kernel a handle's gather option selects (AUTO: lane pairs, measured fastest
// on every workload: per 2^20 ray samples 225 against 250 us per-corner, per 2^18 uniform
// points 81 against 95 us, fp16 table 1.02 against 1.23 ms per 2^22 points).
int forward_gather_kernel(const hashgrid_s* h) {
    switch (h->forward_gather) {
        case HASHGRID_GATHER_CORNER: return hg::kGatherCorner;
        case HASHGRID_GATHER_SECTOR: return hg::kGatherSector;
        case HASHGRID_GATHER_PAIR: return hg::kGatherPair;
        default: return hg::kGatherLanes;
    }
}

// The run walk a handle's backward option selects for F <= 4: lane pairs for AUTO and
// RUN_LANES (measured 356 against 424 us per 2^20 ray samples, 1.74 against 2.10 ms per
// 2^22 uniform points), one lane per run for RUN_MERGE.
bool run_lanes(const hashgrid_s* h) {
    return h->backward_mode == HASHGRID_BACKWARD_RUN_LANES || h->backward_mode == HASHGRID_BACKWARD_AUTO;
}

// Level-major when asked, or (AUTO) when the whole table is larger than most of L2.
constexpr size_t kLevelMajorTableBytes = 96u << 20;

// Level groups of the level-major lane-pair kernels. A level's points in the unit cube reach
// at most min(T, (N_l + 2)^3) entries, so the coarse levels of a large table touch only a
// few MB of their slices. Consecutive levels are grouped while the entries they can reach
// (counted at 4F bytes, the fp32 gradient's width) stay within 32 MB, a quarter of the L2;
// a level above that is a group of its own. One pass per group then reads x and writes the
// output rows once for all its levels. (1 GiB grid, L = 16, F = 4: levels 0-5 reach 26.5 MB
// together and form one group, levels 6-15 one group each.)
constexpr double kLevelGroupBytes = 32.0 * (1 << 20);

void compute_level_groups(hashgrid_s* h) {
    const double T = (double)((uint64_t)1 << h->log2T);
    int g = 0;
    double acc = 0.0;
    h->lp.group_lo[0] = 0;
    for (int l = 0; l < h->L; ++l) {
        const double v = (double)h->res[l] + 2.0;
        const double bytes = std::min(T, v * v * v) * h->F * 4.0;
        if (l > 0 && acc + bytes > kLevelGroupBytes) {
            h->lp.group_lo[++g] = l;
            acc = 0.0;
        }
        acc += bytes;
    }
    h->lp.group_lo[++g] = h->L;
    h->lp.ngroups = g;
}

bool level_major(const hashgrid_s* h) {
    if (h->schedule == HASHGRID_SCHEDULE_LEVEL_MAJOR) return true;
    if (h->schedule == HASHGRID_SCHEDULE_POINT_MAJOR) return false;
    const size_t bytes = (size_t)h->L * ((size_t)1 << h->log2T) * h->F * (h->dtype == HASHGRID_F16 ? 2 : 4);
    return bytes > kLevelMajorTableBytes;
}

template <int F, typename TT>
int launch_forward_levels(const hashgrid_s* h, const float* x, int64_t N, const void* table, float* out,
                          int gather, cudaStream_t s) {
    if (gather == hg::kGatherLanes) {  // two threads per point
        const dim3 grid((unsigned)((2 * N + hg::kLevelBlock - 1) / hg::kLevelBlock), (unsigned)h->lp.ngroups);
        hg::forward_kernel_levels_lanes<F, TT><<<grid, hg::kLevelBlock, 0, s>>>(h->lp, x, N, static_cast<const TT*>(table), out);
        return launch_status("forward");
    }
    const dim3 grid((unsigned)((N + hg::kLevelBlock - 1) / hg::kLevelBlock), (unsigned)h->L);
    hg::forward_kernel_levels<F, TT><<<grid, hg::kLevelBlock, 0, s>>>(h->lp, x, N, static_cast<const TT*>(table), out);
    return launch_status("forward");
}

// Run merging for every mode but ATOMIC (the warp-dedup modes have no level-major form);
// lane pairs for RUN_LANES.
template <int F, typename GT>
int launch_backward_levels(const hashgrid_s* h, const float* x, const float* dout, int64_t N, GT* dtable,
                           cudaStream_t s) {
    if constexpr (F <= 4) {
        if (run_lanes(h)) {
            const int64_t runs = (N + hg::kRun - 1) / hg::kRun;
            const dim3 grid((unsigned)((2 * runs + hg::kLevelBlock - 1) / hg::kLevelBlock), (unsigned)h->lp.ngroups);
            hg::backward_kernel_runs_levels_lanes<F, GT><<<grid, hg::kLevelBlock, 0, s>>>(h->lp, x, dout, N, dtable);
            return launch_status("backward");
        }
        if (h->backward_mode != HASHGRID_BACKWARD_ATOMIC) {
            const int64_t runs = (N + hg::kRun - 1) / hg::kRun;
            const dim3 grid((unsigned)((runs + hg::kLevelBlock - 1) / hg::kLevelBlock), (unsigned)h->L);
            hg::backward_kernel_runs_levels<F, GT><<<grid, hg::kLevelBlock, 0, s>>>(h->lp, x, dout, N, dtable);
            return launch_status("backward");
        }
    }
    const dim3 grid((unsigned)((N + hg::kLevelBlock - 1) / hg::kLevelBlock), (unsigned)h->L);
    hg::backward_kernel_atomic_levels<F, GT><<<grid, hg::kLevelBlock, 0, s>>>(h->lp, x, dout, N, dtable);
    return launch_status("backward");
}

template <int F, typename GT = float>
int launch_backward_runs(const hashgrid_s* h, const float* x, const float* dout, int64_t N,
                         GT* dtable, cudaStream_t s) {
    const bool lanes = run_lanes(h);
    auto k = lanes ? hg::backward_kernel_runs_lanes<F, GT> : hg::backward_kernel_runs<F, GT>;
    const size_t smem = lanes ? hg::run_smem_bytes(h->L, F, hg::kRunPairTile / hg::kRunPair, hg::kRunPair)
                              : hg::run_smem_bytes(h->L, F);
    if (int rc = prepare_smem(k, smem)) return rc;
    const int64_t tile = lanes ? hg::kRunPairTile : hg::kRunTile;
    const unsigned blocks = (unsigned)((N + tile - 1) / tile);
    k<<<blocks, 256, smem, s>>>(h->lp, x, dout, N, dtable);
    return launch_status("backward");
}

// fp16 gradient tables: run merging (every mode but ATOMIC) or per-point reductions.
template <int F>
int launch_backward_half(const hashgrid_s* h, const float* x, const float* dout, int64_t N, __half* dtable,
                         cudaStream_t s) {
    if (level_major(h)) return launch_backward_levels<F, __half>(h, x, dout, N, dtable, s);
    if constexpr (F <= 4) {
        if (h->backward_mode != HASHGRID_BACKWARD_ATOMIC) return launch_backward_runs<F, __half>(h, x, dout, N, dtable, s);
    }
    return launch_backward_mode<F, hg::kAtomicOnly, __half>(h, x, dout, N, dtable, s);
}

template <int F>
int launch_backward(const hashgrid_s* h, const float* x, const float* dout, int64_t N,
                    float* dtable, cudaStream_t s) {
    const bool grouped = h->backward_mode == HASHGRID_BACKWARD_WARP_DEDUP ||
                         h->backward_mode == HASHGRID_BACKWARD_WARP_DEDUP_ADAPTIVE;
    if (!grouped && level_major(h)) return launch_backward_levels<F, float>(h, x, dout, N, dtable, s);
    if constexpr (F <= 4) {
        if (h->backward_mode == HASHGRID_BACKWARD_RUN_MERGE || h->backward_mode == HASHGRID_BACKWARD_AUTO ||
            h->backward_mode == HASHGRID_BACKWARD_RUN_LANES)
            return launch_backward_runs<F>(h, x, dout, N, dtable, s);
        if (h->backward_mode == HASHGRID_BACKWARD_WARP_DEDUP)
            return launch_backward_mode<F, hg::kGroupAlways>(h, x, dout, N, dtable, s);
        if (h->backward_mode == HASHGRID_BACKWARD_WARP_DEDUP_ADAPTIVE)
            return launch_backward_mode<F, hg::kAdaptive>(h, x, dout, N, dtable, s);
    }
    return launch_backward_mode<F, hg::kAtomicOnly>(h, x, dout, N, dtable, s);
}

// dL/dx: warp-owned lane pairs when the gather option selects lane pairs (AUTO, LANES),
// else one thread per (point, level). A warp stages its 16 upstream-gradient rows: 16 warps
// per block for rows of up to 64 floats, 4 above (shared memory).
template <int F, typename TT, int kW>
int launch_backward_input_warp(const hashgrid_s* h, const float* x, const float* dout, int64_t N, const void* table,
                               float* dx, cudaStream_t s) {
    auto k = hg::backward_input_kernel_warp<F, TT, kW>;
    const size_t smem = sizeof(float) * (size_t)kW * hg::kWarpPoints * (h->L * F + hg::row_pad(F));
    if (int rc = prepare_smem(k, smem)) return rc;
    const int64_t pts = (int64_t)kW * hg::kWarpPoints;
    k<<<(unsigned)((N + pts - 1) / pts), 32 * kW, smem, s>>>(h->lp, x, dout, N, static_cast<const TT*>(table), dx);
    return launch_status("backward_input");
}

template <int F, typename TT>
int launch_backward_input(const hashgrid_s* h, const float* x, const float* dout, int64_t N, const void* table,
                          float* dx, cudaStream_t s) {
    if (forward_gather_kernel(h) == hg::kGatherLanes)
        return h->L * F <= 64 ? launch_backward_input_warp<F, TT, 16>(h, x, dout, N, table, dx, s)
                              : launch_backward_input_warp<F, TT, 4>(h, x, dout, N, table, dx, s);
    auto k = hg::backward_input_kernel<F, TT, kTile>;
    const size_t smem = hg::input_grad_smem_bytes(kTile, h->L, F);
    if (int rc = prepare_smem(k, smem)) return rc;
    const unsigned blocks = (unsigned)((N + kTile - 1) / kTile);
    k<<<blocks, tile_threads(h->L), smem, s>>>(h->lp, x, dout, N, static_cast<const TT*>(table), dx);
    return launch_status("backward_input");
}

template <int F, typename TT, int K1>
int launch_mlp_forward(const hashgrid_s* h, const float* x, int64_t N, const void* table, const void* w1,
                       const float* b1, const void* w2, const float* b2, const void* w3, const float* b3, float* y,
                       int* status, cudaStream_t s) {
    // lane-pair producers when the gather option selects lane pairs (F <= 4)
    constexpr bool kCanLanes = F <= 4;
    const bool lanes = kCanLanes && forward_gather_kernel(h) == hg::kGatherLanes;
    auto k = lanes ? hg::mlp::mlp_forward_kernel<F, TT, K1, kCanLanes> : hg::mlp::mlp_forward_kernel<F, TT, K1, false>;
    const size_t smem = hg::mlp::ws_smem_bytes(K1);
    if (int rc = prepare_smem(k, smem)) return rc;
    int dev = 0, sms = 148, smem_sm = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
    // Persistent grid: as many CTAs as fit per SM (registers allow 2; shared memory as
    // computed, with the 1 KB the runtime reserves per CTA). More would only queue behind the
    // resident ones.
    const int fit = (int)((size_t)smem_sm / (smem + 1024));
    const int per_sm = std::max(1, std::min(hg::mlp::kCtasPerSm, fit));
    const int64_t tiles = (N + hg::mlp::kM - 1) / hg::mlp::kM;
    const int64_t cap = (int64_t)sms * per_sm;
    const unsigned blocks = (unsigned)(tiles < cap ? tiles : cap);
    k<<<blocks, hg::mlp::block_threads(F, lanes), smem, s>>>(h->lp, x, N, static_cast<const TT*>(table),
                                               static_cast<const uint16_t*>(w1), b1, static_cast<const uint16_t*>(w2),
                                               b2, static_cast<const uint16_t*>(w3), b3, y, status);
    return launch_status("mlp_forward");
}

template <int F, typename TT>
int dispatch_mlp_forward(const hashgrid_s* h, const float* x, int64_t N, const void* table, const void* w1,
                         const float* b1, const void* w2, const float* b2, const void* w3, const float* b3, float* y,
                         int* status, cudaStream_t s) {
    switch (h->L * F) {
        case 16: return launch_mlp_forward<F, TT, 16>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, status, s);
        case 32: return launch_mlp_forward<F, TT, 32>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, status, s);
        case 48: return launch_mlp_forward<F, TT, 48>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, status, s);
        case 64: return launch_mlp_forward<F, TT, 64>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, status, s);
    }
    return fail(HASHGRID_ERR_ARG, "the MLP needs L*F in {16, 32, 48, 64}, got %d", h->L * F);
}

// D-dimensional inputs (D = 2, 4): per-corner gathers and per-point reductions, with lane
// pairs (two threads per (point, level), split by x offset) when the LANES gather option
// (forward, dL/dx) or the RUN_LANES backward option asks for them, and under AUTO for D = 4.
// Measured per 2^20 uniform points of the default grid: D = 4 forward 533 against 802 us,
// backward 784 against 927, dL/dx 569 against 764; D = 2 forward 185 against 161 us, backward
// 449 against 415 (4 corners: the duplicated locate and hash cost more than the shared
// sectors save).
bool nd_lanes_fwd(const hashgrid_s* h) {
    return h->forward_gather == HASHGRID_GATHER_LANES || (h->forward_gather == HASHGRID_GATHER_AUTO && h->D == 4);
}
bool nd_lanes_bwd(const hashgrid_s* h) {
    return h->backward_mode == HASHGRID_BACKWARD_RUN_LANES || (h->backward_mode == HASHGRID_BACKWARD_AUTO && h->D == 4);
}

int nd_threads(const hashgrid_s* h, bool lanes) {
    const int items = (hg::nd::kTile / (lanes ? 16 : 32)) * h->L;
    return items * 32 < kMaxThreads ? items * 32 : kMaxThreads;
}

template <int D, int F, typename TT>
int launch_nd_forward(const hashgrid_s* h, const float* x, int64_t N, const void* table, float* out, cudaStream_t s) {
    const bool lanes = nd_lanes_fwd(h);
    auto k = lanes ? hg::nd::forward_kernel<D, F, TT, true> : hg::nd::forward_kernel<D, F, TT, false>;
    const size_t smem = hg::nd::tile_smem_bytes(D, h->L, F);
    if (int rc = prepare_smem(k, smem)) return rc;
    k<<<(unsigned)((N + hg::nd::kTile - 1) / hg::nd::kTile), nd_threads(h, lanes), smem, s>>>(
        h->lp, x, N, static_cast<const TT*>(table), out);
    return launch_status("forward");
}

template <int D, int F, typename GT>
int launch_nd_backward(const hashgrid_s* h, const float* x, const float* dout, int64_t N, GT* dtable, cudaStream_t s) {
    const bool lanes = nd_lanes_bwd(h);
    auto k = lanes ? hg::nd::backward_kernel<D, F, GT, true> : hg::nd::backward_kernel<D, F, GT, false>;
    const size_t smem = hg::nd::tile_smem_bytes(D, h->L, F);
    if (int rc = prepare_smem(k, smem)) return rc;
    k<<<(unsigned)((N + hg::nd::kTile - 1) / hg::nd::kTile), nd_threads(h, lanes), smem, s>>>(h->lp, x, dout, N, dtable);
    return launch_status("backward");
}

template <int D, int F, typename TT>
int launch_nd_backward_input(const hashgrid_s* h, const float* x, const float* dout, int64_t N, const void* table,
                             float* dx, cudaStream_t s) {
    const bool lanes = nd_lanes_fwd(h);
    auto k = lanes ? hg::nd::backward_input_kernel<D, F, TT, true> : hg::nd::backward_input_kernel<D, F, TT, false>;
    const size_t smem = hg::nd::tile_smem_bytes(D, h->L, F) + sizeof(float) * (size_t)hg::nd::kTile * h->L * D;
    if (int rc = prepare_smem(k, smem)) return rc;
    k<<<(unsigned)((N + hg::nd::kTile - 1) / hg::nd::kTile), nd_threads(h, lanes), smem, s>>>(
        h->lp, x, dout, N, static_cast<const TT*>(table), dx);
    return launch_status("backward_input");
}

// Calls fn<D, F>() for the handle's D (2 or 4) and F.
template <class Fn>
int nd_dispatch(const hashgrid_s* h, Fn&& fn) {
#define HG_ND_CASE(DD, FF) \
    if (h->D == DD && h->F == FF) return fn(std::integral_constant<int, DD>(), std::integral_constant<int, FF>());
    HG_ND_CASE(2, 1) HG_ND_CASE(2, 2) HG_ND_CASE(2, 4) HG_ND_CASE(2, 8)
    HG_ND_CASE(4, 1) HG_ND_CASE(4, 2) HG_ND_CASE(4, 4) HG_ND_CASE(4, 8)
#undef HG_ND_CASE
    return fail(HASHGRID_ERR_ARG, "corrupt handle");
}

// Buffers of one call for the checked build's range checks: (role, base, bytes).
struct CheckBuf {
    int role;
    const void* p;
    size_t bytes;
};

// Runs fn (the call's launches). In the checked build (HASHGRID_CHECKED) the byte ranges
// of the call's buffers are first recorded for the kernels' range checks (roles the call
// does not use stay unrestricted), and after the launches the device status word is read
// back on the call's stream: a tripped check is cleared and reported as
// HASHGRID_ERR_DEVICE_CHECK. Calls are then synchronous, and calls running at the same
// time on several streams would share the recorded ranges: the checked build is for one
// stream at a time. In the regular build this only calls fn.
template <class Fn>
int run_checked(cudaStream_t s, std::initializer_list<CheckBuf> bufs, const char* what, Fn&& fn) {
#ifdef HASHGRID_CHECKED
    // the status word is read back after the kernel: not possible inside stream capture
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) {
        cudaGetLastError();
        return fail(HASHGRID_ERR_CUDA, "%s: cudaStreamIsCapturing failed", what);
    }
    if (cap != cudaStreamCaptureStatusNone)
        return fail(HASHGRID_ERR_ARG, "%s: the checked build cannot run inside stream capture", what);
    hg::CheckRanges r;
    for (int i = 0; i < hg::kChkRoles; ++i) {
        r.lo[i] = 0;
        r.hi[i] = ~0ull;
    }
    for (const CheckBuf& b : bufs) {
        r.lo[b.role] = (uint64_t)(uintptr_t)b.p;
        r.hi[b.role] = (uint64_t)(uintptr_t)b.p + b.bytes;
    }
    // Test hook: HASHGRID_CHECK_SHRINK_OUT=n records the output buffer n bytes shorter than
    // it is, so that a test can make the checks trip on accesses that still lie inside the
    // caller's buffer.
    if (const char* shrink = std::getenv("HASHGRID_CHECK_SHRINK_OUT")) {
        const uint64_t n = std::strtoull(shrink, nullptr, 10);
        if (r.hi[hg::kChkOut] != ~0ull) r.hi[hg::kChkOut] -= std::min<uint64_t>(n, r.hi[hg::kChkOut] - r.lo[hg::kChkOut]);
    }
    if (cudaMemcpyToSymbolAsync(hg::g_check_ranges, &r, sizeof r, 0, cudaMemcpyHostToDevice, s) != cudaSuccess) {
        cudaGetLastError();
        return fail(HASHGRID_ERR_CUDA, "%s: recording the checked ranges failed", what);
    }
    const int rc = fn();
    if (rc != HASHGRID_OK) return rc;
    unsigned int flags = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&flags, hg::g_check_flags, sizeof flags, 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(HASHGRID_ERR_CUDA, "%s: reading the device status failed: %s", what, cudaGetErrorString(e));
    }
    if (flags != 0) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(hg::g_check_flags, &zero, sizeof zero);
        static const char* names[hg::kChkRoles] = {"x", "table", "output", "dL_dout", "dL_dtable", "adam_m", "adam_v",
                                                   "weights", "bias", "residual", "z", "workspace", "AdamW tensor"};
        std::string which;
        for (int i = 0; i < hg::kChkRoles; ++i)
            if (flags & (1u << i)) which += std::string(which.empty() ? "" : ", ") + names[i];
        return fail(HASHGRID_ERR_DEVICE_CHECK, "%s: a device range check tripped on %s (the access was skipped)", what,
                    which.c_str());
    }
    return rc;
#else
    (void)s;
    (void)bufs;
    (void)what;
    return fn();
#endif
}

size_t table_bytes(const hashgrid_s* h) {
    return (size_t)h->L * ((size_t)1 << h->log2T) * (size_t)h->F * (h->dtype == HASHGRID_F16 ? 2 : 4);
}

int check_layer(const hashgrid_linear_s* layer) {
    if (layer == nullptr) return fail(HASHGRID_ERR_ARG, "layer is NULL");
    return ok();
}

// Bytes of a row-major [rows, cols] array whose rows lie ld elements apart.
size_t strided_bytes(int64_t rows, int64_t cols, int64_t ld, size_t elem) {
    return rows == 0 ? 0 : ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * elem;
}

// One strided array of a layer call: its row stride and then its extent.
int check_rows(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t elem, const char* name) {
    if (ld < cols) return fail(HASHGRID_ERR_ARG, "%s: row stride %lld is below its width %lld", name, (long long)ld, (long long)cols);
    if (rows > 1 && ld >= ((int64_t)1 << 37)) return fail(HASHGRID_ERR_ARG, "%s: row stride %lld is too large", name, (long long)ld);
    // an extent in bytes could pass 64 bits and come out small
    if (rows > 1 && rows - 1 > ((int64_t)1 << 48) / ld)
        return fail(HASHGRID_ERR_ARG, "%s: %lld rows %lld elements apart are more than any memory holds", name, (long long)rows, (long long)ld);
    return check_buffer(p, strided_bytes(rows, cols, ld, elem), name);
}

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 256;

int check_row_count(int64_t N) {
    if (N < 0 || N >= kMaxRows) return fail(HASHGRID_ERR_ARG, "N = %lld outside [0, 2^31 - 256)", (long long)N);
    return ok();
}

int check_workspace(const void* p, size_t have, size_t need, int64_t N) {
    if (need == 0) return ok();
    if (have < need) return fail(HASHGRID_ERR_ARG, "workspace of %zu bytes, %zu are needed for N = %lld", have, need, (long long)N);
    return check_buffer(p, need, "workspace");
}

int check_out_type(const hashgrid_linear_s* layer, int dtype, const char* name) {
    if (dtype != HASHGRID_F32 && dtype != layer->dtype)
        return fail(HASHGRID_ERR_ARG, "%s = %d is neither HASHGRID_F32 nor the layer's dtype %d", name, dtype, layer->dtype);
    return ok();
}

// Rows of bytes, `stride` apart.
struct Region {
    const char* name;
    const void* p;
    int64_t rows, width, stride;
};

Region region(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t elem) {
    if (rows <= 1 || ld == cols) return Region{name, p, 1, rows * cols * (int64_t)elem, rows * cols * (int64_t)elem};
    return Region{name, p, rows, cols * (int64_t)elem, ld * (int64_t)elem};
}
Region region(const char* name, const void* p, size_t bytes) { return Region{name, p, 1, (int64_t)bytes, (int64_t)bytes}; }

// The smallest x >= 0 with lo <= a x mod m <= hi (0 <= a < m, 0 <= lo <= hi < m), or -1. Where no multiple of a lies
// within [lo, hi], a x - m y does for the smallest y with m y mod a in [-hi, -lo] mod a: Euclid's steps.
__int128 first_multiple(__int128 a, __int128 m, __int128 lo, __int128 hi) {
    if (lo == 0) return 0;
    if (a == 0) return -1;
    const __int128 x = (lo + a - 1) / a;
    if (a * x <= hi) return x;
    const __int128 y = first_multiple(m % a, a, a - hi % a, a - lo % a);
    return y < 0 ? -1 : (lo + m * y + a - 1) / a;
}

// Whether any byte belongs to both. Exact, so that columns of one buffer pass as different arrays.
bool overlap(const Region& a, const Region& b) {
    if (a.p == nullptr || b.p == nullptr || a.rows * a.width == 0 || b.rows * b.width == 0) return false;
    const __int128 a0 = (__int128)(uintptr_t)a.p, b0 = (__int128)(uintptr_t)b.p;
    const __int128 a1 = a0 + (__int128)(a.rows - 1) * a.stride + a.width, b1 = b0 + (__int128)(b.rows - 1) * b.stride + b.width;
    if (a1 <= b0 || b1 <= a0) return false;
    // a's first row that ends behind b's start
    const __int128 i = b0 < a0 + a.width ? 0 : (b0 - a0 - a.width) / a.stride + 1, at = a0 + i * a.stride;
    if (at <= b0) return true;
    // the first from there on that begins, in steps of b's rows, less than b's width behind a row's start or less than its own before
    const __int128 m = b.stride, c = (at - b0) % m;
    if (c < b.width || c + a.width > m) return i < a.rows && at < b1;
    const __int128 x = first_multiple(a.stride % m, m, m - a.width + 1 - c, m + b.width - 1 - c);
    return x >= 0 && i + x < a.rows && at + x * a.stride < b1;
}

// No output may overlap another one or an input.
int check_apart(std::initializer_list<Region> outputs, std::initializer_list<Region> inputs) {
    for (const Region* o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Region* other = o + 1; other != outputs.end(); ++other)
            if (overlap(*o, *other)) return fail(HASHGRID_ERR_ARG, "%s and %s overlap", o->name, other->name);
        for (const Region& in : inputs)
            if (overlap(*o, in)) return fail(HASHGRID_ERR_ARG, "%s and %s overlap", o->name, in.name);
    }
    return ok();
}

// prepare_smem once for each kernel, size and device: the attribute call costs as much as a small launch's checks.
template <typename K>
int prepare_smem_once(K kernel, size_t smem) {
    struct Entry {
        const void* kernel;
        int device;
        size_t smem;
    };
    static std::mutex lock;
    static Entry table[64];
    static int used = 0;
    int dev = 0;
    cudaGetDevice(&dev);
    const void* key = reinterpret_cast<const void*>(kernel);
    std::lock_guard<std::mutex> hold(lock);
    for (int i = 0; i < used; ++i)
        if (table[i].kernel == key && table[i].device == dev) {
            if (table[i].smem >= smem) return ok();
            if (int rc = prepare_smem(kernel, smem)) return rc;
            table[i].smem = smem;
            return ok();
        }
    if (int rc = prepare_smem(kernel, smem)) return rc;
    if (used < 64) table[used++] = Entry{key, dev, smem};
    return ok();
}

typedef CUresult (*PFN_tensorMapEncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

PFN_tensorMapEncodeTiled tensor_map_fn() {
    static PFN_tensorMapEncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<PFN_tensorMapEncodeTiled>(p);
    }();
    return fn;
}

int device_sms() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// An operand of a product: a row-major [outer, inner] array of 16-bit elements, rows ld apart. mn:
// its rows run along k (it is read "transposed").
struct Array {
    const void* p;
    int64_t outer, inner, ld;
    bool mn;
    int role;
};

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Launches a kernel that waits itself for what comes before it in the stream (after_previous_kernel), so
// that its start overlaps the end of the previous one.
template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t s, const char* what,
                 const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(HASHGRID_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
    }
    return ok();
}

// What hashgrid_debug_wait_limit set, or nothing (< 0).
std::atomic<int64_t> g_wait_limit{-1};

// How long a layer's kernel waits. Test hook of the checked build: HASHGRID_CHECK_GIVE_UP=role,n,parity makes the nth wait
// of a role's warps give up (copying 1, multiplying 2, writing out 3, making dz 4), in the even (0), odd (1) or all (2) blocks.
hg::linear::Patience patience() {
    const int64_t limit = g_wait_limit.load(std::memory_order_relaxed);
    hg::linear::Patience p = {};
    p.polls = limit < 0 ? hg::mlp::kWaitLimit : (uint32_t)std::min<int64_t>(limit, hg::mlp::kWaitLimit);
#ifdef HASHGRID_CHECKED
    if (const char* text = std::getenv("HASHGRID_CHECK_GIVE_UP"))
        if (std::sscanf(text, "%d,%d,%d", &p.role, &p.nth, &p.parity) != 3) p.role = p.nth = 0;
#endif
    return p;
}

// A device's status word for layer calls that are given none: pinned memory, which the kernels write and the host reads
// at the next call. NULL where there is none to be had, or none yet and `make` is not set.
volatile int* given_up_word(bool make) {
    constexpr int kDevices = 64, kApart = 32;
    static std::mutex lock;
    static std::atomic<int*> words{nullptr};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) {
        cudaGetLastError();
        return nullptr;
    }
    int* p = words.load(std::memory_order_acquire);
    if (p == nullptr && make) {
        std::lock_guard<std::mutex> hold(lock);
        p = words.load(std::memory_order_relaxed);
        if (p == nullptr) {
            // the first call may come inside a stream's capture, which this allocation is no part of
            cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
            cudaThreadExchangeStreamCaptureMode(&mode);
            void* fresh = nullptr;
            const cudaError_t e = cudaHostAlloc(&fresh, kDevices * kApart * sizeof(int), cudaHostAllocPortable | cudaHostAllocMapped);
            cudaThreadExchangeStreamCaptureMode(&mode);
            if (e != cudaSuccess) {
                cudaGetLastError();
                return nullptr;
            }
            p = static_cast<int*>(fresh);
            std::memset(p, 0, kDevices * kApart * sizeof(int));
            words.store(p, std::memory_order_release);
        }
    }
    return p == nullptr ? nullptr : p + dev * kApart;
}

// Reports, once, that an earlier layer call without a status word gave up.
int check_given_up() {
    volatile int* word = given_up_word(false);
    if (word == nullptr || *word == 0) return ok();
    *word = 0;
    return fail(HASHGRID_ERR_TIMEOUT, "an earlier layer call on this device gave up a wait: its outputs are incomplete");
}

// The status word of a layer call.
int* status_word(int* device_status) { return device_status != nullptr ? device_status : const_cast<int*>(given_up_word(true)); }

// How a product is cut.
struct Plan {
    int bn;       // tile width, a multiple of 16
    int cluster;  // blocks that share a tile's K, their shares added through shared memory
    int splits;   // or parts of K that go to a workspace
    bool pair;    // 256-row tiles by pairs of SMs
};

// The width of N's column tiles where they are nt: a multiple of 16, or, where there are several that may leave by TMA
// stores, of the 32 columns of a store (which knows the array's end, not the tile's).
int tile_width(int64_t N, int64_t nt) {
    const int unit = nt > 1 && N % 4 == 0 ? 32 : 16;
    return ceil_div(ceil_div(N, nt), unit) * unit;
}
int wide_tile(int64_t N, int most) { return tile_width(N, ceil_div(N, most)); }

// Where 256 x 256 tiles by pairs of SMs occupy the device and K is long: those. Else 128-row tiles of up to
// 128 columns, two blocks a SM, since with few steps of K what counts is how many warps write out. The
// number of column tiles is the one that costs least in rounds of the device times a tile's width (and
// 24 columns' worth of what a tile costs anyway), down to 64 columns; if the tiles are still fewer than the SMs, K is
// split over up to 8 blocks of a cluster, each with two 64-wide steps at least.
Plan make_plan(int64_t M, int64_t N, int64_t K, bool f32, int sms) {
    const int64_t mt = ceil_div(M, hg::linear::kBm);
    const int64_t pairs = ceil_div(N, 256);
    if (N >= 160 && (int64_t)ceil_div(M, 256) * pairs >= sms / 2 && K >= 512)
        return Plan{ceil_div(ceil_div(N, pairs), 32) * 32, 1, 1, true};
    int64_t best = INT64_MAX;
    Plan p{0, 1, 1, false};
    for (int64_t nt = ceil_div(N, 128); nt <= ceil_div(N, 64); ++nt) {
        const int bn = tile_width(N, nt);
        const int64_t tiles = mt * ceil_div(N, bn), cost = (tiles + 2 * sms - 1) / (2 * sms) * (bn + 24);
        if (cost < best) {
            best = cost;
            p.bn = bn;
        }
    }
    const int64_t tiles = mt * ceil_div(N, p.bn);
    while (p.cluster < 8 && tiles * p.cluster * 2 <= 2 * sms && 4 * p.cluster * hg::linear::kBk <= K) p.cluster *= 2;
    const int64_t steps = ceil_div(K, hg::linear::kBk), most = hg::linear::kSegment16;
    if (f32 || steps <= most * p.cluster) return p;
    // A 16-bit result of a sum that would have to be gathered, by one block an SM: it is split into shares that need not be
    // (65536 x 2048 by 2048: 574 us, gathered 616), or, beyond eight of those, into tiles and shares that leave the last round
    // of one block an SM full. Of clusters of 4 and 8 such blocks 132 and 120 fit (2^19 x 1280 by 1024: 1.9 ms, 4.3 as above).
    for (int c = 2 * p.cluster; c <= 8; c *= 2)
        if (steps <= most * c) {
            p.cluster = c;
            return p;
        }
    best = INT64_MAX;
    for (int64_t nt = ceil_div(N, 128); nt <= ceil_div(N, 64); ++nt)
        for (int c = 1; c <= 8; c *= 2) {
            const int bn = tile_width(N, nt), fit = c == 8 ? sms * 13 / 16 : c == 4 ? sms * 29 / 32 : sms;
            const int64_t cost = (mt * ceil_div(N, bn) * c + fit - 1) / fit * (128 + bn) * (8 / c);
            if (cost < best) {
                best = cost;
                p.bn = bn;
                p.cluster = c;
            }
        }
    return p;
}

// The map of an array that is copied in boxes of box_rows x 64 elements, 128-byte-swizzled.
int set_map(CUtensorMap& map, const Array& a, int box_rows, const char* what) {
    const cuuint64_t dims[2] = {(cuuint64_t)a.inner, (cuuint64_t)a.outer};
    const cuuint64_t strides[1] = {(cuuint64_t)(a.outer > 1 ? a.ld : (a.inner + 7) / 8 * 8) * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, ones[2] = {1, 1};
    PFN_tensorMapEncodeTiled encode = tensor_map_fn();
    const CUresult r = encode == nullptr ? CUDA_ERROR_NOT_SUPPORTED
                                         : encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(a.p), dims, strides, box, ones,
                                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(HASHGRID_ERR_CUDA, "%s: encoding a tensor map failed (%d)", what, (int)r);
    return ok();
}

// The map of an output of `parts` row-major [rows, cols] arrays, stored in chunks of 32 x 32.
int set_store_map(CUtensorMap& map, void* p, int64_t rows, int64_t cols, int64_t ld, int parts, bool f32, const char* what) {
    const cuuint64_t elem = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
    if (rows <= 1 && parts <= 1) ld = (cols + 7) / 8 * 8;  // no row follows
    const cuuint64_t strides[2] = {(cuuint64_t)ld * elem, (cuuint64_t)(parts > 1 ? rows * ld : ld) * elem};
    const cuuint32_t box[3] = {32, 32, 1}, ones[3] = {1, 1, 1};
    PFN_tensorMapEncodeTiled encode = tensor_map_fn();
    const CUresult r = encode == nullptr ? CUDA_ERROR_NOT_SUPPORTED
                                         : encode(&map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, p, dims, strides, box,
                                                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(HASHGRID_ERR_CUDA, "%s: encoding a tensor map failed (%d)", what, (int)r);
    return ok();
}

// One operand's share of a stage, and its tensor map. `wanted` rows (or columns) of it are staged at a
// time; those that the array does not have are left out.
int set_side(hg::linear::Side& s, CUtensorMap& map, const Array& a, int wanted, const char* what) {
    const int64_t extent = a.mn ? a.inner : a.outer;
    s.mn = a.mn;
    if (a.mn) {
        s.box_rows = hg::linear::kBk;
        s.boxes = ceil_div(std::min<int64_t>(wanted, extent), 64);
    } else {
        s.box_rows = (int)std::min<int64_t>(wanted, ceil_div(extent, 8) * 8);
        s.boxes = 1;
    }
    s.bytes = s.box_rows * s.boxes * 128;
    return set_map(map, a, s.box_rows, what);
}

bool vector_rows(const void* p, int64_t ld, size_t elem) { return p == nullptr || ((size_t)ld * elem) % 16 == 0; }

// A product ready to be launched: D[M, N] = A B^T over K on the tensor cores. plan.splits > 1: K is cut into
// so many parts, each an fp32 [M, N] of its own in e.out.
struct Product {
    hg::linear::Gemm g;
    int64_t grid;  // blocks
    size_t smem;
    bool vectors, gather;
};

// low: A's low part, or NULL.
int set_product(Product& p, bool half, const Array& A, const Array* low, const Array& B, int64_t M, int64_t N, int64_t K, const hg::linear::Epilogue& e,
                const Plan& plan, int* status, const char* what) {
    namespace hl = hg::linear;
    const int bn = plan.bn, splits = std::max(plan.splits, plan.cluster), group = plan.pair ? 2 : 1;
    hl::Gemm& g = p.g;
    if (int rc = set_side(g.a, g.ta, A, hl::kBm, what)) return rc;
    if (low != nullptr)
        if (int rc = set_map(g.ta_low, *low, g.a.box_rows, what)) return rc;
    if (int rc = set_side(g.b, g.tb, B, bn / group, what)) return rc;
    g.M = M;
    g.N = N;
    g.bn = bn;
    g.columns = ceil_div(bn, 32) * 32;
    g.tmem_columns = 64;
    while ((int)g.tmem_columns < 2 * g.columns) g.tmem_columns *= 2;
    g.kfold = ceil_div(K, hl::kBk);
    g.kblocks = low != nullptr ? 2 * g.kfold : g.kfold;
    g.kblocks_per_split = ceil_div(g.kblocks, splits);
    g.mt = ceil_div(M, hl::kBm * group);
    g.nt = ceil_div(N, bn);
    const int sms = device_sms();
    const int64_t tiles = (int64_t)g.mt * g.nt;
    if (tiles > (1 << 30)) return fail(HASHGRID_ERR_ARG, "%s: too many tiles", what);
    // B stays in shared memory where one column tile covers it, it is small and its block has several tiles to compute.
    const bool two = e.out_f32 && e.z != nullptr;  // staging areas
    g.resident = splits == 1 && group == 1 && g.nt == 1 && g.kfold * g.b.bytes <= (two ? 8 : 32) * 1024 && g.mt > 2 * sms;
    const int kept = g.resident ? g.kfold * g.b.bytes : 0;
    g.stage_bytes = g.a.bytes + (g.resident ? 0 : g.b.bytes);
    g.cluster = plan.cluster;
    // Two blocks a SM where tensor memory and shared memory allow: one's loads and stores then fill the other's gaps. The MMA
    // reads 128 rows (two boxes) of A whatever the product has: the staging area behind the stages keeps that in bounds.
    p.gather = g.kblocks_per_split > (e.out_f32 ? hl::kSegment : hl::kSegment16);
    const int per_sm = group == 1 && g.tmem_columns <= 256 && !p.gather ? 2 : 1;
    const int budget = (per_sm == 2 ? 113 : 227) * 1024 - 1024;  // less what the kernel has of its own
    g.stages = std::min(hl::kMaxStages, (budget - kept - (int)hl::gemm_smem(0, two)) / g.stage_bytes);
    if (g.cluster > 1)  // a split product's shares lie in the stages
        while (g.stages * g.stage_bytes < 4 * ceil_div(bn, 32) * 4096) ++g.stages;
    if (g.stages < 1) return fail(HASHGRID_ERR_ARG, "%s: no stage fits", what);  // does not happen: a stage has 48 KB at most
    const uint32_t type = half ? 0u : 1u;
    g.idesc = (1u << 4) | (type << 7) | (type << 10) | ((A.mn ? 1u : 0u) << 15) | ((B.mn ? 1u : 0u) << 16) |
              ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(hl::kBm * group >> 4) << 24);
    g.e = e;
    const size_t os = e.out_f32 ? 4 : 2;
    g.split_stride = plan.splits > 1 ? M * N : 0;
    // TMA writes whole 16-byte units: a last one that the product fills in part would take the caller's values behind it along.
    p.vectors = N * os % 16 == 0 && vector_rows(e.out, e.ldo, os) && vector_rows(e.residual, e.ldr, os) && vector_rows(e.z, e.ldz, 2);
    if (p.vectors) {
        if (int rc = set_store_map(g.ty, e.out, M, N, e.ldo, plan.splits, e.out_f32 != 0, what)) return rc;
        if (e.z != nullptr)
            if (int rc = set_store_map(g.tz, e.z, M, N, e.ldz, 1, false, what)) return rc;
    }
    g.status = status;
    p.smem = hl::gemm_smem(g.stages * g.stage_bytes + kept, two);
    g.blocks = (int)(plan.cluster > 1 ? tiles : std::min<int64_t>(tiles, std::max(1, per_sm * sms / splits / group)));
    p.grid = (int64_t)g.blocks * splits * group;
    return ok();
}

// Launches one product, or two of the same plan.pair and plan.cluster.
template <typename T>
int launch_products(const Product* p, int count, const Plan& plan, const char* what, cudaStream_t s) {
    namespace hl = hg::linear;
    hl::Gemms l;
    std::memcpy(&l.of[0], &p[0].g, sizeof(hl::Gemm));
    std::memcpy(&l.of[1], &p[count - 1].g, sizeof(hl::Gemm));
    l.patience = patience();
    l.second = count > 1 ? (int)p[0].grid : 0x7fffffff;
    const int64_t grid = p[0].grid + (count > 1 ? p[1].grid : 0);
    const size_t smem = std::max(p[0].smem, p[count - 1].smem);
    const bool vectors = p[0].vectors && p[count - 1].vectors;
    const bool gather = p[0].gather || p[count - 1].gather;
    static void (*const kernels[8])(const hl::Gemms) = {
        hl::gemm_kernel<T, false, false, false>, hl::gemm_kernel<T, false, false, true>, hl::gemm_kernel<T, false, true, false>,
        hl::gemm_kernel<T, false, true, true>,   hl::gemm_kernel<T, true, false, false>, hl::gemm_kernel<T, true, false, true>,
        hl::gemm_kernel<T, true, true, false>,   hl::gemm_kernel<T, true, true, true>};
    auto k = kernels[4 * plan.pair + 2 * vectors + gather];
    if (int rc = prepare_smem_once(k, smem)) return rc;
    return launch_after(k, dim3((unsigned)grid), hl::kThreads, smem, plan.pair ? 2 : plan.cluster, s, what, l);
}

template <typename T>
int launch_gemm(const Array& A, const Array& B, int64_t M, int64_t N, int64_t K, const hg::linear::Epilogue& e, const Plan& plan,
                int* status, const char* what, cudaStream_t s) {
    Product p;
    if (int rc = set_product(p, std::is_same<T, __half>::value, A, nullptr, B, M, N, K, e, plan, status, what)) return rc;
    return launch_products<T>(&p, 1, plan, what, s);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// TMA copies arrays whose rows begin on 16-byte boundaries; others are copied into such rows first.
bool aligned_rows(const Array& a) { return a.outer <= 1 || a.ld % 8 == 0; }
size_t realigned_bytes(int64_t outer, int64_t inner) { return align256((size_t)outer * ((inner + 7) / 8 * 8) * 2); }

// Adds the copies of those of up to two arrays that need one to `l`, and points them there. Returns the bytes
// of `work` that they take.
size_t add_copies(hg::linear::RealignList& l, Array* const* arrays, int count, char* work) {
    std::memset(&l, 0, sizeof l);
    size_t used = 0;
    int n = 0;
    for (int i = 0; i < count; ++i) {
        Array& a = *arrays[i];
        if (aligned_rows(a)) continue;
        hg::linear::Realign& r = l.a[n++];
        r.p = a.p;
        r.to = reinterpret_cast<uint16_t*>(work + used);
        r.bytes = strided_bytes(a.outer, a.inner, a.ld, 2);
        r.outer = a.outer;
        r.ld = a.ld;
        r.chunks = (a.inner + 7) / 8;
        r.inner = (int)a.inner;
        r.role = a.role;
        l.total += a.outer * r.chunks;
        if (n == 1) l.first = l.total;
        used += realigned_bytes(a.outer, a.inner);
        a = Array{r.to, a.outer, a.inner, r.chunks * 8, a.mn, hg::kChkWork};
    }
    return used;
}

// The launch before the products: `slope` (rows = 0: none) and the copies.
template <typename T>
int launch_prepare(const hg::linear::Slope& slope, bool vectors, const hg::linear::RealignList& copies, const char* what, cudaStream_t s) {
    const int64_t slope_blocks = slope.rows == 0 ? 0 : (int64_t)slope.col_blocks * slope.shares, blocks = slope_blocks + (copies.total + 1023) / 1024;
    if (blocks == 0) return ok();
    if (blocks > 0x7fffffffLL) return fail(HASHGRID_ERR_ARG, "%s: too many rows to realign", what);
    auto k = slope.low != nullptr ? (vectors ? hg::linear::prepare_kernel<T, true, true> : hg::linear::prepare_kernel<T, false, true>)
                                  : (vectors ? hg::linear::prepare_kernel<T, true, false> : hg::linear::prepare_kernel<T, false, false>);
    return launch_after(k, dim3((unsigned)blocks), 256, 0, 1, s, what, slope, copies, (int)slope_blocks);
}

// Numbers of the layer's type that dz is held in: behind a smooth activation one would lose as much as a 16-bit result's own
// rounding, and all that an fp32 one has more (4099 x 173 -> 257, SiLU, fp16: off by 2.9e-4 instead of 2.1e-4, in 19 us
// instead of 22; 2^20 x 64 -> 64, GELU: an fp32 dW off by 1.7e-3 instead of below 4e-5, in 113 us instead of 131).
int dz_pieces(const hashgrid_linear_s* l) { return l->act == HASHGRID_ACT_GELU || l->act == HASHGRID_ACT_SILU ? 2 : 1; }

// The backward pass's workspace: the copies of x and w with aligned rows, dz (where dy is not it), the parts of
// db, the parts of dw.
struct LinearWork {
    int64_t lddz;   // elements
    size_t low;     // offset of dz's low part
    int shares;     // row shares of the db sums
    int splits;     // row shares of dw
    size_t dz, sums, dw, bytes;  // offsets, total
};

constexpr int kWorkSms = 148;  // the workspace's size may not depend on the device

// Whether the one-pass kernel takes a layer: its tile of dy, z and x (x 2 stages) and W fit into shared
// memory, and there are 64 tiles or more.
bool narrow_layer(const hashgrid_linear_s* l, int64_t N) {
    if (l->in > 128 || l->out > 128 || N < 64 * hg::linear::kBm) return false;
    const int boxes_out = ceil_div(l->out, 64), boxes_in = ceil_div(l->in, 64);
    const int stage = (boxes_out * (l->act == HASHGRID_ACT_NONE ? 1 : 2) + boxes_in) * hg::linear::kBox;
    return hg::linear::narrow_smem(2 * stage, ceil_div(l->out, 16) * 16 * boxes_in * 128) <= 226 * 1024;
}

// dw sums over the rows. Where its tiles are fewer than the SMs, the rows are cut into so many shares that
// every SM has a tile of one, each share of four 64-row steps at least.
LinearWork linear_work(const hashgrid_linear_s* l, int64_t N, int64_t lddy, int64_t ldx) {
    LinearWork w;
    w.lddz = (l->out + 7) / 8 * 8;
    w.shares = N <= 512 ? 1 : (int)std::min<int64_t>(std::max(1, 2 * kWorkSms / ceil_div(l->out, 64)), (N + 127) / 128);
    const int64_t tiles = (int64_t)ceil_div(l->out, hg::linear::kBm) * ceil_div(l->in, 128);
    w.splits = N <= 512 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(kWorkSms / tiles, N / (4 * hg::linear::kBk)));
    w.dz = (l->in % 8 != 0 ? realigned_bytes(l->out, l->in) : 0) + (ldx % 8 != 0 ? realigned_bytes(N, l->in) : 0);
    w.low = w.dz + align256((size_t)N * w.lddz * 2);
    w.sums = w.dz + (l->act == HASHGRID_ACT_NONE && lddy % 8 == 0 ? 0 : dz_pieces(l) * align256((size_t)N * w.lddz * 2));
    w.dw = w.sums + align256((size_t)w.shares * l->out * sizeof(float));
    const size_t split = w.splits > 1 ? (size_t)w.splits * l->in * l->out : 0;
    const size_t narrow = narrow_layer(l, N) ? (size_t)kWorkSms * (l->in + 1) * l->out : 0;
    w.bytes = w.dw + align256(std::max(split, narrow) * sizeof(float));
    return w;
}

// The sums of up to two arrays' parts.
template <typename T>
int launch_sums(const hg::linear::Sums* list, int count, const char* what, cudaStream_t s) {
    hg::linear::SumsList l;
    std::memset(&l, 0, sizeof l);
    int64_t blocks = 0;
    for (int i = 0; i < count; ++i) {
        l.a[i] = list[i];
        blocks += (list[i].n + 31) / 32;
        if (i == 0) l.blocks0 = (int)blocks;
    }
    if (count == 0) return ok();
    if (blocks > 0x7fffffffLL) return fail(HASHGRID_ERR_ARG, "%s: too many weights", what);
    return launch_after(hg::linear::sum_parts_kernel<T>, dim3((unsigned)blocks), 256, 0, 1, s, what, l);
}

template <typename T>
int launch_narrow_backward(const hashgrid_linear_s* l, int act, int pieces, const Array& dy, const Array& x, int64_t N, const Array& w, const Array& z, void* dx,
                           int64_t lddx, int dx_dtype, bool want_db, float* parts, int* blocks_out, int* status, const char* what,
                           cudaStream_t s) {
    namespace hl = hg::linear;
    hl::Narrow g;
    std::memset(&g, 0, sizeof g);
    g.rows = N;
    g.in = l->in;
    g.out = l->out;
    g.act = act;
    g.boxes_in = ceil_div(l->in, 64);
    g.boxes_out = ceil_div(l->out, 64);
    g.columns = ceil_div(l->in, 32) * 32;
    g.tmem_columns = 128;
    while ((int)g.tmem_columns < 4 * g.columns) g.tmem_columns *= 2;
    g.k_out = ceil_div(l->out, 16) * 16;
    if (int rc = set_map(g.tdy, dy, hl::kBm, what)) return rc;
    if (int rc = set_map(g.tx, x, hl::kBm, what)) return rc;
    const bool second = act != HASHGRID_ACT_NONE || pieces == 2;
    g.pieces = pieces;
    if (second)
        if (int rc = set_map(g.tz, z, hl::kBm, what)) return rc;
    if (int rc = set_map(g.tw, dx != nullptr ? w : dy, g.k_out, what)) return rc;
    g.stage_bytes = (g.boxes_out * (second ? 2 : 1) + g.boxes_in) * hl::kBox;
    g.w_bytes = g.k_out * g.boxes_in * 128;
    g.stages = hl::kNarrowStages;
    while (g.stages > 2 && hl::narrow_smem(g.stages * g.stage_bytes, g.w_bytes) > 226 * 1024) --g.stages;
    const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
    const uint32_t id = (1u << 4) | (type << 7) | (type << 10) | (1u << 16) | ((uint32_t)(ceil_div(l->in, 16) * 16 >> 3) << 17) |
                        ((uint32_t)(hl::kBm >> 4) << 24);
    g.id_dx = id;
    g.id_dw = id | (1u << 15);
    g.e = hl::Epilogue{nullptr, nullptr, dx, nullptr, 0, lddx, 0, dx_dtype == HASHGRID_F32, hl::kNoAct, hg::kChkOut};
    const size_t xs = dx_dtype == HASHGRID_F32 ? 4 : 2;
    const bool vectors = dx == nullptr || (l->in * xs % 16 == 0 && vector_rows(dx, lddx, xs));
    if (dx != nullptr && vectors)
        if (int rc = set_store_map(g.tdx, dx, N, l->in, lddx, 1, dx_dtype == HASHGRID_F32, what)) return rc;
    g.parts = parts;
    g.want_db = want_db;
    g.status = status;
    g.patience = patience();
    const int blocks = std::min(std::min(kWorkSms, device_sms()), ceil_div(N, hl::kBm));
    const size_t smem = hl::narrow_smem(g.stages * g.stage_bytes, g.w_bytes);
    auto k = l->in <= 64 ? (vectors ? hl::narrow_backward_kernel<T, 1, true> : hl::narrow_backward_kernel<T, 1, false>)
                         : (vectors ? hl::narrow_backward_kernel<T, 2, true> : hl::narrow_backward_kernel<T, 2, false>);
    if (int rc = prepare_smem_once(k, smem)) return rc;
    *blocks_out = blocks;
    return launch_after(k, dim3((unsigned)blocks), hl::kNarrowThreads, smem, 1, s, what, g);
}

size_t forward_work(const hashgrid_linear_s* l, int64_t N, int64_t ldx) {
    return (l->in % 8 != 0 && l->out > 1 ? realigned_bytes(l->out, l->in) : 0) + (ldx % 8 != 0 && N > 1 ? realigned_bytes(N, l->in) : 0);
}

template <typename T>
int launch_linear_forward(const hashgrid_linear_s* l, const void* x, int64_t ldx, int64_t N, const void* w,
                          const hg::linear::Epilogue& e, char* work, int* status, cudaStream_t s) {
    static const char* what = "linear_forward";
    Array A{x, N, l->in, ldx, false, hg::kChkX}, B{w, l->out, l->in, l->in, false, hg::kChkWeights};
    Array* both[2] = {&A, &B};
    hg::linear::RealignList copies;
    add_copies(copies, both, 2, work);
    hg::linear::Slope none = {};
    if (int rc = launch_prepare<T>(none, false, copies, what, s)) return rc;
    return launch_gemm<T>(A, B, N, l->out, l->in, e, make_plan(N, l->out, l->in, e.out_f32 != 0, device_sms()), status, what, s);
}

template <typename T>
int launch_linear_backward(const hashgrid_linear_s* l, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                           int64_t N, const void* w, const void* z, void* dx, int64_t lddx, int dx_dtype, void* dw,
                           int dw_dtype, float* db, char* work, int* status, cudaStream_t s) {
    static const char* what = "linear_backward";
    namespace hl = hg::linear;
    const LinearWork lw = linear_work(l, N, lddy, ldx);
    Array dz{dy, N, l->out, lddy, false, hg::kChkDout};
    Array W{w, l->out, l->in, l->in, true, hg::kChkWeights}, X{x, N, l->in, ldx, true, hg::kChkX};
    const bool plain = l->act == HASHGRID_ACT_NONE, vectors = aligned_rows(dz) && (plain || l->out % 8 == 0);
    // A narrow layer's kernel makes dz and db itself where TMA can read dy and z.
    const bool narrow = dw != nullptr && narrow_layer(l, N), inside = narrow && vectors;
    const bool convert = !inside && (!plain || !aligned_rows(dz)) && (dx != nullptr || dw != nullptr);
    const int pieces = dz_pieces(l);
    const Array low{work + lw.low, N, l->out, lw.lddz, false, hg::kChkWork};
    Array* list[2] = {};
    int n = 0;
    if (dx != nullptr) list[n++] = &W;
    if (dw != nullptr) list[n++] = &X;
    hl::RealignList copies;
    add_copies(copies, list, n, work);
    hl::Sums sums[2];
    int nsums = 0;
    hl::Slope slope = {};
    if (convert || (db != nullptr && !inside)) {
        slope.dy.p = dy;
        slope.dy.bytes = strided_bytes(N, l->out, lddy, 2);
        slope.dy.ld = lddy;
        slope.dy.inner = l->out;
        slope.dy.role = hg::kChkDout;
        slope.z = slope.dy;
        slope.z.p = z;
        slope.z.bytes = strided_bytes(N, l->out, l->out, 2);
        slope.z.ld = l->out;
        slope.z.role = hg::kChkZ;
        slope.rows = N;
        slope.lddz = lw.lddz;
        slope.cols = l->out;
        slope.act = l->act;
        slope.dz = convert ? work + lw.dz : nullptr;
        slope.low = convert && pieces == 2 ? work + lw.low : nullptr;
        slope.sums = db == nullptr ? nullptr : lw.shares > 1 ? reinterpret_cast<float*>(work + lw.sums) : db;
        slope.role = lw.shares > 1 ? hg::kChkWork : hg::kChkBias;
        slope.groups = 1;
        while (slope.groups < 8 && slope.groups * 8 < l->out) slope.groups *= 2;
        slope.col_blocks = ceil_div(l->out, 64);
        slope.shares = lw.shares;
        if (convert) dz = Array{slope.dz, N, l->out, lw.lddz, false, hg::kChkWork};
        if (db != nullptr && lw.shares > 1) sums[nsums++] = hl::Sums{slope.sums, l->out, l->out, lw.shares, 0, db, hg::kChkBias};
    }
    if (int rc = launch_prepare<T>(slope, vectors && l->out % 8 == 0, copies, what, s)) return rc;
    const int64_t nw = (int64_t)l->in * l->out;
    float* out = reinterpret_cast<float*>(work + lw.dw);
    if (narrow) {
        int blocks = 0;
        const Array Z{z, N, l->out, l->out, false, hg::kChkZ};
        if (int rc = launch_narrow_backward<T>(l, inside ? l->act : (int)HASHGRID_ACT_NONE, pieces, dz, X, N, W, inside ? Z : low, dx, lddx, dx_dtype,
                                               inside && db != nullptr, out, &blocks, status, what, s))
            return rc;
        sums[nsums++] = hl::Sums{out, nw + l->out, nw, blocks, dw_dtype == HASHGRID_F32 ? 0 : 1, dw, hg::kChkGrad};
        if (inside && db != nullptr) sums[nsums++] = hl::Sums{out + nw, nw + l->out, l->out, blocks, 0, db, hg::kChkBias};
        return launch_sums<T>(sums, nsums, what, s);
    }
    // dx and dW do not depend on each other: where both are cut alike, and dW's sums are short, they share a
    // launch. dW is cut into parts of the rows that the sums kernel adds where its tiles are few.
    constexpr bool half = std::is_same<T, __half>::value;
    const int sms = device_sms();
    // A product that the tensor cores bound (by pairs), with a 16-bit result, takes dz's high part alone: the result's own
    // rounding is as large, and both parts take twice as long (8192 x 2048 -> 4096, GELU, fp32 dW: 441 us with both parts in both
    // products, 345 with the high one alone in dx).
    auto plan_of = [&](int64_t rows, int64_t cols, int64_t k, bool f32, bool& both) {
        const Plan one = make_plan(rows, cols, k, f32, sms);
        both = pieces == 2 && (f32 || !one.pair);
        return both ? make_plan(rows, cols, 2 * k, f32, sms) : one;
    };
    bool both_x = false, both_w = false;
    Plan px = plan_of(N, l->in, l->out, dx_dtype == HASHGRID_F32, both_x), pw = plan_of(l->out, l->in, N, dw_dtype == HASHGRID_F32, both_w);
    both_w = both_w || (pieces == 2 && lw.splits > 1);
    if (lw.splits > 1) pw = Plan{wide_tile(l->in, 128), 1, lw.splits, false};
    // Up to 16 steps of K one block takes for itself: sharing a launch saves more than splitting K does.
    const bool short_x = ceil_div(l->out, hl::kBk) <= 16, short_w = ceil_div(N, hl::kBk) <= 16 || lw.splits > 1;
    if (short_x && short_w && !px.pair && !pw.pair) px.cluster = pw.cluster = 1;
    const hl::Epilogue ex{nullptr, nullptr, dx, nullptr, 0, lddx, 0, dx_dtype == HASHGRID_F32, hl::kNoAct, hg::kChkOut};
    const bool parts = pw.splits > 1;
    const hl::Epilogue ew{nullptr, nullptr, parts ? out : dw, nullptr, 0, l->in, 0, parts || dw_dtype == HASHGRID_F32,
                          hl::kNoAct, parts ? hg::kChkWork : hg::kChkGrad};
    Product p[2];
    int np = 0;
    Array dzt = dz, lowt = low;
    dzt.mn = lowt.mn = true;
    if (dw != nullptr)
        if (int rc = set_product(p[np++], half, dzt, both_w ? &lowt : nullptr, X, l->out, l->in, N, ew, pw, status, what)) return rc;
    if (dx != nullptr)
        if (int rc = set_product(p[np++], half, dz, both_x ? &low : nullptr, W, N, l->in, l->out, ex, px, status, what)) return rc;
    if (np == 2 && px.pair == pw.pair && px.cluster == pw.cluster && p[0].gather == p[1].gather) {
        if (int rc = launch_products<T>(p, 2, px, what, s)) return rc;
    } else {
        for (int i = 0; i < np; ++i)
            if (int rc = launch_products<T>(&p[i], 1, dw != nullptr && i == 0 ? pw : px, what, s)) return rc;
    }
    if (dw != nullptr && parts) sums[nsums++] = hl::Sums{out, nw, nw, lw.splits, dw_dtype == HASHGRID_F32 ? 0 : 1, dw, hg::kChkGrad};
    return launch_sums<T>(sums, nsums, what, s);
}

int adamw_bytes(int dtype) { return dtype == HASHGRID_F32 ? 4 : dtype == HASHGRID_E4M3 ? 1 : 2; }

bool float_type(int dtype) { return dtype == HASHGRID_F32 || dtype == HASHGRID_F16 || dtype == HASHGRID_BF16; }

// Checks one tensor of an AdamW list.
int check_adamw_tensor(const hashgrid_adamw_tensor& t, int k) {
    char name[64];
    if (t.n < 0 || t.n >= ((int64_t)1 << 38)) return fail(HASHGRID_ERR_ARG, "tensor %d: n = %lld outside [0, 2^38)", k, (long long)t.n);
    if (!float_type(t.param_dtype) || !float_type(t.grad_dtype))
        return fail(HASHGRID_ERR_ARG, "tensor %d: param_dtype %d and grad_dtype %d must be HASHGRID_F32, _F16 or _BF16", k, t.param_dtype, t.grad_dtype);
    if (t.state_dtype != HASHGRID_F32 && t.state_dtype != HASHGRID_E4M3)
        return fail(HASHGRID_ERR_ARG, "tensor %d: state_dtype %d is neither HASHGRID_F32 nor HASHGRID_E4M3", k, t.state_dtype);
    if (t.copy != nullptr && t.copy_dtype != HASHGRID_F16 && t.copy_dtype != HASHGRID_BF16)
        return fail(HASHGRID_ERR_ARG, "tensor %d: copy_dtype %d is neither HASHGRID_F16 nor HASHGRID_BF16", k, t.copy_dtype);
    if (!std::isfinite(t.lr_scale) || !std::isfinite(t.weight_decay) || t.weight_decay < 0.f)
        return fail(HASHGRID_ERR_ARG, "tensor %d: lr_scale %g and weight_decay %g must be finite, weight_decay >= 0", k, t.lr_scale, t.weight_decay);
    const bool coded = t.state_dtype == HASHGRID_E4M3;
    if (!coded && (t.m_scale != nullptr || t.v_scale != nullptr))
        return fail(HASHGRID_ERR_ARG, "tensor %d: fp32 states have no scales", k);
    if (t.n == 0) return ok();
    const size_t n = (size_t)t.n, scales = (n + HASHGRID_ADAMW_BLOCK - 1) / HASHGRID_ADAMW_BLOCK * sizeof(float);
    struct { const void* p; size_t bytes; const char* what; size_t align; bool need; } arrays[] = {
        {t.param, n * adamw_bytes(t.param_dtype), "param", 16, true},
        {t.grad, n * adamw_bytes(t.grad_dtype), "grad", 16, true},
        {t.m, n * adamw_bytes(t.state_dtype), "m", 16, true},
        {t.v, n * adamw_bytes(t.state_dtype), "v", 16, true},
        {t.m_scale, scales, "m_scale", 4, coded},
        {t.v_scale, scales, "v_scale", 4, coded},
        {t.copy, n * 2, "copy", 16, t.copy != nullptr},
    };
    for (const auto& a : arrays) {
        if (!a.need) continue;
        snprintf(name, sizeof name, "tensor %d: %s", k, a.what);
        if (int rc = check_buffer(a.p, a.bytes, name, a.align)) return rc;
    }
    return ok();
}

// No two arrays of a list may share bytes: the kernel's warps run in no order.
int check_adamw_overlap(const hashgrid_adamw_tensor* tensors, int count) {
    struct Range { uintptr_t lo, hi; int k; };
    std::vector<Range> r;
    for (int k = 0; k < count; ++k) {
        const hashgrid_adamw_tensor& t = tensors[k];
        const size_t n = (size_t)t.n, scales = (n + HASHGRID_ADAMW_BLOCK - 1) / HASHGRID_ADAMW_BLOCK * sizeof(float);
        auto add = [&](const void* p, size_t bytes) {
            if (p != nullptr && bytes != 0) r.push_back({(uintptr_t)p, (uintptr_t)p + bytes, k});
        };
        add(t.param, n * adamw_bytes(t.param_dtype));
        add(t.grad, n * adamw_bytes(t.grad_dtype));
        add(t.m, n * adamw_bytes(t.state_dtype));
        add(t.v, n * adamw_bytes(t.state_dtype));
        add(t.m_scale, scales);
        add(t.v_scale, scales);
        add(t.copy, n * 2);
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    for (size_t i = 1; i < r.size(); ++i)
        if (r[i].lo < r[i - 1].hi)
            return fail(HASHGRID_ERR_ARG, "arrays of tensors %d and %d overlap", r[i - 1].k, r[i].k);
    return ok();
}

template <int kCap>
int launch_adamw(const hashgrid_adamw_s* o, const hashgrid_adamw_s::Launch& l, hg::adamw::Params a, cudaStream_t s) {
    hg::adamw::List<kCap> list;
    list.count = (uint32_t)l.count;
    list.blocks = l.blocks;
    list.where = l.where;
    std::memcpy(list.t, o->tensors.data() + l.begin, sizeof(hg::adamw::Tensor) * l.count);
    std::memcpy(list.first, o->first.data() + l.begin, sizeof(uint32_t) * l.count);
    for (int i = 0; i < l.count; ++i) {
        const float lr_scale = list.t[i].rate, decay = list.t[i].keep;
        list.t[i].rate = lr_scale * a.lr;
        list.t[i].keep = (float)(1.0 - (double)lr_scale * (double)a.lr * (double)decay);
    }
    const unsigned blocks = (l.blocks + hg::adamw::kWarps - 1) / hg::adamw::kWarps;
    return launch_after(hg::adamw::step_kernel<kCap>, dim3(blocks), 32 * hg::adamw::kWarps, 0, 1, s, "adamw_step", list, a);
}

}  // namespace

extern "C" {

int hashgrid_create(int L, int F, int log2T, int N_min, int N_max, int dtype, hashgrid_t* out) {
    if (out == nullptr) return fail(HASHGRID_ERR_ARG, "out handle pointer is NULL");
    *out = nullptr;
    if (L < 1 || L > HASHGRID_MAX_LEVELS)
        return fail(HASHGRID_ERR_ARG, "L = %d outside [1, %d]", L, HASHGRID_MAX_LEVELS);
    if (F != 1 && F != 2 && F != 4 && F != 8)
        return fail(HASHGRID_ERR_ARG, "F = %d not in {1, 2, 4, 8}", F);
    if (log2T < HASHGRID_MIN_LOG2T || log2T > HASHGRID_MAX_LOG2T)
        return fail(HASHGRID_ERR_ARG, "log2T = %d outside [%d, %d]", log2T, HASHGRID_MIN_LOG2T,
                    HASHGRID_MAX_LOG2T);
    if (N_min < 1 || N_max < N_min || N_max > HASHGRID_MAX_RESOLUTION)
        return fail(HASHGRID_ERR_ARG, "resolutions N_min = %d, N_max = %d outside 1 <= N_min <= N_max <= %d",
                    N_min, N_max, HASHGRID_MAX_RESOLUTION);
    if (dtype != HASHGRID_F32 && dtype != HASHGRID_F16)
        return fail(HASHGRID_ERR_ARG, "dtype = %d is neither HASHGRID_F32 nor HASHGRID_F16", dtype);
    if (L == 1 && N_min != N_max)
        return fail(HASHGRID_ERR_ARG, "L = 1 needs N_min == N_max (the growth factor divides by L - 1)");
    hashgrid_s* h = new (std::nothrow) hashgrid_s;
    if (h == nullptr) return fail(HASHGRID_ERR_OOM, "out of host memory");
    std::memset(h, 0, sizeof(*h));
    h->D = 3;
    h->L = L; h->F = F; h->log2T = log2T; h->N_min = N_min; h->N_max = N_max; h->dtype = dtype;
    compute_resolutions(L, N_min, N_max, h->res);
    h->lp.L = L;
    h->lp.T = (uint64_t)1 << log2T;
    h->lp.mask = (uint32_t)(h->lp.T - 1);
    for (int l = 0; l < L; ++l) h->lp.scale[l] = (float)h->res[l];
    compute_level_groups(h);
    *out = h;
    return ok();
}

int hashgrid_create_nd(int D, int L, int F, int log2T, int N_min, int N_max, int dtype, hashgrid_t* out) {
    if (out != nullptr) *out = nullptr;
    if (D != 2 && D != 3 && D != 4) return fail(HASHGRID_ERR_ARG, "D = %d is not 2, 3 or 4", D);
    int rc = hashgrid_create(L, F, log2T, N_min, N_max, dtype, out);
    if (rc == HASHGRID_OK) (*out)->D = D;
    return rc;
}

int hashgrid_dims(hashgrid_t h) { return h == nullptr ? 0 : h->D; }

int hashgrid_destroy(hashgrid_t h) {
    delete h;
    return ok();
}

int hashgrid_resolutions(hashgrid_t h, int* res_out) {
    if (int rc = check_handle(h)) return rc;
    if (res_out == nullptr) return fail(HASHGRID_ERR_ARG, "res_out is NULL");
    std::memcpy(res_out, h->res, sizeof(int) * h->L);
    return ok();
}

size_t hashgrid_table_elems(hashgrid_t h) {
    if (h == nullptr) return 0;
    return (size_t)h->L * ((size_t)1 << h->log2T) * (size_t)h->F;
}

int hashgrid_output_width(hashgrid_t h) { return h == nullptr ? 0 : h->L * h->F; }

int hashgrid_set_option(hashgrid_t h, int option, int value) {
    if (int rc = check_handle(h)) return rc;
    switch (option) {
        case HASHGRID_OPT_FORWARD_GATHER:
            if (value < HASHGRID_GATHER_AUTO || value > HASHGRID_GATHER_LANES)
                return fail(HASHGRID_ERR_ARG, "forward gather mode %d is not a HASHGRID_GATHER_* value", value);
            h->forward_gather = value;
            return ok();
        case HASHGRID_OPT_SCHEDULE:
            if (value < HASHGRID_SCHEDULE_AUTO || value > HASHGRID_SCHEDULE_LEVEL_MAJOR)
                return fail(HASHGRID_ERR_ARG, "schedule %d is not a HASHGRID_SCHEDULE_* value", value);
            h->schedule = value;
            return ok();
        case HASHGRID_OPT_BACKWARD_MODE:
            if (value < HASHGRID_BACKWARD_AUTO || value > HASHGRID_BACKWARD_RUN_LANES)
                return fail(HASHGRID_ERR_ARG, "backward mode %d is not a HASHGRID_BACKWARD_* value", value);
            if ((value == HASHGRID_BACKWARD_WARP_DEDUP || value == HASHGRID_BACKWARD_RUN_MERGE ||
                 value == HASHGRID_BACKWARD_WARP_DEDUP_ADAPTIVE || value == HASHGRID_BACKWARD_RUN_LANES) && h->F > 4)
                return fail(HASHGRID_ERR_ARG, "backward mode %d needs F <= 4, F = %d", value, h->F);
            h->backward_mode = value;
            return ok();
    }
    return fail(HASHGRID_ERR_ARG, "unknown option %d", option);
}

int hashgrid_get_option(hashgrid_t h, int option, int* value) {
    if (int rc = check_handle(h)) return rc;
    if (value == nullptr) return fail(HASHGRID_ERR_ARG, "value is NULL");
    switch (option) {
        case HASHGRID_OPT_FORWARD_GATHER: *value = h->forward_gather; return ok();
        case HASHGRID_OPT_BACKWARD_MODE: *value = h->backward_mode; return ok();
        case HASHGRID_OPT_SCHEDULE: *value = h->schedule; return ok();
    }
    return fail(HASHGRID_ERR_ARG, "unknown option %d", option);
}

int hashgrid_params(hashgrid_t h, int* L, int* F, int* log2T, int* N_min, int* N_max, int* dtype) {
    if (int rc = check_handle(h)) return rc;
    if (L) *L = h->L;
    if (F) *F = h->F;
    if (log2T) *log2T = h->log2T;
    if (N_min) *N_min = h->N_min;
    if (N_max) *N_max = h->N_max;
    if (dtype) *dtype = h->dtype;
    return ok();
}

int hashgrid_forward(hashgrid_t h, const float* x, int64_t N, const void* table, float* out,
                     void* cuda_stream) {
    if (int rc = check_handle(h)) return rc;
    if (int rc = check_N(N, kTile)) return rc;
    if (N == 0) return ok();
    const size_t W = (size_t)h->L * h->F;
    if (int rc = check_buffer(x, (size_t)N * h->D * sizeof(float), "x")) return rc;
    if (int rc = check_buffer(table, table_bytes(h), "table")) return rc;
    if (int rc = check_buffer(out, (size_t)N * W * sizeof(float), "out")) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return run_checked(s, {{hg::kChkX, x, (size_t)N * h->D * sizeof(float)}, {hg::kChkTable, table, table_bytes(h)},
                           {hg::kChkOut, out, (size_t)N * W * sizeof(float)}},
                       "forward", [&]() -> int {
    const bool half = h->dtype == HASHGRID_F16;
    if (h->D != 3)
        return nd_dispatch(h, [&](auto d, auto f) {
            return half ? launch_nd_forward<decltype(d)::value, decltype(f)::value, __half>(h, x, N, table, out, s)
                        : launch_nd_forward<decltype(d)::value, decltype(f)::value, float>(h, x, N, table, out, s);
        });
    // Sector gathers issue 256-bit loads, which need a 32-byte-aligned table.
    const bool aligned32 = reinterpret_cast<uintptr_t>(table) % 32 == 0;
    if (h->forward_gather == HASHGRID_GATHER_SECTOR && !aligned32)
        return fail(HASHGRID_ERR_ALIGN, "sector gathers need a 32-byte-aligned table (%p)", table);
    const int sector = forward_gather_kernel(h);
    if (level_major(h)) {
        const int lg = sector == hg::kGatherLanes ? hg::kGatherLanes : hg::kGatherCorner;
        switch (h->F) {
            case 1: return half ? launch_forward_levels<1, __half>(h, x, N, table, out, lg, s) : launch_forward_levels<1, float>(h, x, N, table, out, lg, s);
            case 2: return half ? launch_forward_levels<2, __half>(h, x, N, table, out, lg, s) : launch_forward_levels<2, float>(h, x, N, table, out, lg, s);
            case 4: return half ? launch_forward_levels<4, __half>(h, x, N, table, out, lg, s) : launch_forward_levels<4, float>(h, x, N, table, out, lg, s);
            case 8: return half ? launch_forward_levels<8, __half>(h, x, N, table, out, lg, s) : launch_forward_levels<8, float>(h, x, N, table, out, lg, s);
        }
    }
    switch (h->F) {
        case 1: return half ? launch_forward<1, __half>(h, x, N, table, out, sector, s) : launch_forward<1, float>(h, x, N, table, out, sector, s);
        case 2: return half ? launch_forward<2, __half>(h, x, N, table, out, sector, s) : launch_forward<2, float>(h, x, N, table, out, sector, s);
        case 4: return half ? launch_forward<4, __half>(h, x, N, table, out, sector, s) : launch_forward<4, float>(h, x, N, table, out, sector, s);
        case 8: return half ? launch_forward<8, __half>(h, x, N, table, out, sector, s) : launch_forward<8, float>(h, x, N, table, out, sector, s);
    }
    return fail(HASHGRID_ERR_ARG, "corrupt handle");
    });
}

int hashgrid_backward(hashgrid_t h, const float* x, const float* dL_dout, int64_t N, float* dL_dtable,
                      void* cuda_stream) {
    if (int rc = check_handle(h)) return rc;
    if (int rc = check_N(N, kTile)) return rc;
    if (N == 0) return ok();
    const size_t W = (size_t)h->L * h->F;
    if (int rc = check_buffer(x, (size_t)N * h->D * sizeof(float), "x")) return rc;
    if (int rc = check_buffer(dL_dout, (size_t)N * W * sizeof(float), "dL_dout")) return rc;
    if (int rc = check_buffer(dL_dtable, hashgrid_table_elems(h) * sizeof(float), "dL_dtable")) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return run_checked(s, {{hg::kChkX, x, (size_t)N * h->D * sizeof(float)}, {hg::kChkDout, dL_dout, (size_t)N * W * sizeof(float)},
                           {hg::kChkGrad, dL_dtable, hashgrid_table_elems(h) * sizeof(float)}},
                       "backward", [&]() -> int {
    if (h->D != 3)
        return nd_dispatch(h, [&](auto d, auto f) {
            return launch_nd_backward<decltype(d)::value, decltype(f)::value, float>(h, x, dL_dout, N, dL_dtable, s);
        });
    switch (h->F) {
        case 1: return launch_backward<1>(h, x, dL_dout, N, dL_dtable, s);
        case 2: return launch_backward<2>(h, x, dL_dout, N, dL_dtable, s);
        case 4: return launch_backward<4>(h, x, dL_dout, N, dL_dtable, s);
        case 8: return launch_backward<8>(h, x, dL_dout, N, dL_dtable, s);
    }
    return fail(HASHGRID_ERR_ARG, "corrupt handle");
    });
}

int hashgrid_backward_half(hashgrid_t h, const float* x, const float* dL_dout, int64_t N, void* dL_dtable,
                           void* cuda_stream) {
    if (int rc = check_handle(h)) return rc;
    if (int rc = check_N(N, kTile)) return rc;
    if (N == 0) return ok();
    const size_t W = (size_t)h->L * h->F;
    if (int rc = check_buffer(x, (size_t)N * h->D * sizeof(float), "x")) return rc;
    if (int rc = check_buffer(dL_dout, (size_t)N * W * sizeof(float), "dL_dout")) return rc;
    if (int rc = check_buffer(dL_dtable, hashgrid_table_elems(h) * 2, "dL_dtable")) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    __half* d = static_cast<__half*>(dL_dtable);
    return run_checked(s, {{hg::kChkX, x, (size_t)N * h->D * sizeof(float)}, {hg::kChkDout, dL_dout, (size_t)N * W * sizeof(float)},
                           {hg::kChkGrad, dL_dtable, hashgrid_table_elems(h) * 2}},
                       "backward_half", [&]() -> int {
    if (h->D != 3)
        return nd_dispatch(h, [&](auto dd, auto f) {
            return launch_nd_backward<decltype(dd)::value, decltype(f)::value, __half>(h, x, dL_dout, N, d, s);
        });
    switch (h->F) {
        case 1: return launch_backward_half<1>(h, x, dL_dout, N, d, s);
        case 2: return launch_backward_half<2>(h, x, dL_dout, N, d, s);
        case 4: return launch_backward_half<4>(h, x, dL_dout, N, d, s);
        case 8: return launch_backward_half<8>(h, x, dL_dout, N, d, s);
    }
    return fail(HASHGRID_ERR_ARG, "corrupt handle");
    });
}

int hashgrid_backward_input(hashgrid_t h, const float* x, const float* dL_dout, int64_t N, const void* table,
                            float* dL_dx, void* cuda_stream) {
    if (int rc = check_handle(h)) return rc;
    if (int rc = check_N(N, kTile)) return rc;
    if (N == 0) return ok();
    const size_t W = (size_t)h->L * h->F;
    if (int rc = check_buffer(x, (size_t)N * h->D * sizeof(float), "x")) return rc;
    if (int rc = check_buffer(dL_dout, (size_t)N * W * sizeof(float), "dL_dout")) return rc;
    if (int rc = check_buffer(table, table_bytes(h), "table")) return rc;
    if (int rc = check_buffer(dL_dx, (size_t)N * h->D * sizeof(float), "dL_dx")) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return run_checked(s, {{hg::kChkX, x, (size_t)N * h->D * sizeof(float)}, {hg::kChkDout, dL_dout, (size_t)N * W * sizeof(float)},
                           {hg::kChkTable, table, table_bytes(h)}, {hg::kChkOut, dL_dx, (size_t)N * h->D * sizeof(float)}},
                       "backward_input", [&]() -> int {
    const bool half = h->dtype == HASHGRID_F16;
    if (h->D != 3)
        return nd_dispatch(h, [&](auto d, auto f) {
            constexpr int DD = decltype(d)::value, FF = decltype(f)::value;
            return half ? launch_nd_backward_input<DD, FF, __half>(h, x, dL_dout, N, table, dL_dx, s)
                        : launch_nd_backward_input<DD, FF, float>(h, x, dL_dout, N, table, dL_dx, s);
        });
    switch (h->F) {
        case 1: return half ? launch_backward_input<1, __half>(h, x, dL_dout, N, table, dL_dx, s) : launch_backward_input<1, float>(h, x, dL_dout, N, table, dL_dx, s);
        case 2: return half ? launch_backward_input<2, __half>(h, x, dL_dout, N, table, dL_dx, s) : launch_backward_input<2, float>(h, x, dL_dout, N, table, dL_dx, s);
        case 4: return half ? launch_backward_input<4, __half>(h, x, dL_dout, N, table, dL_dx, s) : launch_backward_input<4, float>(h, x, dL_dout, N, table, dL_dx, s);
        case 8: return half ? launch_backward_input<8, __half>(h, x, dL_dout, N, table, dL_dx, s) : launch_backward_input<8, float>(h, x, dL_dout, N, table, dL_dx, s);
    }
    return fail(HASHGRID_ERR_ARG, "corrupt handle");
    });
}

int hashgrid_adam_step(hashgrid_t h, void* table, float* adam_m, float* adam_v, float* dL_dtable, int64_t step,
                       float lr, float beta1, float beta2, float eps, int zero_grad, void* cuda_stream) {
    if (int rc = check_handle(h)) return rc;
    if (step < 1) return fail(HASHGRID_ERR_ARG, "step = %lld must be >= 1", (long long)step);
    if (!(beta1 >= 0.f && beta1 < 1.f) || !(beta2 >= 0.f && beta2 < 1.f))
        return fail(HASHGRID_ERR_ARG, "betas (%g, %g) must lie in [0, 1)", beta1, beta2);
    if (!(eps > 0.f) || !std::isfinite(eps) || !std::isfinite(lr))
        return fail(HASHGRID_ERR_ARG, "lr = %g and eps = %g must be finite, eps > 0", lr, eps);
    const size_t n = hashgrid_table_elems(h);
    if (int rc = check_buffer(table, table_bytes(h), "table")) return rc;
    if (int rc = check_buffer(adam_m, n * sizeof(float), "adam_m")) return rc;
    if (int rc = check_buffer(adam_v, n * sizeof(float), "adam_v")) return rc;
    if (int rc = check_buffer(dL_dtable, n * sizeof(float), "dL_dtable")) return rc;
    hg::AdamParams a;
    a.lr = lr;
    a.b1 = beta1;
    a.b2 = beta2;
    a.eps = eps;
    a.c1 = (float)(1.0 / (1.0 - std::pow((double)beta1, (double)step)));
    a.c2 = (float)(1.0 / (1.0 - std::pow((double)beta2, (double)step)));
    const int64_t n4 = (int64_t)(n / 4);  // L*T*F is a multiple of 16
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t want = (n4 + 255) / 256;
    const unsigned blocks = (unsigned)(want < (int64_t)sms * 16 ? want : (int64_t)sms * 16);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return run_checked(s, {{hg::kChkTable, table, table_bytes(h)}, {hg::kChkM, adam_m, n * sizeof(float)},
                           {hg::kChkV, adam_v, n * sizeof(float)}, {hg::kChkGrad, dL_dtable, n * sizeof(float)}},
                       "adam_step", [&]() -> int {
        if (h->dtype == HASHGRID_F16)
            hg::adam_kernel<__half><<<blocks, 256, 0, s>>>(static_cast<__half*>(table), adam_m, adam_v, dL_dtable, n4, a, zero_grad);
        else
            hg::adam_kernel<float><<<blocks, 256, 0, s>>>(static_cast<float*>(table), adam_m, adam_v, dL_dtable, n4, a, zero_grad);
        return launch_status("adam_step");
    });
}

int hashgrid_mlp_forward(hashgrid_t h, const float* x, int64_t N, const void* table, const void* w1,
                         const float* b1, const void* w2, const float* b2, const void* w3, const float* b3, float* y,
                         int* device_status, void* cuda_stream) {
    if (int rc = check_handle(h)) return rc;
    if (h->D != 3) return fail(HASHGRID_ERR_ARG, "the MLP takes 3-D points, the handle has D = %d", h->D);
    const int K1 = h->L * h->F;
    if (K1 % 16 != 0 || K1 > 64)
        return fail(HASHGRID_ERR_ARG, "the MLP needs L*F in {16, 32, 48, 64}, got %d", K1);
    if (int rc = check_N(N, hg::mlp::kM)) return rc;
    if (N == 0) return ok();
    using namespace hg::mlp;
    if (int rc = check_buffer(x, (size_t)N * h->D * sizeof(float), "x")) return rc;
    if (int rc = check_buffer(table, table_bytes(h), "table")) return rc;
    if (int rc = check_buffer(w1, (size_t)kHid * K1 * 2, "w1")) return rc;
    if (int rc = check_buffer(b1, kHid * sizeof(float), "b1")) return rc;
    if (int rc = check_buffer(w2, (size_t)kHid * kHid * 2, "w2")) return rc;
    if (int rc = check_buffer(b2, kHid * sizeof(float), "b2")) return rc;
    if (int rc = check_buffer(w3, (size_t)kOut * kHid * 2, "w3")) return rc;
    if (int rc = check_buffer(b3, kOut * sizeof(float), "b3")) return rc;
    if (int rc = check_buffer(y, (size_t)N * kOut * sizeof(float), "y")) return rc;
    if (device_status != nullptr)
        if (int rc = check_buffer(device_status, sizeof(int), "device_status")) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return run_checked(s, {{hg::kChkX, x, (size_t)N * h->D * sizeof(float)}, {hg::kChkTable, table, table_bytes(h)},
                           {hg::kChkOut, y, (size_t)N * kOut * sizeof(float)}},
                       "mlp_forward", [&]() -> int {
    const bool half = h->dtype == HASHGRID_F16;
    switch (h->F) {
        case 1: return half ? dispatch_mlp_forward<1, __half>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, device_status, s)
                            : dispatch_mlp_forward<1, float>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, device_status, s);
        case 2: return half ? dispatch_mlp_forward<2, __half>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, device_status, s)
                            : dispatch_mlp_forward<2, float>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, device_status, s);
        case 4: return half ? dispatch_mlp_forward<4, __half>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, device_status, s)
                            : dispatch_mlp_forward<4, float>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, device_status, s);
        case 8: return half ? dispatch_mlp_forward<8, __half>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, device_status, s)
                            : dispatch_mlp_forward<8, float>(h, x, N, table, w1, b1, w2, b2, w3, b3, y, device_status, s);
    }
    return fail(HASHGRID_ERR_ARG, "corrupt handle");
    });
}

int hashgrid_debug_indices(hashgrid_t h, const float* x, int64_t N, uint32_t* idx_out, void* cuda_stream) {
    if (int rc = check_handle(h)) return rc;
    if (int rc = check_N(N, 1)) return rc;
    if (N == 0) return ok();
    if (int rc = check_buffer(x, (size_t)N * h->D * sizeof(float), "x")) return rc;
    if (int rc = check_buffer(idx_out, (size_t)N * h->L * ((size_t)1 << h->D) * sizeof(uint32_t), "idx_out")) return rc;
    const int64_t total = N * h->L;
    const int threads = 256;
    const int64_t blocks = (total + threads - 1) / threads;
    if (blocks > 0x7fffffffLL) return fail(HASHGRID_ERR_ARG, "N too large for the index export");
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return run_checked(s, {{hg::kChkX, x, (size_t)N * h->D * sizeof(float)},
                           {hg::kChkOut, idx_out, (size_t)N * h->L * ((size_t)1 << h->D) * sizeof(uint32_t)}},
                       "debug_indices", [&]() -> int {
        if (h->D == 2)
            hg::nd::indices_kernel<2><<<(unsigned)blocks, threads, 0, s>>>(h->lp, x, N, idx_out);
        else if (h->D == 4)
            hg::nd::indices_kernel<4><<<(unsigned)blocks, threads, 0, s>>>(h->lp, x, N, idx_out);
        else
            hg::indices_kernel<<<(unsigned)blocks, threads, 0, s>>>(h->lp, x, N, idx_out);
        return launch_status("debug_indices");
    });
}

int hashgrid_linear_status(void) { return check_given_up(); }

int hashgrid_debug_wait_limit(int64_t polls) {
    g_wait_limit.store(polls, std::memory_order_relaxed);
    return ok();
}

int hashgrid_linear_create(int in, int out, int dtype, int activation, hashgrid_linear_t* layer) {
    if (layer == nullptr) return fail(HASHGRID_ERR_ARG, "layer handle pointer is NULL");
    *layer = nullptr;
    if (in < 1 || in > HASHGRID_MAX_WIDTH || out < 1 || out > HASHGRID_MAX_WIDTH)
        return fail(HASHGRID_ERR_ARG, "in = %d and out = %d must lie in [1, %d]", in, out, HASHGRID_MAX_WIDTH);
    if (dtype != HASHGRID_F16 && dtype != HASHGRID_BF16)
        return fail(HASHGRID_ERR_ARG, "dtype = %d is neither HASHGRID_F16 nor HASHGRID_BF16", dtype);
    if (activation < HASHGRID_ACT_NONE || activation > HASHGRID_ACT_SILU)
        return fail(HASHGRID_ERR_ARG, "activation = %d is not a HASHGRID_ACT_* value", activation);
    hashgrid_linear_s* l = new (std::nothrow) hashgrid_linear_s;
    if (l == nullptr) return fail(HASHGRID_ERR_OOM, "out of host memory");
    l->in = in;
    l->out = out;
    l->dtype = dtype;
    l->act = activation;
    *layer = l;
    return ok();
}

int hashgrid_linear_destroy(hashgrid_linear_t layer) {
    delete layer;
    return ok();
}

int hashgrid_linear_params(hashgrid_linear_t l, int* in, int* out, int* dtype, int* activation) {
    if (int rc = check_layer(l)) return rc;
    if (in) *in = l->in;
    if (out) *out = l->out;
    if (dtype) *dtype = l->dtype;
    if (activation) *activation = l->act;
    return ok();
}

int hashgrid_linear_forward(hashgrid_linear_t l, const void* x, int64_t ldx, int64_t N, const void* w, const float* b,
                            const void* residual, int64_t ldr, void* y, int64_t ldy, int y_dtype, void* z,
                            void* workspace, size_t workspace_bytes, int* device_status, void* cuda_stream) {
    if (int rc = check_layer(l)) return rc;
    if (int rc = check_row_count(N)) return rc;
    if (int rc = check_out_type(l, y_dtype, "y_dtype")) return rc;
    if (N == 0) return ok();
    const size_t ys = y_dtype == HASHGRID_F32 ? 4 : 2;
    if (int rc = check_rows(x, N, l->in, ldx, 2, "x")) return rc;
    if (int rc = check_buffer(w, (size_t)l->in * l->out * 2, "w")) return rc;
    if (b != nullptr)
        if (int rc = check_buffer(b, (size_t)l->out * sizeof(float), "b")) return rc;
    if (residual != nullptr)
        if (int rc = check_rows(residual, N, l->out, ldr, ys, "residual")) return rc;
    if (int rc = check_rows(y, N, l->out, ldy, ys, "y")) return rc;
    if (z != nullptr)
        if (int rc = check_buffer(z, (size_t)N * l->out * 2, "z")) return rc;
    const size_t need = forward_work(l, N, ldx);
    if (int rc = check_workspace(workspace, workspace_bytes, need, N)) return rc;
    if (device_status != nullptr)
        if (int rc = check_buffer(device_status, sizeof(int), "device_status")) return rc;
    const bool in_place = residual == y && (ldr == ldy || N == 1);
    if (int rc = check_apart({region("y", y, N, l->out, ldy, ys), region("z", z, N, l->out, l->out, 2), region("workspace", workspace, need),
                              region("device_status", device_status, sizeof(int))},
                             {region("x", x, N, l->in, ldx, 2), region("w", w, l->out, l->in, l->in, 2), region("b", b, 1, l->out, l->out, 4),
                              region("residual", in_place ? nullptr : residual, N, l->out, ldr, ys)}))
        return rc;
    if (int rc = check_given_up()) return rc;
    device_status = status_word(device_status);
    const hg::linear::Epilogue e{b, residual, y, z, ldr, ldy, l->out, y_dtype == HASHGRID_F32, l->act, hg::kChkOut};
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return run_checked(s, {{hg::kChkX, x, strided_bytes(N, l->in, ldx, 2)}, {hg::kChkWeights, w, (size_t)l->in * l->out * 2},
                           {hg::kChkBias, b, (size_t)l->out * sizeof(float)}, {hg::kChkResidual, residual, strided_bytes(N, l->out, ldr, ys)},
                           {hg::kChkOut, y, strided_bytes(N, l->out, ldy, ys)}, {hg::kChkZ, z, (size_t)N * l->out * 2},
                           {hg::kChkWork, workspace, need}},
                       "linear_forward", [&]() -> int {
        char* ws = static_cast<char*>(workspace);
        return l->dtype == HASHGRID_F16 ? launch_linear_forward<__half>(l, x, ldx, N, w, e, ws, device_status, s)
                                        : launch_linear_forward<__nv_bfloat16>(l, x, ldx, N, w, e, ws, device_status, s);
    });
}

size_t hashgrid_linear_forward_workspace(hashgrid_linear_t layer, int64_t N, int64_t ldx) {
    if (layer == nullptr || N < 1 || N >= kMaxRows) return 0;
    return forward_work(layer, N, ldx);
}

size_t hashgrid_linear_backward_workspace(hashgrid_linear_t layer, int64_t N, int64_t lddy, int64_t ldx) {
    if (layer == nullptr || N < 1 || N >= kMaxRows) return 0;
    return linear_work(layer, N, lddy, ldx).bytes;
}

int hashgrid_linear_backward(hashgrid_linear_t l, const void* dL_dy, int64_t lddy, const void* x, int64_t ldx, int64_t N,
                             const void* w, const void* z, void* dL_dx, int64_t lddx, int dx_dtype, void* dL_dw,
                             int dw_dtype, float* dL_db, void* workspace, size_t workspace_bytes, int* device_status,
                             void* cuda_stream) {
    if (int rc = check_layer(l)) return rc;
    if (int rc = check_row_count(N)) return rc;
    if (int rc = check_out_type(l, dx_dtype, "dx_dtype")) return rc;
    if (int rc = check_out_type(l, dw_dtype, "dw_dtype")) return rc;
    const size_t xs = dx_dtype == HASHGRID_F32 ? 4 : 2, wb = (size_t)l->in * l->out * (dw_dtype == HASHGRID_F32 ? 4 : 2);
    const size_t bb = (size_t)l->out * sizeof(float);
    if (dL_dw != nullptr)
        if (int rc = check_buffer(dL_dw, wb, "dL_dw")) return rc;
    if (dL_db != nullptr)
        if (int rc = check_buffer(dL_db, bb, "dL_db")) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    if (N == 0) {
        if (dL_dw != nullptr && cudaMemsetAsync(dL_dw, 0, wb, s) != cudaSuccess) return launch_status("linear_backward");
        if (dL_db != nullptr && cudaMemsetAsync(dL_db, 0, bb, s) != cudaSuccess) return launch_status("linear_backward");
        return ok();
    }
    if (dL_dx == nullptr && dL_dw == nullptr && dL_db == nullptr) return ok();
    if (int rc = check_rows(dL_dy, N, l->out, lddy, 2, "dL_dy")) return rc;
    if (dL_dw != nullptr)
        if (int rc = check_rows(x, N, l->in, ldx, 2, "x")) return rc;
    if (dL_dx != nullptr) {
        if (int rc = check_buffer(w, (size_t)l->in * l->out * 2, "w")) return rc;
        if (int rc = check_rows(dL_dx, N, l->in, lddx, xs, "dL_dx")) return rc;
    }
    if (l->act != HASHGRID_ACT_NONE)
        if (int rc = check_buffer(z, (size_t)N * l->out * 2, "z")) return rc;
    const size_t need = linear_work(l, N, lddy, ldx).bytes;
    if (int rc = check_workspace(workspace, workspace_bytes, need, N)) return rc;
    if (device_status != nullptr)
        if (int rc = check_buffer(device_status, sizeof(int), "device_status")) return rc;
    if (int rc = check_apart({region("dL_dx", dL_dx, N, l->in, lddx, xs), region("dL_dw", dL_dw, wb), region("dL_db", dL_db, bb),
                              region("workspace", workspace, need), region("device_status", device_status, sizeof(int))},
                             {region("dL_dy", dL_dy, N, l->out, lddy, 2), region("x", dL_dw != nullptr ? x : nullptr, N, l->in, ldx, 2),
                              region("w", dL_dx != nullptr ? w : nullptr, l->out, l->in, l->in, 2),
                              region("z", l->act != HASHGRID_ACT_NONE ? z : nullptr, N, l->out, l->out, 2)}))
        return rc;
    if (int rc = check_given_up()) return rc;
    device_status = status_word(device_status);
    return run_checked(s, {{hg::kChkX, x, strided_bytes(N, l->in, ldx, 2)}, {hg::kChkWeights, w, (size_t)l->in * l->out * 2},
                           {hg::kChkBias, dL_db, bb}, {hg::kChkDout, dL_dy, strided_bytes(N, l->out, lddy, 2)},
                           {hg::kChkZ, z, (size_t)N * l->out * 2}, {hg::kChkWork, workspace, need},
                           {hg::kChkOut, dL_dx, dL_dx ? strided_bytes(N, l->in, lddx, xs) : 0}, {hg::kChkGrad, dL_dw, wb}},
                       "linear_backward", [&]() -> int {
        char* ws = static_cast<char*>(workspace);
        return l->dtype == HASHGRID_F16
                   ? launch_linear_backward<__half>(l, dL_dy, lddy, x, ldx, N, w, z, dL_dx, lddx, dx_dtype, dL_dw, dw_dtype, dL_db, ws, device_status, s)
                   : launch_linear_backward<__nv_bfloat16>(l, dL_dy, lddy, x, ldx, N, w, z, dL_dx, lddx, dx_dtype, dL_dw, dw_dtype, dL_db, ws, device_status, s);
    });
}

int hashgrid_adamw_create(const hashgrid_adamw_tensor* tensors, int count, hashgrid_adamw_t* opt) {
    if (opt == nullptr) return fail(HASHGRID_ERR_ARG, "optimiser handle pointer is NULL");
    *opt = nullptr;
    if (tensors == nullptr) return fail(HASHGRID_ERR_ARG, "tensors is NULL");
    if (count < 1 || count > HASHGRID_ADAMW_MAX_TENSORS)
        return fail(HASHGRID_ERR_ARG, "count = %d outside [1, %d]", count, HASHGRID_ADAMW_MAX_TENSORS);
    for (int k = 0; k < count; ++k)
        if (int rc = check_adamw_tensor(tensors[k], k)) return rc;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return fail(HASHGRID_ERR_CUDA, "cudaGetDevice failed");
    }
    try {
        if (int rc = check_adamw_overlap(tensors, count)) return rc;
        auto* o = new hashgrid_adamw_s;
        *opt = o;
        o->device = dev;
        auto blocks_of = [](int64_t n) { return ((uint64_t)n + HASHGRID_ADAMW_BLOCK - 1) / HASHGRID_ADAMW_BLOCK; };
        for (int k = 0; k < count;) {
            // one launch: as many tensors as its list takes, at most 2^31 blocks
            uint64_t blocks = 0;
            int end = k, have = 0;
            for (; end < count && have < hg::adamw::kLarge; ++end) {
                const uint64_t own = blocks_of(tensors[end].n);
                if (have > 0 && blocks + own > ((uint64_t)1 << 31)) break;
                blocks += own;
                have += own != 0;
            }
            const int begin = (int)o->tensors.size();
            uint32_t first = 0;
            for (; k < end; ++k) {
                const hashgrid_adamw_tensor& t = tensors[k];
                if (t.n == 0) continue;
                hg::adamw::Tensor d;
                d.p = t.param;
                d.g = t.grad;
                d.m = t.m;
                d.v = t.v;
                d.ms = t.m_scale;
                d.vs = t.v_scale;
                d.copy = t.copy;
                d.n = t.n;
                o->first.push_back(first);
                d.types = (uint32_t)t.param_dtype | (uint32_t)t.grad_dtype << 4 | (uint32_t)t.state_dtype << 8 |
                          (uint32_t)(t.copy ? t.copy_dtype : (int)hg::adamw::kNone) << 12 | (uint32_t)k << 16;
                d.rate = t.lr_scale;
                d.keep = t.weight_decay;
                o->tensors.push_back(d);
                first += (uint32_t)blocks_of(t.n);
            }
            if (have == 0) continue;
            hashgrid_adamw_s::Launch l{begin, have, (uint32_t)blocks, {}};
            while ((blocks - 1) >> l.where.shift >= (uint64_t)hg::adamw::kBuckets) ++l.where.shift;
            for (int j = 0, at = 0; j < hg::adamw::kBuckets + 2; ++j) {
                while (at + 1 < have && o->first[begin + at + 1] <= (uint64_t)j << l.where.shift) ++at;
                l.where.tensor[j] = (uint16_t)at;
            }
            o->launches.push_back(l);
        }
    } catch (const std::bad_alloc&) {
        delete *opt;
        *opt = nullptr;
        return fail(HASHGRID_ERR_OOM, "out of host memory");
    }
    return ok();
}

int hashgrid_adamw_destroy(hashgrid_adamw_t opt) {
    delete opt;
    return ok();
}

int hashgrid_adamw_step(hashgrid_adamw_t o, int64_t step, const int64_t* device_step, float lr, float beta1, float beta2,
                        float eps, uint32_t seed, int zero_grad, void* cuda_stream) {
    if (o == nullptr) return fail(HASHGRID_ERR_ARG, "optimiser handle is NULL");
    if (device_step == nullptr && step < 1) return fail(HASHGRID_ERR_ARG, "step = %lld must be >= 1", (long long)step);
    if (!(beta1 >= 0.f && beta1 < 1.f) || !(beta2 >= 0.f && beta2 < 1.f))
        return fail(HASHGRID_ERR_ARG, "betas (%g, %g) must lie in [0, 1)", beta1, beta2);
    if (!(eps >= FLT_MIN) || !std::isfinite(eps) || !std::isfinite(lr))
        return fail(HASHGRID_ERR_ARG, "lr = %g and eps = %g must be finite, eps at least 2^-126", lr, eps);
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return fail(HASHGRID_ERR_CUDA, "cudaGetDevice failed");
    }
    if (dev != o->device) return fail(HASHGRID_ERR_ARG, "the tensors live on device %d but device %d is current", o->device, dev);
    if (device_step != nullptr)
        if (int rc = check_buffer(device_step, sizeof(int64_t), "device_step", 8)) return rc;
    hg::adamw::Params a;
    a.lr = lr;
    a.b1 = beta1;
    a.b2 = beta2;
    a.o1 = (float)(1.0 - (double)beta1);
    a.o2 = (float)(1.0 - (double)beta2);
    a.eps = eps;
    a.db1 = beta1;
    a.db2 = beta2;
    a.c1 = device_step ? 0.f : (float)(1.0 / (1.0 - std::pow((double)beta1, (double)step)));
    a.root2 = device_step ? 0.f : (float)std::sqrt(1.0 / (1.0 - std::pow((double)beta2, (double)step)));
    a.seed = seed;
    a.step = (uint32_t)step;
    a.zero_grad = zero_grad;
    a.device_step = device_step;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return run_checked(s, {}, "adamw_step", [&]() -> int {
        for (const auto& l : o->launches)
            if (int rc = l.count <= hg::adamw::kSmall ? launch_adamw<hg::adamw::kSmall>(o, l, a, s)
                                                      : launch_adamw<hg::adamw::kLarge>(o, l, a, s))
                return rc;
        return ok();
    });
}

int hashgrid_probe(int kind, int width, int pattern, void* buf, size_t buf_bytes, int64_t ops, float* sink,
                   int64_t* ops_done, void* cuda_stream) {
    if (kind != HASHGRID_PROBE_GATHER && kind != HASHGRID_PROBE_RED && kind != HASHGRID_PROBE_RED_F16)
        return fail(HASHGRID_ERR_ARG, "probe kind %d is not a HASHGRID_PROBE_* kind", kind);
    const bool red = kind != HASHGRID_PROBE_GATHER;
    if (!(width == 4 || width == 8 || width == 16 || (width == 32 && !red)))
        return fail(HASHGRID_ERR_ARG, "probe width %d not supported by this kind", width);
    if (pattern < HASHGRID_PROBE_RANDOM || pattern > HASHGRID_PROBE_STREAM)
        return fail(HASHGRID_ERR_ARG, "probe pattern %d is not a HASHGRID_PROBE_* pattern", pattern);
    if ((pattern == HASHGRID_PROBE_SECTOR_PAIR || pattern == HASHGRID_PROBE_LINE_PAIR) && width != 16)
        return fail(HASHGRID_ERR_ARG, "the sector- and line-pair patterns take 16-byte units");
    if (buf_bytes < 256 || (buf_bytes & (buf_bytes - 1)) != 0 || buf_bytes / width > ((size_t)1 << 32))
        return fail(HASHGRID_ERR_ARG, "probe buffer of %zu bytes: need a power of two from 256 to 2^32 units",
                    buf_bytes);
    if (ops < 1) return fail(HASHGRID_ERR_ARG, "ops = %lld must be >= 1", (long long)ops);
    if (int rc = check_buffer(buf, buf_bytes, "buf")) return rc;
    if (width == 32 && reinterpret_cast<uintptr_t>(buf) % 32 != 0)
        return fail(HASHGRID_ERR_ALIGN, "32-byte gathers need a 32-byte-aligned buffer (%p)", buf);
    if (!red)
        if (int rc = check_buffer(sink, sizeof(float), "sink")) return rc;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t blocks = (int64_t)sms * 8;
    const int64_t per_iter = blocks * hg::probe::kThreads * hg::probe::kOpsPerIter;
    const int64_t iters = (ops + per_iter - 1) / per_iter;
    if (iters > 0x7fffffffLL) return fail(HASHGRID_ERR_ARG, "ops = %lld is too many", (long long)ops);
    if (ops_done != nullptr) *ops_done = iters * per_iter;
    const uint32_t mask = (uint32_t)(buf_bytes / width - 1);
    char* b = static_cast<char*>(buf);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const dim3 grid((unsigned)blocks), block(hg::probe::kThreads);
    const int it = (int)iters;
    const uint32_t seed = 0x2545f491u;
    using namespace hg::probe;
    if (kind == HASHGRID_PROBE_RED) {
        switch (width) {
            case 4: probe_kernel<4, kRedF32><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
            case 8: probe_kernel<8, kRedF32><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
            default: probe_kernel<16, kRedF32><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
        }
    } else if (kind == HASHGRID_PROBE_RED_F16) {
        switch (width) {
            case 4: probe_kernel<4, kRedF16><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
            case 8: probe_kernel<8, kRedF16><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
            default: probe_kernel<16, kRedF16><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
        }
    } else {
        switch (width) {
            case 4: probe_kernel<4, kGather><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
            case 8: probe_kernel<8, kGather><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
            case 16: probe_kernel<16, kGather><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
            default: probe_kernel<32, kGather><<<grid, block, 0, s>>>(b, mask, pattern, it, seed, sink); break;
        }
    }
    return launch_status("probe");
}

const char* hashgrid_last_error(void) { return g_last_error.c_str(); }

const char* hashgrid_version(void) { return HASHGRID_VERSION_STRING; }

}  // extern "C"
