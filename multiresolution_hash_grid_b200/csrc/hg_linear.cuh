// hg_linear.cuh -- linear layers with their gradients.
//
//   forward:  z = x W^T + b;  y = act(z) + residual
//   backward: dz = dy act'(z);  dx = dz W;  dW = dz^T x;  db = sum over rows of dz
//
// All three products are D[m][n] = sum_k A(m, k) B(n, k) with 16-bit operands, exact products
// and fp32 sums.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "hg_check.cuh"
#include "hg_mlp.cuh"

namespace hg {
namespace linear {

enum Act { kNoAct = 0, kRelu = 1, kGelu = 2, kSilu = 3 };

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }

__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case kRelu: return z > 0.f ? z : 0.f;
        case kGelu: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
        case kSilu: return z / (1.f + expf(-z));
    }
    return z;
}

// act'(z). GELU: Phi(z) + z phi(z); SILU: s (1 + z (1 - s)).
__device__ __forceinline__ float slope(float z, int act) {
    switch (act) {
        case kRelu: return z > 0.f ? 1.f : 0.f;
        case kGelu:
            return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
        case kSilu: {
            const float s = 1.f / (1.f + expf(-z));
            return s * (1.f + z * (1.f - s));
        }
    }
    return 1.f;
}

// What happens to D[row][col] on its way out; out is of type T or fp32.
struct Epilogue {
    const float* bias;     // [cols] or NULL
    const void* residual;  // of the output's type, or NULL
    void* out;
    void* z;               // of type T, or NULL
    int64_t ldr, ldo, ldz;
    int out_f32, act;
    int role;              // CheckRole of out
    int vectors;           // every array takes 16-byte vectors at columns that are multiples of 8
};

template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) { return mlp::pack_bf16(a, b); }
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// One value: any alignment, any width.
template <typename T>
__device__ __forceinline__ void emit(const Epilogue& e, int64_t row, int64_t col, float acc) {
    float z = acc;
    if (e.bias != nullptr && in_bounds<kChkBias>(e.bias + col, 4)) z += e.bias[col];
    if (e.z != nullptr) {
        T* p = static_cast<T*>(e.z) + row * e.ldz + col;
        if (in_bounds<kChkZ>(p, sizeof(T))) *p = from_float<T>(z);
    }
    float y = activate(z, e.act);
    if (e.out_f32) {
        if (e.residual != nullptr) {
            const float* r = static_cast<const float*>(e.residual) + row * e.ldr + col;
            if (in_bounds<kChkResidual>(r, 4)) y += *r;
        }
        float* p = static_cast<float*>(e.out) + row * e.ldo + col;
        if (in_bounds_role(e.role, p, 4)) *p = y;
    } else {
        if (e.residual != nullptr) {
            const T* r = static_cast<const T*>(e.residual) + row * e.ldr + col;
            if (in_bounds<kChkResidual>(r, sizeof(T))) y += to_float(*r);
        }
        T* p = static_cast<T*>(e.out) + row * e.ldo + col;
        if (in_bounds_role(e.role, p, sizeof(T))) *p = from_float<T>(y);
    }
}

// Eight neighbouring values (col a multiple of 8), bias already added, as 16-byte vectors.
template <typename T>
__device__ __forceinline__ void emit8(const Epilogue& e, int64_t row, int64_t col, float (&y)[8]) {
    if (e.z != nullptr) {
        T* p = static_cast<T*>(e.z) + row * e.ldz + col;
        if (in_bounds<kChkZ>(p, 16))
            *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
    }
    switch (e.act) {
        case kRelu:
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = activate(y[j], kRelu);
            break;
        case kGelu:
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = activate(y[j], kGelu);
            break;
        case kSilu:
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = activate(y[j], kSilu);
            break;
    }
    if (e.out_f32) {
        if (e.residual != nullptr) {
            const float* r = static_cast<const float*>(e.residual) + row * e.ldr + col;
            if (in_bounds<kChkResidual>(r, 32)) {
                const float4 a = *reinterpret_cast<const float4*>(r), b = *reinterpret_cast<const float4*>(r + 4);
                y[0] += a.x; y[1] += a.y; y[2] += a.z; y[3] += a.w;
                y[4] += b.x; y[5] += b.y; y[6] += b.z; y[7] += b.w;
            }
        }
        float* p = static_cast<float*>(e.out) + row * e.ldo + col;
        if (in_bounds_role(e.role, p, 32)) {
            *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(y[4], y[5], y[6], y[7]);
        }
    } else {
        if (e.residual != nullptr) {
            const T* r = static_cast<const T*>(e.residual) + row * e.ldr + col;
            if (in_bounds<kChkResidual>(r, 16)) {
                const uint4 q = *reinterpret_cast<const uint4*>(r);
                const float2 a = unpack2<T>(q.x), b = unpack2<T>(q.y), c = unpack2<T>(q.z), d = unpack2<T>(q.w);
                y[0] += a.x; y[1] += a.y; y[2] += b.x; y[3] += b.y;
                y[4] += c.x; y[5] += c.y; y[6] += d.x; y[7] += d.y;
            }
        }
        T* p = static_cast<T*>(e.out) + row * e.ldo + col;
        if (in_bounds_role(e.role, p, 16))
            *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
    }
}

// ---------------------------------------------------------------------------------------
// The product D[m][n] = sum_k A(m, k) B(n, k) on the tensor cores: tcgen05.mma of 128 x bn x 16
// with the accumulator in tensor memory.
//
// An operand is a row-major array with k along its rows ("k-major": x and W of the forward
// product) or along its columns ("mn-major": W in dx = dz W, dz and x in dW = dz^T x); the
// tensor cores take both, so nothing is transposed in memory. It is staged 64 values of k at a
// time in the 128-byte-swizzled layout: rows of 64 contiguous elements (128 bytes), eight to a
// 1024-byte group, 16-byte chunk c of row r at chunk c ^ (r % 8). K-major: a row of it is an m (or
// n) and holds 64 k. Mn-major: a row is a k and holds 64 m, one such box per 64 m.
//
// Warps: 0-7 read finished accumulators (two for each quarter of the 128 TMEM lanes, taking
// turns at 32-column chunks), 8 issues the MMAs, 9 issues the TMA copies. Arrays whose rows do
// not start on 16-byte boundaries cannot be copied by TMA: eight more warps load those with
// plain loads and write the same layout. Two accumulators alternate, so that the next tile's
// MMAs run while the last one is written out. Persistent over tiles, n fastest.
//
// Way out: a 32 x 32 chunk goes from TMEM (a lane holds a row) through 4 KB of shared memory a
// warp, so that four neighbouring lanes then hold 32 neighbouring columns of a row: bias,
// residual, z and y move in whole 16-byte vectors and 64-byte row pieces. Every value stays
// fp32 until it is stored.
// ---------------------------------------------------------------------------------------
constexpr int kBm = 128, kBk = 64;
constexpr int kOutWarps = 8, kLoadWarps = 8;
constexpr int kThreads = 32 * (kOutWarps + 2);          // without the loading warps
constexpr int kThreadsDirect = kThreads + 32 * kLoadWarps;
constexpr int kMaxStages = 8;
constexpr int kStageA = kBm * kBk * 2;
constexpr int kStaging = kOutWarps * 32 * 32 * 4;

struct Side {             // one operand
    const void* p;
    int64_t ld;           // elements between its rows
    uint64_t bytes;       // extent
    int64_t outer, inner; // rows and columns of the array
    int mn, direct;       // k runs along its columns; not copied by TMA
    int box_rows, boxes;  // boxes of box_rows x 64 elements that make up a stage of it
    int role;             // CheckRole
};

struct Gemm {
    CUtensorMap ta, tb;
    Side a, b;
    int64_t M, N;
    int bn, columns;      // tile width; columns from one accumulator to the next
    int stages, stage_bytes;
    int kblocks, kblocks_per_split;
    int mt, nt;
    uint32_t idesc, tmem_columns;
    Epilogue e;
    int64_t split_stride; // elements of fp32 output from one split to the next
    int* status;
};

__host__ __device__ constexpr size_t gemm_smem(int stages, int stage_bytes) {
    return 1024 + (size_t)stages * stage_bytes + kStaging + (2 * kMaxStages + 4 + 1) * 8 + 16;
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void arrive_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}\n" ::"r"(bar), "r"(bytes) : "memory");
}

// Shared-memory descriptor of a 128-byte-swizzled operand: version 1 (bits 46-47), swizzle code
// 2 (bits 61-63), 8-row groups 1024 bytes apart (stride offset); `leading` is the distance of
// 64-wide boxes of an mn-major operand (unused for a k-major one).
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t saddr, uint32_t leading) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((leading >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// 32 consecutive fp32 accumulator columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// A bounded wait that also ends, with false, once another role of the block has given up.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    for (uint32_t it = 0; it < mlp::kWaitLimit; ++it) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        if ((it & 255u) == 255u && *abort_flag != 0) return false;
    }
    *abort_flag = 1;
    return false;
}

// Position in a ring of stages.
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// 16 bytes of a row from a source of any 2-byte alignment: the two aligned 16-byte units that hold
// them, shifted together. Where those would pass the array's end, or for fewer than 8
// elements, one element at a time.
__device__ __forceinline__ uint4 load_chunk(const Side& s, int64_t row, int64_t col) {
    uint4 out = make_uint4(0u, 0u, 0u, 0u);
    if (row >= s.outer || col >= s.inner) return out;
    const char* base = static_cast<const char*>(s.p);
    const uint64_t off = (uint64_t)(row * s.ld + col) * 2, lo = off & ~15ull;
    if (col + 8 <= s.inner && lo + 32 <= s.bytes) {
        if (!in_bounds_role(s.role, base + lo, 32)) return out;
        const uint4 p = __ldg(reinterpret_cast<const uint4*>(base + lo));
        const uint32_t sh = (uint32_t)(off & 15u);
        if (sh == 0) return p;
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(base + lo + 16));
        uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
        if (sh & 8u) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (sh & 4u) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        const uint32_t bits = (sh & 2u) * 8u;
        return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
    }
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (col + j < s.inner && in_bounds_role(s.role, base + off + 2 * j, 2))
            w[j >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(base + off + 2 * j) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One stage of an operand by plain loads: i0 its first m (or n), k0 its first k.
__device__ __forceinline__ void load_direct(const Side& s, uint8_t* dst, int64_t i0, int64_t k0, int t) {
    const int chunks = s.box_rows * 8, total = chunks * s.boxes;
    const int64_t row0 = s.mn ? k0 : i0, col0 = s.mn ? i0 : k0;
#pragma unroll 4
    for (int i = t; i < total; i += 32 * kLoadWarps) {
        const int box = i / chunks, r = (i - box * chunks) >> 3, c = i & 7;
        const uint4 v = load_chunk(s, row0 + r, col0 + box * 64 + c * 8);
        *reinterpret_cast<uint4*>(dst + box * s.box_rows * 128 + r * 128 + ((c ^ (r & 7)) << 4)) = v;
    }
}

template <typename T, bool kDirect>
__global__ void __launch_bounds__(kDirect ? kThreadsDirect : kThreads, kDirect ? 1 : 2) gemm_kernel(const __grid_constant__ Gemm g) {
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint8_t* staging = sm + (size_t)g.stages * g.stage_bytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStaging);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 5);
    __shared__ volatile int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sm0 = (uint32_t)__cvta_generic_to_shared(sm), bar0 = (uint32_t)__cvta_generic_to_shared(bars);
    // barriers: full[stage], empty[stage], accumulator done[2], accumulator free[2], drain
    const uint32_t full = bar0, empty = bar0 + 8 * kMaxStages, done = empty + 8 * kMaxStages, room = done + 16, drain = room + 16;
    const bool tma_a = !kDirect || !g.a.direct, tma_b = !kDirect || !g.b.direct;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < g.stages; ++s) {
            mlp::mbar_init(full + 8 * s, (tma_a || tma_b ? 1 : 0) + (tma_a && tma_b ? 0 : kLoadWarps));
            mlp::mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mlp::mbar_init(done + 8 * i, 1);
            mlp::mbar_init(room + 8 * i, kOutWarps);
        }
        mlp::mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"((uint32_t)__cvta_generic_to_shared(tslot)),
                     "r"(g.tmem_columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    mlp::fence_before();
    __syncthreads();
    mlp::fence_after();
    const uint32_t tmem = *tslot;
    const int tiles = g.mt * g.nt, kb0 = blockIdx.y * g.kblocks_per_split;
    const int kbs = max(0, min(g.kblocks_per_split, g.kblocks - kb0));

    if (warp == kOutWarps + 1) {
        // ------------------------------- TMA copies -------------------------------
        if (lane == 0 && (tma_a || tma_b)) {
            const uint32_t bytes = (tma_a ? g.a.box_rows * g.a.boxes * 128 : 0) + (tma_b ? g.b.box_rows * g.b.boxes * 128 : 0);
            Ring r;
            uint32_t issued = 0;  // copies so far, at most counted to the number of stages
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int m0 = t / g.nt * kBm, n0 = t % g.nt * g.bn;
                for (int kb = 0; kb < kbs; ++kb) {
                    if (!(ok = wait_bounded(empty + 8 * r.stage, r.phase ^ 1u, &abort_flag))) break;
                    const uint32_t bar = full + 8 * r.stage, sa = sm0 + r.stage * g.stage_bytes, sb = sa + kStageA;
                    const int k0 = (kb0 + kb) * kBk;
                    arrive_expect(bar, bytes);
                    if (tma_a)
                        for (int j = 0; j < g.a.boxes; ++j)
                            tma_load(sa + j * g.a.box_rows * 128, &g.ta, g.a.mn ? m0 + 64 * j : k0, g.a.mn ? k0 : m0, bar);
                    if (tma_b)
                        for (int j = 0; j < g.b.boxes; ++j)
                            tma_load(sb + j * g.b.box_rows * 128, &g.tb, g.b.mn ? n0 + 64 * j : k0, g.b.mn ? k0 : n0, bar);
                    r.next(g.stages);
                    issued = min(issued + 1, (uint32_t)g.stages);
                }
            }
            // given up: the copies in flight still write to this block's shared memory
            for (; !ok && issued > 0; --issued) {
                if (r.stage == 0) {
                    r.stage = g.stages;
                    r.phase ^= 1u;
                }
                --r.stage;
                mlp::wait_parity(full + 8 * r.stage, r.phase);
            }
        }
    } else if (warp == kOutWarps) {
        // ---------------------------------- MMAs ----------------------------------
        if (lane == 0) {
            Ring r;
            uint32_t i = 0;
            bool ok = true;
            const uint32_t step_a = g.a.mn ? 2048 : 32, step_b = g.b.mn ? 2048 : 32;
            for (int t = blockIdx.x; t < tiles && ok && kbs > 0; t += gridDim.x, ++i) {
                const uint32_t acc = tmem + (i & 1u) * g.columns;
                if (!(ok = wait_bounded(room + 8 * (i & 1u), ((i >> 1) & 1u) ^ 1u, &abort_flag))) break;
                mlp::fence_after();
                for (int kb = 0; kb < kbs; ++kb) {
                    if (!(ok = wait_bounded(full + 8 * r.stage, r.phase, &abort_flag))) break;
                    mlp::fence_after();
                    const uint32_t sa = sm0 + r.stage * g.stage_bytes, sb = sa + kStageA;
#pragma unroll
                    for (int k = 0; k < kBk / 16; ++k)
                        mlp::mma(acc, swizzled_desc(sa + k * step_a, 64 * 128), swizzled_desc(sb + k * step_b, 64 * 128), g.idesc,
                                 (kb | k) != 0 ? 1u : 0u);
                    mlp::commit(empty + 8 * r.stage);
                    r.next(g.stages);
                }
                if (ok) mlp::commit(done + 8 * (i & 1u));
            }
            if (!ok) {
                mlp::commit(drain);
                mlp::wait_parity(drain, 0);
            }
        }
    } else if (kDirect && warp > kOutWarps + 1) {
        // ------------------------------- plain loads -------------------------------
        const int lt = threadIdx.x - kThreads;
        Ring r;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const int64_t m0 = (int64_t)(t / g.nt) * kBm, n0 = (int64_t)(t % g.nt) * g.bn;
            for (int kb = 0; kb < kbs; ++kb) {
                ok = wait_bounded(empty + 8 * r.stage, r.phase ^ 1u, &abort_flag);
                if (__any_sync(0xffffffffu, !ok)) {
                    ok = false;
                    break;
                }
                uint8_t* sa = sm + r.stage * g.stage_bytes;
                const int64_t k0 = (int64_t)(kb0 + kb) * kBk;
                if (g.a.direct) load_direct(g.a, sa, m0, k0, lt);
                if (g.b.direct) load_direct(g.b, sa + kStageA, n0, k0, lt);
                mlp::fence_async_smem();
                __syncwarp();
                if (lane == 0) mlp::mbar_arrive(full + 8 * r.stage);
                r.next(g.stages);
            }
        }
    } else {
        // -------------------------------- way out ---------------------------------
        const int quarter = warp & 3, chunks = (g.bn + 31) / 32;
        float4* st = reinterpret_cast<float4*>(staging + warp * 4096);
        Epilogue e = g.e;
        if (g.split_stride != 0) e.out = static_cast<float*>(e.out) + blockIdx.y * g.split_stride;
        uint32_t i = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
            const int64_t m0 = (int64_t)(t / g.nt) * kBm + 32 * quarter, n0 = (int64_t)(t % g.nt) * g.bn;
            const int rows = (int)min((int64_t)32, g.M - m0);
            const int64_t cols = min(g.N, n0 + g.bn);
            if (kbs > 0) {
                ok = wait_bounded(done + 8 * (i & 1u), (i >> 1) & 1u, &abort_flag);
                if (__any_sync(0xffffffffu, !ok)) break;
                mlp::fence_after();
            }
            for (int c = warp >> 2; c < chunks; c += 2) {
                uint32_t v[32];
                __syncwarp();
                if (kbs > 0) {
                    tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + (i & 1u) * g.columns + 32 * c, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                }
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    st[lane * 8 + (u ^ (lane & 7))] = make_float4(__uint_as_float(v[4 * u]), __uint_as_float(v[4 * u + 1]),
                                                                  __uint_as_float(v[4 * u + 2]), __uint_as_float(v[4 * u + 3]));
                __syncwarp();
                const int64_t c0 = n0 + 32 * c;
                if (e.vectors) {
                    const int64_t col = c0 + 8 * (lane & 3);
                    if (col + 8 <= cols) {
                        float b[8] = {};
                        if (e.bias != nullptr && in_bounds<kChkBias>(e.bias + col, 32)) {
                            const float4 lo = __ldg(reinterpret_cast<const float4*>(e.bias + col)),
                                         hi = __ldg(reinterpret_cast<const float4*>(e.bias + col + 4));
                            b[0] = lo.x; b[1] = lo.y; b[2] = lo.z; b[3] = lo.w;
                            b[4] = hi.x; b[5] = hi.y; b[6] = hi.z; b[7] = hi.w;
                        }
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const int r = 8 * p + (lane >> 2);
                            if (r >= rows) break;
                            const float4 lo = st[r * 8 + ((2 * (lane & 3)) ^ (r & 7))], hi = st[r * 8 + ((2 * (lane & 3) + 1) ^ (r & 7))];
                            float y[8] = {lo.x + b[0], lo.y + b[1], lo.z + b[2], lo.w + b[3],
                                          hi.x + b[4], hi.y + b[5], hi.z + b[6], hi.w + b[7]};
                            emit8<T>(e, m0 + r, col, y);
                        }
                    } else {
                        const float* sf = reinterpret_cast<const float*>(st);
                        for (int p = 0; p < 4; ++p) {
                            const int r = 8 * p + (lane >> 2);
                            if (r >= rows) break;
                            for (int j = 0; j < 8; ++j)
                                if (col + j < cols)
                                    emit<T>(e, m0 + r, col + j, sf[r * 32 + (((2 * (lane & 3) + (j >> 2)) ^ (r & 7)) << 2) + (j & 3)]);
                        }
                    }
                } else if (c0 + lane < cols) {
                    const float* sf = reinterpret_cast<const float*>(st);
                    for (int r = 0; r < rows; ++r) emit<T>(e, m0 + r, c0 + lane, sf[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)]);
                }
            }
            if (kbs > 0) {
                mlp::fence_before();
                __syncwarp();
                if (lane == 0) mlp::mbar_arrive(room + 8 * (i & 1u));
            }
        }
    }
    __syncwarp();
    mlp::fence_before();
    __syncthreads();
    mlp::fence_after();
    if (threadIdx.x == 0 && abort_flag != 0 && g.status != nullptr) atomicExch(g.status, 1);
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.tmem_columns) : "memory");
}

// dz = dy act'(z), rounded to T, into dz (NULL: not wanted), and the sums of the unrounded dz
// over this block's rows into sums[blockIdx.y][col] (NULL: not wanted). A block takes 32
// columns, its 8 warps every eighth row of its share.
template <typename T>
__global__ void __launch_bounds__(256) slope_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ z,
                                                    int64_t rows, int cols, int act, T* __restrict__ dz, int64_t lddz,
                                                    float* __restrict__ sums) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    const int64_t share = (rows + gridDim.y - 1) / gridDim.y, r0 = blockIdx.y * share, r1 = min(rows, r0 + share);
    float s = 0.f;
    if (col < cols)
        for (int64_t r = r0 + warp; r < r1; r += 8) {
            float d = in_bounds<kChkDout>(dy + r * lddy + col, 2) ? to_float(dy[r * lddy + col]) : 0.f;
            if (act != kNoAct && in_bounds<kChkZ>(z + r * cols + col, 2)) d *= slope(to_float(z[r * cols + col]), act);
            if (dz != nullptr && in_bounds<kChkWork>(dz + r * lddz + col, 2)) dz[r * lddz + col] = from_float<T>(d);
            s += d;
        }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < cols && sums != nullptr) {
#pragma unroll
        for (int w = 1; w < 8; ++w) s += part[w][lane];
        if (in_bounds<kChkWork>(sums + (int64_t)blockIdx.y * cols + col, 4)) sums[(int64_t)blockIdx.y * cols + col] = s;
    }
}

// out[i] = sum over parts of sums[part][i], in order.
template <typename T>
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ sums, int parts, int64_t n, T* __restrict__ out, int role) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
    for (int p = 0; p < parts; ++p)
        if (in_bounds<kChkWork>(sums + p * n + i, 4)) s += sums[p * n + i];
    if (in_bounds_role(role, out + i, sizeof(T))) out[i] = from_float<T>(s);
}

}  // namespace linear
}  // namespace hg
