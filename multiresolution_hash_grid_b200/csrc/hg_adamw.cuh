// hg_adamw.cuh -- one AdamW step over a list of tensors.
//
// Per element, at step t (fp32, each operation rounded to nearest, no contraction, so that
// the 8-bit codes that follow from it are reproducible bit for bit):
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
//   p = p (1 - lr wd) - lr (m c1) / (sqrt(v c2) + eps),  c = 1 / (1 - b^t).
// States are fp32, or e4m3 codes with one fp32 scale per 256 elements; v is held as its
// square root there, since 8 bits of v itself would span half the orders of magnitude.
//
// A pass over memory: 28 bytes an element with fp32 parameter, gradient and states, 16 with
// 8-bit states, against some 60 (fp32) to 130 (stochastic rounding) instructions.
//
// A warp takes one block of 256 elements, lane j elements 4j..4j+3 and 128+4j..: every array,
// whatever its type, is read and written in whole coalesced vectors (16, 8 or 4 bytes a lane),
// and a block's largest magnitude is a shuffle reduction within the warp. The list of tensors
// travels as a kernel parameter: no device copy of it to keep, and a captured graph holds it
// by value.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "hg_check.cuh"
#include "hg_probe.cuh"

namespace hg {
namespace adamw {

constexpr int kBlock = 256;                      // elements per scale and per warp item
constexpr int kWarps = 8;                        // warps per thread block
constexpr float kTop = 448.f;                    // largest e4m3 value

enum Type { kF32 = 0, kF16 = 1, kBf16 = 2, kE4m3 = 3, kNone = 15 };

struct Tensor {
    void* p;
    void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    void* copy;
    int64_t n;
    uint32_t first;   // index of the tensor's first 256-element block in the launch
    uint32_t types;   // param | grad << 4 | state << 8 | copy << 12 | place in the caller's list << 16
    float lr_scale, decay;
};

struct Params {
    float lr, b1, b2, o1, o2, eps, c1, c2;  // o = 1 - b
    double db1, db2;
    uint32_t seed, step;
    int zero_grad;
    const int64_t* device_step;
};

// Lists of up to kSmall tensors take less kernel-parameter space than long ones.
constexpr int kSmall = 40, kLarge = 400;
template <int kCap>
struct List {
    uint32_t count, blocks;
    Tensor t[kCap];
};

template <int R>
__device__ __forceinline__ bool inside(const void* base, int64_t n, int64_t i, int k) {
#ifdef HASHGRID_CHECKED
    if (i < 0 || i + k > n) {
        atomicOr(&g_check_flags, 1u << R);
        return false;
    }
#endif
    (void)base; (void)n; (void)i; (void)k;
    return true;
}

__device__ __forceinline__ float2 unpack(uint32_t w, int type) {
    if (type == kF16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ uint32_t pack(float a, float b, int type) {
    if (type == kF16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Elements i..i+3 of an array of `n`, as fp32 (zeros beyond its end). i is a multiple of 4 and
// the base 16-byte aligned, so a group of four lies on its own size.
__device__ __forceinline__ void load4(const void* base, int type, int64_t i, int64_t n, float (&x)[4]) {
    if (i + 4 <= n) {
        if (!inside<kChkAdamw>(base, n, i, 4)) return;
        if (type == kF32) {
            const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
            x[0] = q.x; x[1] = q.y; x[2] = q.z; x[3] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
            const float2 lo = unpack(q.x, type), hi = unpack(q.y, type);
            x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[k] = 0.f;
        if (i + k < n && inside<kChkAdamw>(base, n, i + k, 1)) {
            if (type == kF32) x[k] = static_cast<const float*>(base)[i + k];
            else x[k] = unpack(static_cast<const uint16_t*>(base)[i + k], type).x;
        }
    }
}

__device__ __forceinline__ void store4(void* base, int type, int64_t i, int64_t n, const float (&x)[4]) {
    if (i + 4 <= n) {
        if (!inside<kChkAdamw>(base, n, i, 4)) return;
        if (type == kF32)
            *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(x[0], x[1], x[2], x[3]);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) =
                make_uint2(pack(x[0], x[1], type), pack(x[2], x[3], type));
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (i + k < n && inside<kChkAdamw>(base, n, i + k, 1)) {
            if (type == kF32) static_cast<float*>(base)[i + k] = x[k];
            else static_cast<uint16_t*>(base)[i + k] = (uint16_t)pack(x[k], 0.f, type);
        }
}

__device__ __forceinline__ uint32_t load_codes(const void* base, int64_t i, int64_t n) {
    const uint8_t* c = static_cast<const uint8_t*>(base);
    if (i + 4 <= n) return inside<kChkAdamw>(base, n, i, 4) ? *reinterpret_cast<const uint32_t*>(c + i) : 0u;
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (i + k < n && inside<kChkAdamw>(base, n, i + k, 1)) w |= (uint32_t)c[i + k] << (8 * k);
    return w;
}

__device__ __forceinline__ void store_codes(void* base, int64_t i, int64_t n, uint32_t w) {
    uint8_t* c = static_cast<uint8_t*>(base);
    if (i + 4 <= n) {
        if (inside<kChkAdamw>(base, n, i, 4)) *reinterpret_cast<uint32_t*>(c + i) = w;
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (i + k < n && inside<kChkAdamw>(base, n, i + k, 1)) c[i + k] = (uint8_t)(w >> (8 * k));
}

__device__ __forceinline__ void decode(uint32_t w, float scale, float (&x)[4]) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
    x[0] = __fmul_rn(a.x, scale);
    x[1] = __fmul_rn(a.y, scale);
    x[2] = __fmul_rn(b.x, scale);
    x[3] = __fmul_rn(b.y, scale);
}

// y >= 0 with its mantissa cut to three bits after a random part of a code was added: for
// y < 2^-6, where e4m3 is spaced evenly by 2^-9, 2^-6 is added first, which puts y where floats
// of three mantissa bits have that very spacing.
__device__ __forceinline__ float stochastic(float y, uint32_t r16) {
    const float low = y < 0x1p-6f ? 0x1p-6f : 0.f;
    const uint32_t bits = (__float_as_uint(__fadd_rn(y, low)) + (r16 * 16u + 8u)) & ~0xFFFFFu;
    return fminf(__fsub_rn(__uint_as_float(bits), low), kTop);
}

// Codes of 2 x 4 values x (the lane's share of a 256-element block), and the block's scale.
// kRoot: the values are square roots, and a positive one is coded as 2^-9 at least.
template <bool kRoot>
__device__ __forceinline__ float encode(const float (&x)[2][4], const uint32_t (&h)[2][4], bool nearest, uint32_t (&w)[2]) {
    float top = 0.f;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float y = fabsf(x[a][k]);
            top = fmaxf(top, y < __int_as_float(0x7f800000) ? y : 0.f);  // neither infinity nor NaN
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = __fdiv_rn(top, kTop);
    // a block whose reciprocal overflows holds nothing that its codes could stand for
    float inverse = top > 0x1p-100f ? __fdiv_rn(kTop, top) : 0.f;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        float q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float v = x[a][k];
            float y = __fmul_rn(fabsf(v), inverse);
            if (!nearest) y = stochastic(y, kRoot ? h[a][k] >> 16 : h[a][k] & 0xffffu);
            if (kRoot && v > 0.f) y = fmaxf(y, 0x1p-9f);
            y = v < 0.f ? -y : y;
            if (!(fabsf(v) < __int_as_float(0x7f800000))) y = __int_as_float(0x7fc00000);
            q[k] = y;
        }
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
        w[a] = lo | hi << 16;
    }
    return scale;
}

template <int kCap>
__global__ void __launch_bounds__(32 * kWarps) step_kernel(const __grid_constant__ List<kCap> list, const Params a) {
    float c1 = a.c1, c2 = a.c2;
    uint32_t step = a.step;
    if (a.device_step != nullptr) {
        const int64_t t = *a.device_step;
        if (t < 1) return;
        step = (uint32_t)t;
        c1 = (float)(1.0 / (1.0 - pow(a.db1, (double)t)));
        c2 = (float)(1.0 / (1.0 - pow(a.db2, (double)t)));
    }
    const int lane = threadIdx.x & 31;
    const uint32_t b = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (b >= list.blocks) return;
    uint32_t lo = 0, hi = list.count;  // the last tensor whose first block is at most b
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (list.t[mid].first <= b) lo = mid; else hi = mid;
    }
    const Tensor& T = list.t[lo];
    const int64_t n = T.n, blk = b - T.first, base = blk * kBlock;
    const int tp = T.types & 15, tg = (T.types >> 4) & 15, ts = (T.types >> 8) & 15, tc = (T.types >> 12) & 15;
    const int64_t at[2] = {base + 4 * lane, base + 128 + 4 * lane};

    float p[2][4], g[2][4], m[2][4], v[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        load4(T.g, tg, at[k], n, g[k]);
        load4(T.p, tp, at[k], n, p[k]);
    }
    if (ts == kF32) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            load4(T.m, kF32, at[k], n, m[k]);
            load4(T.v, kF32, at[k], n, v[k]);
        }
    } else {
        const float ms = T.ms[blk], vs = T.vs[blk];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            decode(load_codes(T.m, at[k], n), ms, m[k]);
            decode(load_codes(T.v, at[k], n), vs, v[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[k][j] = __fmul_rn(v[k][j], v[k][j]);
        }
    }
    const float rate = __fmul_rn(T.lr_scale, a.lr);
    const float keep = (float)(1.0 - (double)T.lr_scale * (double)a.lr * (double)T.decay);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gj = g[k][j];
            m[k][j] = __fadd_rn(__fmul_rn(m[k][j], a.b1), __fmul_rn(gj, a.o1));
            v[k][j] = __fadd_rn(__fmul_rn(v[k][j], a.b2), __fmul_rn(__fmul_rn(gj, gj), a.o2));
            const float d = __fadd_rn(__fsqrt_rn(__fmul_rn(v[k][j], c2)), a.eps);
            const float u = __fmul_rn(rate, __fdiv_rn(__fmul_rn(m[k][j], c1), d));
            p[k][j] = __fsub_rn(__fmul_rn(p[k][j], keep), u);
        }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        store4(T.p, tp, at[k], n, p[k]);
        if (tc != kNone) store4(T.copy, tc, at[k], n, p[k]);
        if (a.zero_grad) {
            const float z[4] = {0.f, 0.f, 0.f, 0.f};
            store4(T.g, tg, at[k], n, z);
        }
    }
    if (ts == kF32) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            store4(T.m, kF32, at[k], n, m[k]);
            store4(T.v, kF32, at[k], n, v[k]);
        }
        return;
    }
    uint32_t h[2][4] = {}, w[2];
    const bool nearest = a.seed == 0;
    if (!nearest) {
        const uint32_t key = probe::mix32(a.seed * 0x9E3779B1u + step * 0x85EBCA77u + (T.types >> 16) * 0xC2B2AE3Du +
                                          (uint32_t)((uint64_t)base >> 32) * 0x27D4EB2Fu);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) h[k][j] = probe::mix32((uint32_t)(at[k] + j) ^ key);
    }
    const float ms = encode<false>(m, h, nearest, w);
    store_codes(T.m, at[0], n, w[0]);
    store_codes(T.m, at[1], n, w[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[k][j] = __fsqrt_rn(v[k][j]);
    const float vs = encode<true>(v, h, nearest, w);
    store_codes(T.v, at[0], n, w[0]);
    store_codes(T.v, at[1], n, w[1]);
    if (lane == 0) {
        T.ms[blk] = ms;
        T.vs[blk] = vs;
    }
}

}  // namespace adamw
}  // namespace hg
