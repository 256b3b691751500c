// hg_adamw.cuh -- one AdamW step over a list of tensors.
//
// Per element, at step t (fp32, each operation rounded to nearest, no contraction, so that
// the 8-bit codes that follow from it are reproducible bit for bit):
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
//   p = p (1 - lr wd) - lr (m c1) / (sqrt(v) sqrt(c2) + eps),  c = 1 / (1 - b^t)
// (one root serves the step and the 8-bit state).
// States are fp32, or e4m3 codes with one fp32 scale per 256 elements; v is held as its
// square root there, since 8 bits of v itself would span half the orders of magnitude.
//
// A pass over memory: 28 bytes an element with fp32 parameter, gradient and states, 16 with
// 8-bit states, against 36 (fp32 states) to 93 (8-bit states, stochastic rounding) instructions.
//
// A warp takes one block of 256 elements, lane j elements 4j..4j+3 and 128+4j..: every array,
// whatever its type, is read and written in whole coalesced vectors (16, 8 or 4 bytes a lane),
// and a block's largest magnitude is a shuffle reduction within the warp. The list of tensors
// travels as a kernel parameter: no device copy of it to keep, and a captured graph holds it
// by value. (A warp that walked four neighbouring blocks, to find their tensor and rates once, was
// slower: 77 against 73.5 us for 2^24 fp32 elements.)
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
    uint32_t types;   // param | grad << 4 | state << 8 | copy << 12 | place in the caller's list << 16
    float rate, keep;  // lr * lr_scale, 1 - rate * weight_decay (in the handle: lr_scale and weight_decay)
};

struct Params {
    float lr, b1, b2, o1, o2, eps, c1, root2;  // o = 1 - b, c1 = 1/(1-b1^t), root2 = sqrt(1/(1-b2^t))
    double db1, db2;
    uint32_t seed, step;
    int zero_grad;
    const int64_t* device_step;
};

// Lists of up to kSmall tensors take less kernel-parameter space than long ones.
constexpr int kSmall = 40, kLarge = 380;
// Where a block's tensor is searched for: block b >> shift's entry is the last tensor that begins at or before the
// bucket. (Searching the whole list took 7 of 48 us of a step with 8-bit states over 160 tensors.)
constexpr int kBuckets = 128;
struct Buckets {
    uint32_t shift;
    uint16_t tensor[kBuckets + 2];
};

template <int kCap>
struct List {
    uint32_t count, blocks;
    uint32_t first[kCap];  // index of a tensor's first 256-element block
    Buckets where;
    Tensor t[kCap];
};

template <int R>
__device__ __forceinline__ bool inside(int64_t n, int64_t i, int k) {
#ifdef HASHGRID_CHECKED
    if (i < 0 || i + k > n) {
        atomicOr(&g_check_flags, 1u << R);
        return false;
    }
#endif
    (void)n; (void)i; (void)k;
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

// Elements i..i+3 of an array of `n`, as fp32 pairs (zeros beyond its end). i is a multiple of 4
// and the base 16-byte aligned, so a group of four lies on its own size.
template <bool kFull>
__device__ __forceinline__ void load4(const void* base, int type, int64_t i, int64_t n, float2* x) {
    if (kFull || i + 4 <= n) {
        if (!inside<kChkAdamw>(n, i, 4)) {
            x[0] = x[1] = make_float2(0.f, 0.f);
        } else if (type == kF32) {
            const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
            x[0] = make_float2(q.x, q.y);
            x[1] = make_float2(q.z, q.w);
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
            x[0] = unpack(q.x, type);
            x[1] = unpack(q.y, type);
        }
    } else {
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            y[k] = 0.f;
            if (i + k < n && inside<kChkAdamw>(n, i + k, 1)) {
                if (type == kF32) y[k] = static_cast<const float*>(base)[i + k];
                else y[k] = unpack(static_cast<const uint16_t*>(base)[i + k], type).x;
            }
        }
        x[0] = make_float2(y[0], y[1]);
        x[1] = make_float2(y[2], y[3]);
    }
}

template <bool kFull>
__device__ __forceinline__ void store4(void* base, int type, int64_t i, int64_t n, const float2* x) {
    if (kFull || i + 4 <= n) {
        if (!inside<kChkAdamw>(n, i, 4)) return;
        if (type == kF32)
            *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) =
                make_uint2(pack(x[0].x, x[0].y, type), pack(x[1].x, x[1].y, type));
    } else {
        const float y[4] = {x[0].x, x[0].y, x[1].x, x[1].y};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n && inside<kChkAdamw>(n, i + k, 1)) {
                if (type == kF32) static_cast<float*>(base)[i + k] = y[k];
                else static_cast<uint16_t*>(base)[i + k] = (uint16_t)pack(y[k], 0.f, type);
            }
    }
}

template <bool kFull>
__device__ __forceinline__ uint32_t load_codes(const void* base, int64_t i, int64_t n) {
    const uint8_t* c = static_cast<const uint8_t*>(base);
    uint32_t w = 0;
    if (kFull || i + 4 <= n) {
        if (inside<kChkAdamw>(n, i, 4)) w = *reinterpret_cast<const uint32_t*>(c + i);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n && inside<kChkAdamw>(n, i + k, 1)) w |= (uint32_t)c[i + k] << (8 * k);
    }
    return w;
}

template <bool kFull>
__device__ __forceinline__ void store_codes(void* base, int64_t i, int64_t n, uint32_t w) {
    uint8_t* c = static_cast<uint8_t*>(base);
    if (kFull || i + 4 <= n) {
        if (inside<kChkAdamw>(n, i, 4)) *reinterpret_cast<uint32_t*>(c + i) = w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n && inside<kChkAdamw>(n, i + k, 1)) c[i + k] = (uint8_t)(w >> (8 * k));
    }
}

// The two e4m3 codes in the low half of w, without their scale.
__device__ __forceinline__ float2 decode2(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    return __half22float2(__half2(h));
}

// Pairs of fp32 operations, each rounded to nearest. Sums stay single: a packed product followed by
// a packed sum came out contracted (one rounding less than the states' definition has).
__device__ __forceinline__ uint64_t pair(float2 a) { return (uint64_t)__float_as_uint(a.y) << 32 | __float_as_uint(a.x); }
__device__ __forceinline__ float2 unpair(uint64_t a) {
    return make_float2(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)));
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)));
    return unpair(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
    return unpair(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, both(-1.f), a); }  // one rounding

// The e4m3 code of y in [0, 448], rounded up with the probability of the part cut off (`up` of 2^20
// parts of a code are added and the rest cut). Times 2^-120, e4m3's smallest normal number is
// fp32's, and the code is the top of the float's bits, subnormal codes included.
__device__ __forceinline__ uint32_t stochastic_code(float y, uint32_t up) {
    return (__float_as_uint(__fmul_rn(fminf(fabsf(y), kTop), 0x1p-120f)) + up) >> 20;
}

__device__ __forceinline__ float reciprocal(float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}

// The largest finite magnitude of a 256-element block, 4 x 2 of whose values are this lane's. `finite`:
// nothing else is among them.
__device__ __forceinline__ float block_top(const float2 (&x)[4], bool& finite) {
    const float inf = __uint_as_float(0x7f800000u);
    float top = 0.f;
    float2 spoiled = both(0.f);  // stays 0 while everything is finite
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        top = fmaxf(fmaxf(top, fabsf(x[a].x)), fabsf(x[a].y));
        spoiled = fma2(x[a], both(0.f), spoiled);
    }
    finite = !__any_sync(0xffffffffu, !(spoiled.x + spoiled.y == 0.f));
    if (!finite) {
        top = 0.f;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (fabsf(x[a].x) < inf) top = fmaxf(top, fabsf(x[a].x));
            if (fabsf(x[a].y) < inf) top = fmaxf(top, fabsf(x[a].y));
        }
    }
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // magnitudes order as their bits do
}

// Codes of the lane's values times `inverse` = 448 / their block's top. kRoot: the values are
// square roots, and a positive one is coded as 2^-9 at least.
template <bool kRoot>
__device__ __forceinline__ void encode(const float2 (&x)[4], const uint32_t (&h)[8], bool nearest, float inverse, bool finite,
                                       uint32_t (&w)[2]) {
    const float inf = __uint_as_float(0x7f800000u);
    uint32_t c[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        float2 y = mul2(x[a], both(inverse));
        if (nearest) {
            if (kRoot) y = make_float2(fmaxf(y.x, x[a].x > 0.f ? 0x1p-9f : 0.f), fmaxf(y.y, x[a].y > 0.f ? 0x1p-9f : 0.f));
            c[a] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
        } else {
            uint32_t c0 = stochastic_code(y.x, ((kRoot ? h[2 * a] >> 12 : h[2 * a] << 4) & 0xffff0u) | 8u);
            uint32_t c1 = stochastic_code(y.y, ((kRoot ? h[2 * a + 1] >> 12 : h[2 * a + 1] << 4) & 0xffff0u) | 8u);
            if (kRoot) {
                c0 = max(c0, min(__float_as_uint(x[a].x), 1u));
                c1 = max(c1, min(__float_as_uint(x[a].y), 1u));
            } else {
                c0 |= __float_as_uint(y.x) >> 24 & 0x80u;
                c1 |= __float_as_uint(y.y) >> 24 & 0x80u;
            }
            c[a] = c0 | c1 << 8;
        }
        if (!finite) {
            if (!(fabsf(x[a].x) < inf)) c[a] = (c[a] & 0xff00u) | 0x7fu;
            if (!(fabsf(x[a].y) < inf)) c[a] = (c[a] & 0xffu) | 0x7f00u;
        }
    }
    w[0] = __byte_perm(c[0], c[1], 0x5410);
    w[1] = __byte_perm(c[2], c[3], 0x5410);
}

struct Rates {
    float c1, root2;  // 1/(1-b1^t), sqrt(1/(1-b2^t))
    uint32_t step;
};

// One 256-element block. kP, kG, kS: the types of parameter, gradient and states where the compiler
// may know them (-1: only the list does); kFull: the block lies wholly inside the tensor.
template <int kP, int kG, int kS, bool kFull>
__device__ __forceinline__ void step_block(const Tensor& T, const Params& a, const Rates& r, int64_t blk, int lane) {
    const int tp = kP >= 0 ? kP : (int)(T.types & 15), tg = kG >= 0 ? kG : (int)(T.types >> 4 & 15),
              ts = kS >= 0 ? kS : (int)(T.types >> 8 & 15), tc = (int)(T.types >> 12 & 15);
    const int64_t base = blk * kBlock;
    const int64_t n = T.n;
    const int64_t at[2] = {base + 4 * lane, base + 128 + 4 * lane};
    float2 p[4], g[4], m[4], v[4], root[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        load4<kFull>(T.g, tg, at[k], n, g + 2 * k);
        load4<kFull>(T.p, tp, at[k], n, p + 2 * k);
    }
    if (ts == kF32) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            load4<kFull>(T.m, kF32, at[k], n, m + 2 * k);
            load4<kFull>(T.v, kF32, at[k], n, v + 2 * k);
        }
    } else {
        const float ms = T.ms[blk], vs = T.vs[blk];
        uint32_t cm[2], cv[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            cm[k] = load_codes<kFull>(T.m, at[k], n);
            cv[k] = load_codes<kFull>(T.v, at[k], n);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m[k] = mul2(decode2(cm[k >> 1] >> 16 * (k & 1)), both(ms));
            v[k] = mul2(decode2(cv[k >> 1] >> 16 * (k & 1)), both(vs));
            v[k] = mul2(v[k], v[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m[k] = add2(mul2(m[k], both(a.b1)), mul2(g[k], both(a.o1)));
        v[k] = add2(mul2(v[k], both(a.b2)), mul2(mul2(g[k], g[k]), both(a.o2)));
        // correctly rounded, since v's codes follow from it: an approximate root was 4% faster with 8-bit states, and put one code
        // in 10^5 beside its place
        root[k] = make_float2(__fsqrt_rn(v[k].x), __fsqrt_rn(v[k].y));
        const float2 d = add2(mul2(root[k], both(r.root2)), both(a.eps)), s = mul2(m[k], both(r.c1));
        // the quotient alone is not correctly rounded (2 ulp of a step): a division in full costs a tenth of an 8-bit step
        p[k] = sub2(mul2(p[k], both(T.keep)), mul2(both(T.rate), mul2(s, make_float2(reciprocal(d.x), reciprocal(d.y)))));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        store4<kFull>(T.p, tp, at[k], n, p + 2 * k);
        if (tc != kNone) store4<kFull>(T.copy, tc, at[k], n, p + 2 * k);
        if (a.zero_grad) {
            const float2 z[2] = {};
            store4<kFull>(T.g, tg, at[k], n, z);
        }
    }
    if (ts == kF32) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            store4<kFull>(T.m, kF32, at[k], n, m + 2 * k);
            store4<kFull>(T.v, kF32, at[k], n, v + 2 * k);
        }
        return;
    }
    uint32_t h[8] = {}, w[2];
    const bool nearest = a.seed == 0;
    if (!nearest) {
        const uint32_t key = probe::mix32(a.seed * 0x9E3779B1u + r.step * 0x85EBCA77u + (T.types >> 16) * 0xC2B2AE3Du +
                                          (uint32_t)((uint64_t)base >> 32) * 0x27D4EB2Fu);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = probe::mix32(((uint32_t)at[k >> 2] + (k & 3)) ^ key);
    }
    bool mf, vf;
    const float mt = block_top(m, mf), vt = block_top(root, vf);
    // One division a lane gives all four quotients: lane 0 and 1 the scale and the inverse of m, 2 and 3 of
    // v. A block whose inverse could overflow is stored as zeros.
    const float t = lane & 2 ? vt : mt;
    float q = __fdiv_rn(lane & 1 ? kTop : t, lane & 1 ? t : kTop);
    if ((lane & 1) && !(t > 0x1p-100f)) q = 0.f;
    encode<false>(m, h, nearest, __shfl_sync(0xffffffffu, q, 1), mf, w);
    store_codes<kFull>(T.m, at[0], n, w[0]);
    store_codes<kFull>(T.m, at[1], n, w[1]);
    encode<true>(root, h, nearest, __shfl_sync(0xffffffffu, q, 3), vf, w);
    store_codes<kFull>(T.v, at[0], n, w[0]);
    store_codes<kFull>(T.v, at[1], n, w[1]);
    if (lane == 0) T.ms[blk] = q;
    if (lane == 2) T.vs[blk] = q;
}

template <int kCap>
__global__ void __launch_bounds__(32 * kWarps, 4) step_kernel(const __grid_constant__ List<kCap> list, const Params a) {
    const int lane = threadIdx.x & 31;
    const uint32_t b = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (b >= list.blocks) return;
    uint32_t lo = list.where.tensor[b >> list.where.shift], hi = list.where.tensor[(b >> list.where.shift) + 1] + 1u;
    // the last tensor whose first block is at most b: lo or one up to, not including, hi
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (list.first[mid] <= b) lo = mid; else hi = mid;
    }
    after_previous_kernel();
    Rates r{a.c1, a.root2, a.step};
    if (a.device_step != nullptr) {
        const int64_t t = *a.device_step;
        if (t < 1) return;
        r.step = (uint32_t)t;
        r.c1 = (float)(1.0 / (1.0 - pow(a.db1, (double)t)));
        r.root2 = (float)sqrt(1.0 / (1.0 - pow(a.db2, (double)t)));
    }
    const Tensor& T = list.t[lo];
    const int64_t blk = b - list.first[lo];
    if ((blk + 1) * kBlock > T.n) return step_block<-1, -1, -1, false>(T, a, r, blk, lane);
    switch (T.types & 0xfffu) {
#define HG_ADAMW_CASE(P, G, S) \
    case P | G << 4 | S << 8: return step_block<P, G, S, true>(T, a, r, blk, lane);
        HG_ADAMW_CASE(kF32, kF32, kF32)
        HG_ADAMW_CASE(kF32, kBf16, kF32)
        HG_ADAMW_CASE(kBf16, kBf16, kF32)
        HG_ADAMW_CASE(kF16, kF16, kF32)
        HG_ADAMW_CASE(kF32, kF32, kE4m3)
        HG_ADAMW_CASE(kF32, kBf16, kE4m3)
        HG_ADAMW_CASE(kBf16, kBf16, kE4m3)
        HG_ADAMW_CASE(kF16, kF16, kE4m3)
#undef HG_ADAMW_CASE
    }
    step_block<-1, -1, -1, true>(T, a, r, blk, lane);  // rarer pairs of types
}

}  // namespace adamw
}  // namespace hg
