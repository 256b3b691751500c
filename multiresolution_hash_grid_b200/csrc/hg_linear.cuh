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

#include <type_traits>

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

// Pairs of fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float2 a) { return (uint64_t)__float_as_uint(a.y) << 32 | __float_as_uint(a.x); }
__device__ __forceinline__ float2 unpair(uint64_t a) {
    return make_float2(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)));
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
    return unpair(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)));
    return unpair(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)));
    return unpair(d);
}
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float2 rcp2(float2 a) { return make_float2(rcp_approx(a.x), rcp_approx(a.y)); }

// The activations come without branches and two at a time, since a layer's output passes through
// one warp instruction after another while the tensor cores wait for its accumulator.
//
// GELU z Phi(z): with the upper tail Q(|z|) = 1 - Phi(|z|) it is max(z, 0) - |z| Q(|z|). Q by Abramowitz
// and Stegun 7.1.26: erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + 0.3275911 x), off by at
// most 1.5e-7, which is 7.5e-8 |z| here, 1.3 half steps of fp32. `e` gives exp(-z^2 / 2).
__device__ __forceinline__ float2 upper_tail(float2 a, float2& e) {
    const float2 s = mul2(mul2(a, a), both(-0.72134752f));  // -a^2 / 2 in powers of two
    e = make_float2(exp2_approx(s.x), exp2_approx(s.y));
    const float2 t = rcp2(fma2(a, both(0.23164190f), both(1.f)));
    float2 q = fma2(t, both(0.5307027145f), both(-0.7265760135f));
    q = fma2(q, t, both(0.7107068705f));
    q = fma2(q, t, both(-0.142248368f));
    q = fma2(q, t, both(0.127414796f));
    return mul2(mul2(q, t), e);
}
__device__ __forceinline__ float2 magnitude(float2 z) { return make_float2(fabsf(z.x), fabsf(z.y)); }

__device__ __forceinline__ float2 gelu2(float2 z) {
    float2 e;
    const float2 a = make_float2(fminf(fabsf(z.x), 64.f), fminf(fabsf(z.y), 64.f));  // Q is 0 there, and 0 times infinity none
    const float2 q = upper_tail(a, e);
    return fma2(make_float2(-a.x, -a.y), q, make_float2(z.x > 0.f ? z.x : z.x != z.x ? z.x : 0.f, z.y > 0.f ? z.y : z.y != z.y ? z.y : 0.f));
}
// 1 / (1 + exp(-z)); exp2's argument is rounded, which costs |z| 2^-24.
__device__ __forceinline__ float2 sigmoid2(float2 z) {
    const float2 s = mul2(z, both(-1.44269504f));
    return rcp2(add2(make_float2(exp2_approx(s.x), exp2_approx(s.y)), both(1.f)));
}

// kN values, kN even.
template <int kN>
__device__ __forceinline__ void activate(float (&y)[kN], int act) {
    switch (act) {
        case kRelu:
#pragma unroll
            for (int j = 0; j < kN; ++j) asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(y[j]));  // a NaN stays one
            break;
        case kGelu:
#pragma unroll
            for (int j = 0; j < kN; j += 2) {
                const float2 r = gelu2(make_float2(y[j], y[j + 1]));
                y[j] = r.x;
                y[j + 1] = r.y;
            }
            break;
        case kSilu:
#pragma unroll
            for (int j = 0; j < kN; j += 2) {
                const float2 z = make_float2(y[j], y[j + 1]), r = mul2(z, sigmoid2(z));
                y[j] = r.x;
                y[j + 1] = r.y;
            }
            break;
    }
}

// z within +-bound: the slopes are 0 or 1 to the last place there, where an infinite z (one that overflowed its 16 bits)
// would make 0 times infinity. A NaN stays one.
__device__ __forceinline__ float2 within(float2 z, float bound) {
    return make_float2(z.x > bound ? bound : z.x < -bound ? -bound : z.x, z.y > bound ? bound : z.y < -bound ? -bound : z.y);
}

// d[j] act'(z[j]). GELU: Phi(z) + z phi(z); SILU: s (1 + z (1 - s)).
template <int kN>
__device__ __forceinline__ void times_slope(float (&d)[kN], const float (&z)[kN], int act) {
    switch (act) {
        case kRelu:
#pragma unroll
            for (int j = 0; j < kN; ++j) d[j] = z[j] <= 0.f ? 0.f : d[j];  // at a NaN the gradient, a NaN itself, goes on
            break;
        case kGelu:
#pragma unroll
            for (int j = 0; j < kN; j += 2) {
                const float2 v = within(make_float2(z[j], z[j + 1]), 64.f), a = magnitude(v);
                float2 e;
                const float2 q = upper_tail(a, e);
                const float2 cdf = make_float2(v.x > 0.f ? 1.f - q.x : q.x, v.y > 0.f ? 1.f - q.y : q.y);
                const float2 s = fma2(mul2(v, both(0.39894228f)), e, cdf);
                d[j] *= s.x;
                d[j + 1] *= s.y;
            }
            break;
        case kSilu:
#pragma unroll
            for (int j = 0; j < kN; j += 2) {
                const float2 v = within(make_float2(z[j], z[j + 1]), 80.f), s = sigmoid2(v);
                const float2 r = mul2(s, fma2(v, fma2(s, both(-1.f), both(1.f)), both(1.f)));
                d[j] *= r.x;
                d[j + 1] *= r.y;
            }
            break;
    }
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

__device__ __forceinline__ float bias1(const Epilogue& e, int64_t col) {
    return e.bias != nullptr && in_bounds<kChkBias>(e.bias + col, 4) ? __ldg(e.bias + col) : 0.f;
}

template <typename T>
__device__ __forceinline__ float residual1(const Epilogue& e, int64_t row, int64_t col) {
    if (e.residual == nullptr) return 0.f;
    if (e.out_f32) {
        const float* r = static_cast<const float*>(e.residual) + row * e.ldr + col;
        return in_bounds<kChkResidual>(r, 4) ? *r : 0.f;
    }
    const T* r = static_cast<const T*>(e.residual) + row * e.ldr + col;
    return in_bounds<kChkResidual>(r, sizeof(T)) ? to_float(*r) : 0.f;
}

template <typename T>
__device__ __forceinline__ void store_z1(const Epilogue& e, int64_t row, int64_t col, float z) {
    T* p = static_cast<T*>(e.z) + row * e.ldz + col;
    if (in_bounds<kChkZ>(p, sizeof(T))) *p = from_float<T>(z);
}

template <typename T>
__device__ __forceinline__ void store_y1(const Epilogue& e, void* out, int64_t row, int64_t col, float y) {
    if (e.out_f32) {
        float* p = static_cast<float*>(out) + row * e.ldo + col;
        if (in_bounds_role(e.role, p, 4)) *p = y;
    } else {
        T* p = static_cast<T*>(out) + row * e.ldo + col;
        if (in_bounds_role(e.role, p, sizeof(T))) *p = from_float<T>(y);
    }
}

// Where value (row, column) of a 32 x 32 chunk of floats lies: 16-byte units of a row are exchanged by
// its number, so that both a lane that writes a row and four lanes that read one meet no bank twice.
__device__ __forceinline__ int unit_of(int row, int unit) { return row * 8 + (unit ^ (row & 7)); }

__device__ __forceinline__ void bias8(const Epilogue& e, int64_t col, float (&b)[8]) {
    if (e.bias == nullptr || !in_bounds<kChkBias>(e.bias + col, 32)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = 0.f;
        return;
    }
    const float4 lo = __ldg(reinterpret_cast<const float4*>(e.bias + col)), hi = __ldg(reinterpret_cast<const float4*>(e.bias + col + 4));
    b[0] = lo.x; b[1] = lo.y; b[2] = lo.z; b[3] = lo.w;
    b[4] = hi.x; b[5] = hi.y; b[6] = hi.z; b[7] = hi.w;
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float* y) {
    return make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
}

// The nearest finite numbers of type T (a NaN stays one).
template <typename T> __device__ __forceinline__ uint32_t pack2_finite(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2_finite<__half>(float a, float b) {
    uint32_t w;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
template <> __device__ __forceinline__ uint32_t pack2_finite<__nv_bfloat16>(float a, float b) {
    uint32_t w;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
// d as the sum of two numbers of type T, each the nearest to what is left: off by the square of a rounding of T. The high
// one is finite, so that a d beyond T's range is not an infinity less an infinity; an infinite d is so in the low one.
template <typename T>
__device__ __forceinline__ uint32_t split2(float a, float b, uint32_t& low) {
    const uint32_t high = pack2_finite<T>(a, b);
    const float2 rest = fma2(unpack2<T>(high), both(-1.f), make_float2(a, b));
    low = pack2<T>(rest.x, rest.y);
    return high;
}
template <typename T>
__device__ __forceinline__ uint4 split8(const float* d, uint4& low) {
    uint4 high;
    high.x = split2<T>(d[0], d[1], low.x);
    high.y = split2<T>(d[2], d[3], low.y);
    high.z = split2<T>(d[4], d[5], low.z);
    high.w = split2<T>(d[6], d[7], low.w);
    return high;
}

// kRows rows (row, row + 8, ...) of eight neighbouring values, bias already added, in 16-byte
// vectors. Rows from `rows` on are not there. q: the 16-bit residuals, if there are any.
template <typename T, int kRows>
__device__ __forceinline__ void emit_vectors(const Epilogue& e, void* out, int64_t row, int64_t rows, int64_t col, float (&y)[kRows][8],
                                             const uint4 (&q)[kRows]) {
    if (e.z != nullptr) {
        T* p = static_cast<T*>(e.z) + row * e.ldz + col;
#pragma unroll
        for (int r = 0; r < kRows; ++r, p += 8 * e.ldz)
            if (row + 8 * r < rows && in_bounds<kChkZ>(p, 16)) *reinterpret_cast<uint4*>(p) = pack8<T>(y[r]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) activate(y[r], e.act);
    if (e.out_f32) {
        if (e.residual != nullptr) {
            const float* p = static_cast<const float*>(e.residual) + row * e.ldr + col;
#pragma unroll
            for (int r = 0; r < kRows; ++r, p += 8 * e.ldr)
                if (row + 8 * r < rows && in_bounds<kChkResidual>(p, 32)) {
                    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
                    y[r][0] += a.x; y[r][1] += a.y; y[r][2] += a.z; y[r][3] += a.w;
                    y[r][4] += b.x; y[r][5] += b.y; y[r][6] += b.z; y[r][7] += b.w;
                }
        }
        float* p = static_cast<float*>(out) + row * e.ldo + col;
#pragma unroll
        for (int r = 0; r < kRows; ++r, p += 8 * e.ldo)
            if (row + 8 * r < rows && in_bounds_role(e.role, p, 32)) {
                *reinterpret_cast<float4*>(p) = make_float4(y[r][0], y[r][1], y[r][2], y[r][3]);
                *reinterpret_cast<float4*>(p + 4) = make_float4(y[r][4], y[r][5], y[r][6], y[r][7]);
            }
        return;
    }
    if (e.residual != nullptr) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float2 a = unpack2<T>(q[r].x), b = unpack2<T>(q[r].y), c = unpack2<T>(q[r].z), d = unpack2<T>(q[r].w);
            y[r][0] += a.x; y[r][1] += a.y; y[r][2] += b.x; y[r][3] += b.y;
            y[r][4] += c.x; y[r][5] += c.y; y[r][6] += d.x; y[r][7] += d.y;
        }
    }
    T* p = static_cast<T*>(out) + row * e.ldo + col;
#pragma unroll
    for (int r = 0; r < kRows; ++r, p += 8 * e.ldo)
        if (row + 8 * r < rows && in_bounds_role(e.role, p, 16)) *reinterpret_cast<uint4*>(p) = pack8<T>(y[r]);
}

// The 16-bit residuals of kRows rows of eight neighbouring values.
template <typename T, int kRows>
__device__ __forceinline__ void load_residuals(const Epilogue& e, int64_t row, int64_t rows, int64_t col, uint4 (&q)[kRows]) {
    const T* p = static_cast<const T*>(e.residual) + row * e.ldr + col;
#pragma unroll
    for (int r = 0; r < kRows; ++r, p += 8 * e.ldr)
        q[r] = row + 8 * r < rows && in_bounds<kChkResidual>(p, 16) ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
}

// Eight rows of a column, bias already added. kFull: all of them are there. What depends on the call alone
// is decided once for all eight, so that their loads go out together.
template <typename T, bool kFull>
__device__ __forceinline__ void emit_column8(const Epilogue& e, void* out, int64_t row, int rows, int64_t col, float (&y)[8]) {
    float res[8] = {};
    if (e.residual != nullptr) {
        if (e.out_f32) {
            const float* p = static_cast<const float*>(e.residual) + row * e.ldr + col;
#pragma unroll
            for (int k = 0; k < 8; ++k, p += e.ldr)
                if ((kFull || k < rows) && in_bounds<kChkResidual>(p, 4)) res[k] = *p;
        } else {
            const T* p = static_cast<const T*>(e.residual) + row * e.ldr + col;
            T raw[8] = {};
#pragma unroll
            for (int k = 0; k < 8; ++k, p += e.ldr)
                if ((kFull || k < rows) && in_bounds<kChkResidual>(p, sizeof(T))) raw[k] = *p;
#pragma unroll
            for (int k = 0; k < 8; ++k) res[k] = to_float(raw[k]);
        }
    }
    if (e.z != nullptr) {
        T* p = static_cast<T*>(e.z) + row * e.ldz + col;
#pragma unroll
        for (int k = 0; k < 8; ++k, p += e.ldz)
            if ((kFull || k < rows) && in_bounds<kChkZ>(p, sizeof(T))) *p = from_float<T>(y[k]);
    }
    activate(y, e.act);
    if (e.out_f32) {
        float* p = static_cast<float*>(out) + row * e.ldo + col;
#pragma unroll
        for (int k = 0; k < 8; ++k, p += e.ldo)
            if ((kFull || k < rows) && in_bounds_role(e.role, p, 4)) *p = y[k] + res[k];
    } else {
        T* p = static_cast<T*>(out) + row * e.ldo + col;
#pragma unroll
        for (int k = 0; k < 8; ++k, p += e.ldo)
            if ((kFull || k < rows) && in_bounds_role(e.role, p, sizeof(T))) *p = from_float<T>(y[k] + res[k]);
    }
}

// ---------------------------------------------------------------------------------------
// The product D[m][n] = sum_k A(m, k) B(n, k) on the tensor cores: tcgen05.mma of 128 x bn x 16,
// or of 256 x bn x 16 by a pair of SMs, with the accumulator in tensor memory.
//
// An operand is a row-major array with k along its rows ("k-major": x and W of the forward
// product) or along its columns ("mn-major": W in dx = dz W, dz and x in dW = dz^T x); the
// tensor cores take both, so nothing is transposed in memory. TMA stages it 64 values of k at
// a time in the 128-byte-swizzled layout: rows of 64 contiguous elements (128 bytes), eight to a
// 1024-byte group, 16-byte chunk c of row r at chunk c ^ (r % 8). K-major: a row of it is an m (or
// n) and holds 64 k. Mn-major: a row is a k and holds 64 m, one such box per 64 m. Rows of A that the
// product does not have are not staged; the MMA then multiplies what lies there, and those
// rows of the accumulator are not read. Where one column tile covers all of N and B is small, B is
// staged once and stays.
//
// Warps: 0-7 read finished accumulators (two for each quarter of the 128 TMEM lanes, taking
// turns at 32-column chunks), 8 issues the MMAs, 9 the TMA copies. Two accumulators alternate,
// so that the next tile's MMAs run while the last one is written out. Persistent over tiles, n
// fastest.
//
// A pair (kPair) computes 256 x bn: each block stages its own 128 rows of A and half of B, which
// halves the shared-memory reads of B per MMA and leaves room for more stages; the first block
// issues the MMAs of both, and each writes out its own 128 rows.
//
// Long sums (kGather): the tensor cores' additions cut off instead of rounding, which for random operands
// loses 1.1e-9 of the result for each k (measured: 9.1e-6 for K = 8192, where plain fp32 has 9.6e-7, and 5.3e-4 for
// K = 2^19). So every kSegment steps the accumulator is added to fp32 registers and begins again, where the
// result is fp32, or where a 16-bit one sums more than kSegment16 steps: what those lose, 5e-5, is a
// tenth of fp16's half step, and gathering takes one block an SM instead of two.
//
// Way out: a lane reads 32 columns of its row from TMEM, adds bias, applies the activation and adds
// the residual in fp32, and rounds. Where rows begin on 16-byte boundaries (kVectors) the chunk of 32 x 32
// goes to 4 KB of shared memory a warp, and from there by TMA, which also keeps to the array's bounds: a
// third of the instructions that 16-byte stores with their addresses and guards took (2^20 x 32 ->
// 64: 71 us with those). Otherwise it passes through shared memory as fp32, and a lane takes
// a column, so that a warp still writes 32 neighbours at a time.
// ---------------------------------------------------------------------------------------
constexpr int kBm = 128, kBk = 64;
constexpr int kOutWarps = 8;
constexpr int kThreads = 32 * (kOutWarps + 2);
constexpr int kMaxStages = 16;
constexpr int kSegment16 = 768;
constexpr int kSegment = 12;  // 64-wide steps of K (16 took it to the 1e-6 of plain fp32 sums, 12 leaves a quarter of room)
constexpr int kStaging = kOutWarps * 32 * 32 * 4;

// How long the warps of a kernel wait. The checked build can make the nth wait of a role give up at once, in the
// blocks of one parity or (2) in all.
struct Patience {
    uint32_t polls;
#ifdef HASHGRID_CHECKED
    int role, nth, parity;
#endif
};
enum Role { kCopies = 1, kMmas = 2, kOut = 3, kSlopes = 4 };

struct Side {             // one operand's share of a stage: `boxes` boxes of box_rows x 64 elements
    int mn;               // k runs along the array's columns
    int box_rows, boxes;
    int bytes;            // of all boxes, what TMA delivers (a multiple of 1024)
};

struct Gemm {
    CUtensorMap ta, ta_low, tb, ty, tz;
    Side a, b;
    int64_t M, N;
    int bn, columns;      // tile width; columns from one accumulator to the next
    int stages, stage_bytes;
    int resident;         // B is staged once, behind the stages
    int cluster;          // blocks that share a tile's K (their shares meet in shared memory), or 1
    int kblocks, kblocks_per_split;
    int kfold;            // steps from here on multiply A's low part (ta_low) by B once more; kblocks where A has none
    int mt, nt;
    int blocks;           // blocks (or pairs) that take turns at the tiles of a split
    uint32_t idesc, tmem_columns;
    Epilogue e;
    int64_t split_stride; // elements of fp32 output from one split to the next
    int* status;
};

// One launch computes one product or two that do not depend on each other (dx and dW): blocks from
// `second` on take the second.
// (Blocks with more than 64 columns of tensor memory take 100 KB of shared memory or more, so that two of them share an
// SM at most, and have 256 columns at most where two can; the others take 66 KB or more. So the columns of the
// blocks on an SM always fit, and no block waits for another launch's while its own cluster waits for it.)
struct Gemms {
    Gemm of[2];
    int second;
    Patience patience;
};

__host__ __device__ constexpr size_t gemm_smem(int stage_bytes_in_all, bool two = false) {
    return 1024 + (size_t)stage_bytes_in_all + (two ? 2 : 1) * kStaging + (2 * kMaxStages + 6) * 8 + 16;
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// Into this block's memory, with the arrival counted by a barrier of the pair's first block.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc));
}
// Arrives at the barrier of the same address in both blocks once the MMAs so far are done.
__device__ __forceinline__ void commit_pair(uint32_t mbar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(mbar),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void arrive_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}\n" ::"r"(bar), "r"(bytes) : "memory");
}
// Counts `bytes` as copied that nothing will copy any more.
__device__ __forceinline__ void count_copied(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t cluster_address(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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

// A warp's waits.
struct Waits {
    volatile int* abort_flag;  // of the block
    uint32_t polls;
#ifdef HASHGRID_CHECKED
    int left;
#endif
    __device__ __forceinline__ Waits(volatile int* flag, const Patience& p, Role role) : abort_flag(flag), polls(p.polls) {
#ifdef HASHGRID_CHECKED
        left = p.role == role && (p.parity == 2 || p.parity == (int)(blockIdx.x & 1u)) ? p.nth : 0;
#else
        (void)role;
#endif
    }
};

// A bounded wait of a whole warp, which also ends once another role of the block has given up. All lanes get the
// same answer, false if any of them gave up, and none goes on before the others: a lane that fell behind by two
// phases of a barrier would wait for a parity that had passed, and lanes that disagreed would part for good. A block
// of a pair (kPair) tells the other one that it gave up.
template <bool kPair>
__device__ __forceinline__ bool warp_waits(uint32_t bar, uint32_t parity, Waits& w) {
    uint32_t done = 0, polls = w.polls;
#ifdef HASHGRID_CHECKED
    if (w.left > 0 && --w.left == 0) polls = 0;
#endif
    for (uint32_t it = 0; it < polls; ++it) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done || ((it & 255u) == 255u && *w.abort_flag != 0)) break;
    }
    const bool all = __all_sync(0xffffffffu, done);
    if (!all) {
        *w.abort_flag = 1;
        if (kPair) {
            uint32_t rank;
            asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
            asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(
                             cluster_address((uint32_t)__cvta_generic_to_shared(const_cast<int*>(w.abort_flag)), rank ^ 1u)),
                         "r"(1)
                         : "memory");
        }
    }
    return all;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}

// Stores a chunk from shared memory; the thread then commits its stores as a group.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map), "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A lane's row of a chunk (32 values) into the warp's 4 KB: 16-bit rows of 64 bytes, whose 16-byte units are
// exchanged by (row / 2) % 4 (the 64-byte swizzle), fp32 rows of 128 bytes, by row % 8.
template <typename T>
__device__ __forceinline__ void stage_row16(uint8_t* st, int lane, const float (&y)[32]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) *reinterpret_cast<uint4*>(st + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) = pack8<T>(y + 8 * u);
}
__device__ __forceinline__ void stage_row32(uint8_t* st, int lane, const float (&y)[32]) {
#pragma unroll
    for (int u = 0; u < 8; ++u)
        *reinterpret_cast<float4*>(st + lane * 128 + ((u ^ (lane & 7)) << 4)) = make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
}

// The status word may be the host's memory.
__device__ __forceinline__ void report_given_up(int* status) {
    if (status == nullptr) return;
    *static_cast<volatile int*>(status) = 1;
    __threadfence_system();
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

// The tiles of a block (or pair), n fastest, without a division a tile.
struct Tiles {
    int m, n, dm, dn, mt, nt;
    __device__ __forceinline__ Tiles(const Gemm& g, int first, int step)
        : m(first / g.nt), n(first % g.nt), dm(step / g.nt), dn(step % g.nt), mt(g.mt), nt(g.nt) {}
    __device__ __forceinline__ bool more() const { return m < mt; }
    __device__ __forceinline__ void next() {
        m += dm;
        n += dn;
        if (n >= nt) {
            n -= nt;
            ++m;
        }
    }
};

__device__ __forceinline__ float4 cluster_load(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t cluster_load64(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

template <typename T, bool kPair, bool kVectors, bool kGather>
__global__ void __launch_bounds__(kThreads, kPair || kGather ? 1 : 2) gemm_kernel(const __grid_constant__ Gemms list) {
    const int which = (int)blockIdx.x >= list.second;
    const Gemm& g = list.of[which];
    const int block = (int)blockIdx.x - (which ? list.second : 0);
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    const int kept = g.resident ? g.kfold * g.b.bytes : 0;
    uint8_t* staging = sm + (size_t)g.stages * g.stage_bytes + kept;
    uint64_t* bars = reinterpret_cast<uint64_t*>(staging + (g.e.out_f32 && g.e.z != nullptr ? 2 : 1) * kStaging);  // fp32 y and z side by side
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 6);
    __shared__ volatile int abort_flag;
    __shared__ uint64_t copies_issued;  // stages that the copying warp filled
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // the shuffle tells the compiler that it is uniform
    const uint32_t sm0 = (uint32_t)__cvta_generic_to_shared(sm), bar0 = (uint32_t)__cvta_generic_to_shared(bars);
    const uint32_t sb0 = sm0 + g.stages * g.stage_bytes;  // B, where it stays
    // barriers: full[stage], empty[stage], accumulator done[2], accumulator free[2], B staged, drain
    const uint32_t full = bar0, empty = bar0 + 8 * kMaxStages, done = empty + 8 * kMaxStages, room = done + 16, bfull = room + 16,
                   drain = bfull + 8;
    const uint32_t rank = kPair ? block & 1u : 0u;
    if (threadIdx.x == 32 * (kOutWarps + 1)) {
        abort_flag = 0;
        for (int s = 0; s < g.stages; ++s) {
            mlp::mbar_init(full + 8 * s, 1);
            mlp::mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mlp::mbar_init(done + 8 * i, 1);
            mlp::mbar_init(room + 8 * i, kPair ? 2 * kOutWarps : kOutWarps);
        }
        mlp::mbar_init(bfull, 1);
        mlp::mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        const uint32_t slot = (uint32_t)__cvta_generic_to_shared(tslot);
        if (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(g.tmem_columns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(g.tmem_columns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    mlp::fence_before();
    __syncthreads();
    if (kPair) cluster_sync();  // the other block's barriers and tensor memory are there
    mlp::fence_after();
    after_previous_kernel();
    const uint32_t tmem = *tslot;
    const int first = kPair ? block >> 1 : g.cluster > 1 ? block / g.cluster : block % g.blocks, step = g.blocks;
    const int part = kPair ? 0 : g.cluster > 1 ? block % g.cluster : block / g.blocks;  // of K
    const int kb0 = part * g.kblocks_per_split, kbs = max(0, min(g.kblocks_per_split, g.kblocks - kb0));

    if (warp == kOutWarps + 1) {
        // ------------------------------- TMA copies -------------------------------
        // (as in the MMA warp, all lanes walk and one issues)
        Waits waits(&abort_flag, list.patience, kCopies);
        const bool issues = elect_one();
        const uint32_t bytes = g.a.bytes + (g.resident ? 0 : g.b.bytes);
        if (g.resident && kbs > 0 && issues) {
            arrive_expect(bfull, kept);
            for (int kb = 0; kb < g.kfold; ++kb)
                for (int j = 0; j < g.b.boxes; ++j)
                    tma_load(sb0 + kb * g.b.bytes + j * g.b.box_rows * 128, &g.tb, g.b.mn ? 64 * j : kb * kBk, g.b.mn ? kb * kBk : 0, bfull);
        }
        Ring r;
        uint64_t issued = 0;
        bool ok = true;
        const int a_boxes = g.a.boxes, b_boxes = g.resident ? 0 : g.b.boxes, a_step = g.a.box_rows * 128, b_step = g.b.box_rows * 128;
        const bool a_mn = g.a.mn != 0, b_mn = g.b.mn != 0;
        const uint32_t full0 = kPair ? cluster_address(full, 0) : full;
        for (Tiles t(g, first, step); t.more() && ok; t.next()) {
            const int m0 = (kPair ? 2 * t.m + (int)rank : t.m) * kBm, n0 = t.n * g.bn + (kPair ? (int)rank * (g.bn / 2) : 0);
            for (int end, kb = 0; kb < kbs && ok; kb = end) {  // A as it is, and then its low part
                const bool low = kb0 + kb >= g.kfold;
                const CUtensorMap* ta = low ? &g.ta_low : &g.ta;
                end = low ? kbs : min(kbs, g.kfold - kb0);
                for (int k0 = (kb0 + kb - (low ? g.kfold : 0)) * kBk; kb < end; ++kb, k0 += kBk) {
                    if (!(ok = warp_waits<kPair>(empty + 8 * r.stage, r.phase ^ 1u, waits))) break;
                    const uint32_t bar = full0 + 8 * r.stage, sa = sm0 + r.stage * g.stage_bytes, sb = sa + g.a.bytes;
                    if (!kPair && issues) arrive_expect(bar, bytes);
                    if (kPair && rank == 0 && issues) arrive_expect(full + 8 * r.stage, 2 * bytes);  // both blocks' copies
                    for (int j = 0; j < a_boxes; ++j) {
                        const int x = a_mn ? m0 + 64 * j : k0, y = a_mn ? k0 : m0;
                        if (kPair && issues) tma_load_pair(sa + j * a_step, ta, x, y, bar);
                        if (!kPair && issues) tma_load(sa + j * a_step, ta, x, y, bar);
                    }
                    for (int j = 0; j < b_boxes; ++j) {
                        const int x = b_mn ? n0 + 64 * j : k0, y = b_mn ? k0 : n0;
                        if (kPair && issues) tma_load_pair(sb + j * b_step, &g.tb, x, y, bar);
                        if (!kPair && issues) tma_load(sb + j * b_step, &g.tb, x, y, bar);
                    }
                    r.next(g.stages);
                    ++issued;
                }
            }
        }
        if (lane == 0) copies_issued = issued;
        // the block (and with it its barriers) stays until the MMAs' last reports of free stages have arrived
        Ring last = r;
        for (int s = 0; s < g.stages && ok; ++s, last.next(g.stages)) ok = warp_waits<kPair>(empty + 8 * last.stage, last.phase ^ 1u, waits);
    } else if (warp == kOutWarps) {
        // ---------------------------------- MMAs ----------------------------------
        // The whole warp walks through the loop and one lane issues: with everything uniform the descriptors stay
        // in uniform registers, which the instruction wants (from a branch of lane 0 alone it took 385 instead of 332
        // thousand cycles for 8192 x 4096 x 4096).
        if (rank == 0) {
            const bool issues = elect_one();
            Waits waits(&abort_flag, list.patience, kMmas);
            Ring r;
            uint32_t i = 0;
            bool ok = kbs == 0 || !g.resident || warp_waits<kPair>(bfull, 0, waits);
            // Descriptors count addresses in units of 16 bytes: a stage and a step of 16 k are additions to them.
            const uint32_t step_a = g.a.mn ? 128 : 2, step_b = g.b.mn ? 128 : 2, stage = g.stage_bytes >> 4;
            const uint32_t next_b = g.resident ? g.b.bytes >> 4 : 0;
            const uint64_t a0 = swizzled_desc(sm0, 64 * 128), b0 = swizzled_desc(g.resident ? sb0 : sm0 + g.a.bytes, 64 * 128);
            for (Tiles t(g, first, step); t.more() && ok && kbs > 0; t.next(), ++i) {
                uint32_t acc = tmem + (i & 1u) * g.columns;
                if (!(ok = warp_waits<kPair>(room + 8 * (i & 1u), ((i >> 1) & 1u) ^ 1u, waits))) break;
                mlp::fence_after();
                int kseg = 0;
                for (int kb = 0; kb < kbs; ++kb, ++kseg) {
                    if (kGather && kseg == kSegment) {  // this segment's sums go to registers, the next one starts from zero
                        if (kPair && issues) commit_pair(done + 8 * (i & 1u));
                        if (!kPair && issues) mlp::commit(done + 8 * (i & 1u));
                        ++i;
                        kseg = 0;
                        acc = tmem + (i & 1u) * g.columns;
                        if (!(ok = warp_waits<kPair>(room + 8 * (i & 1u), ((i >> 1) & 1u) ^ 1u, waits))) break;
                        mlp::fence_after();
                    }
                    if (!(ok = warp_waits<kPair>(full + 8 * r.stage, r.phase, waits))) break;
                    mlp::fence_after();
                    const uint64_t da = a0 + (uint32_t)r.stage * stage, db = b0 + (g.resident ? (uint32_t)(kb < g.kfold ? kb : kb - g.kfold) * next_b : (uint32_t)r.stage * stage);
#pragma unroll
                    for (int k = 0; k < kBk / 16; ++k) {
                        if (kPair && issues) mma_pair(acc, da + k * step_a, db + k * step_b, g.idesc, (kseg | k) != 0 ? 1u : 0u);
                        if (!kPair && issues) mlp::mma(acc, da + k * step_a, db + k * step_b, g.idesc, (kseg | k) != 0 ? 1u : 0u);
                    }
                    if (kPair && issues) commit_pair(empty + 8 * r.stage);
                    if (!kPair && issues) mlp::commit(empty + 8 * r.stage);
                    r.next(g.stages);
                }
                if (kPair && ok && issues) commit_pair(done + 8 * (i & 1u));
                if (!kPair && ok && issues) mlp::commit(done + 8 * (i & 1u));
            }
        }
    } else {
        // -------------------------------- way out ---------------------------------
        Waits waits(&abort_flag, list.patience, kOut);
        const int quarter = warp & 3, half = warp >> 2, chunks = (g.bn + 31) / 32;
        const Epilogue e = g.e;  // in registers: read through the chosen product, each store would make it suspect
        [[maybe_unused]] void* out = g.split_stride != 0 ? static_cast<float*>(e.out) + part * g.split_stride : e.out;
        uint32_t i = 0;
        for (Tiles t(g, first, step); t.more(); t.next()) {
            const int64_t m0 = (int64_t)(kPair ? 2 * t.m + (int)rank : t.m) * kBm + 32 * quarter;
            const int n0 = t.n * g.bn, cols = (int)min(g.N, (int64_t)n0 + g.bn);
            const int rows = (int)min((int64_t)32, g.M - m0);
            // the 16-bit residuals of a lane's row
            auto load_residual = [&](int c, uint4 (&q)[4]) {
                const int c0 = n0 + 32 * c;
                if (!kVectors || g.cluster > 1 || e.residual == nullptr || e.out_f32 || c0 + 32 > cols || lane >= rows) return;
                const T* p = static_cast<const T*>(e.residual) + (m0 + lane) * e.ldr + c0;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (in_bounds<kChkResidual>(p + 8 * u, 16)) q[u] = *reinterpret_cast<const uint4*>(p + 8 * u);
            };
            // one chunk's sums, a row a lane, on their way
            auto emit_chunk = [&](int c, float (&y)[32], const uint4 (&q)[4]) {
                const int c0 = n0 + 32 * c;
                const bool inside = c0 + 32 <= cols;
                if (g.cluster > 1 || !kVectors) {
                    // a split product leaves its share in the stages' memory, where the cluster's other blocks read it
                    float4* st = reinterpret_cast<float4*>(g.cluster > 1 ? sm + (quarter * chunks + c) * 4096 : staging + warp * 4096);
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 8; ++u) st[unit_of(lane, u)] = make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
                    __syncwarp();
                    if (!kVectors && g.cluster == 1 && c0 + lane < cols) {
                        const float* sf = reinterpret_cast<const float*>(st);
                        const float bias = bias1(e, c0 + lane);
#pragma unroll 1
                        for (int r0 = 0; r0 < rows; r0 += 8) {
                            float s[8];
#pragma unroll
                            for (int p = 0; p < 8; ++p) s[p] = sf[unit_of(r0 + p, lane >> 2) * 4 + (lane & 3)] + bias;
                            if (rows - r0 >= 8) emit_column8<T, true>(e, out, m0 + r0, 8, c0 + lane, s);
                            else emit_column8<T, false>(e, out, m0 + r0, rows - r0, c0 + lane, s);
                        }
                    }
                    return;
                }
                if (e.bias != nullptr) {
                    if (inside) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float4 b = in_bounds<kChkBias>(e.bias + c0 + 4 * u, 16) ? __ldg(reinterpret_cast<const float4*>(e.bias + c0) + u)
                                                                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                            y[4 * u] += b.x; y[4 * u + 1] += b.y; y[4 * u + 2] += b.z; y[4 * u + 3] += b.w;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j < cols) y[j] += bias1(e, c0 + j);
                    }
                }
                uint8_t* sy = staging + warp * 4096;  // y, and 16-bit z behind it
                uint8_t* sz = e.out_f32 ? staging + (kOutWarps + warp) * 4096 : sy + 2048;
                if (lane == 0) store_wait_read();  // the last chunk has left
                __syncwarp();
                if (e.z != nullptr) stage_row16<T>(sz, lane, y);
                activate(y, e.act);
                if (e.residual != nullptr) {
                    if (inside && !e.out_f32) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float2 r0 = unpack2<T>(q[u].x), r1 = unpack2<T>(q[u].y), r2 = unpack2<T>(q[u].z), r3 = unpack2<T>(q[u].w);
                            y[8 * u] += r0.x; y[8 * u + 1] += r0.y; y[8 * u + 2] += r1.x; y[8 * u + 3] += r1.y;
                            y[8 * u + 4] += r2.x; y[8 * u + 5] += r2.y; y[8 * u + 6] += r3.x; y[8 * u + 7] += r3.y;
                        }
                    } else if (inside && lane < rows) {
                        const float* p = static_cast<const float*>(e.residual) + (m0 + lane) * e.ldr + c0;
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            if (in_bounds<kChkResidual>(p + 4 * u, 16)) {
                                const float4 r = *reinterpret_cast<const float4*>(p + 4 * u);
                                y[4 * u] += r.x; y[4 * u + 1] += r.y; y[4 * u + 2] += r.z; y[4 * u + 3] += r.w;
                            }
                    } else if (lane < rows) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j < cols) y[j] += residual1<T>(e, m0 + lane, c0 + j);
                    }
                }
                if (e.out_f32) stage_row32(sy, lane, y);
                else stage_row16<T>(sy, lane, y);
                mlp::fence_async_smem();
                __syncwarp();
                if (lane == 0 && c0 < cols) {
                    if (e.z != nullptr) tma_store(&g.tz, (uint32_t)__cvta_generic_to_shared(sz), c0, (int)m0, 0);
                    tma_store(&g.ty, (uint32_t)__cvta_generic_to_shared(sy), c0, (int)m0, part);
                    store_commit();
                }
            };
            auto wait_accumulator = [&]() {
                const bool ok = warp_waits<kPair>(done + 8 * (i & 1u), (i >> 1) & 1u, waits);
                mlp::fence_after();
                return ok;
            };
            auto free_accumulator = [&]() {
                mlp::fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair) arrive_cluster(cluster_address(room + 8 * (i & 1u), 0));
                    else mlp::mbar_arrive(room + 8 * (i & 1u));
                }
                ++i;
            };
            const uint32_t row_of_tmem = tmem + ((uint32_t)(32 * quarter) << 16);
            if (kGather) {
                constexpr int kMine = kPair ? 4 : 2;  // chunks of a warp
                float acc[kMine][32];
#pragma unroll
                for (int k = 0; k < kMine; ++k)
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[k][j] = 0.f;
                for (int kb = 0; kb < kbs; kb += kSegment) {
                    if (!wait_accumulator()) goto out_of_time;
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        if (2 * k + half >= chunks || rows <= 0) continue;
                        uint32_t v[32];
                        __syncwarp();
                        tmem_ld32(row_of_tmem + (i & 1u) * g.columns + 32 * (2 * k + half), v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc[k][j] += __uint_as_float(v[j]);
                    }
                    free_accumulator();
                }
#pragma unroll
                for (int k = 0; k < kMine; ++k) {
                    if (2 * k + half >= chunks || rows <= 0) continue;
                    uint4 q[4] = {};
                    load_residual(2 * k + half, q);
                    emit_chunk(2 * k + half, acc[k], q);
                }
                continue;
            }
            bool waited = kbs == 0;
            for (int c = half; c < chunks && rows > 0; c += 2) {
                uint4 q[4] = {};
                load_residual(c, q);  // on its way while the accumulator is waited for and read
                __syncwarp();
                if (!waited && !wait_accumulator()) goto out_of_time;
                waited = true;
                uint32_t v[32];
                float y[32];
                if (kbs > 0) {
                    tmem_ld32(row_of_tmem + (i & 1u) * g.columns + 32 * c, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(v[j]);
                emit_chunk(c, y, q);
            }
            if (kbs > 0) {
                if (!waited && !wait_accumulator()) goto out_of_time;  // a warp without a chunk keeps in step all the same
                free_accumulator();
            }
        }
    out_of_time:
        if (kVectors && lane == 0) store_wait();
    }
    __syncwarp();
    if (!kPair && g.cluster > 1) {
        // K is split over the cluster's blocks: their shares of the tile are added in rank order, every block
        // writing out the rows of its turn.
        cluster_sync();
        const int chunks = (g.bn + 31) / 32, quarters = (int)min((int64_t)4, (g.M - (int64_t)(first / g.nt) * kBm + 31) / 32);
        const int64_t tm = (int64_t)(first / g.nt) * kBm;
        const int tn = (first % g.nt) * g.bn, cols = (int)min(g.N, (int64_t)tn + g.bn);
        if (warp < kOutWarps && abort_flag == 0)
            for (int u = warp * g.cluster + part; u < quarters * chunks * 4; u += kOutWarps * g.cluster) {
                const int chunk = u >> 2, r = 8 * (u & 3) + (lane >> 2);  // chunk = quarter * chunks + column chunk
                const int64_t row = tm + 32 * (chunk / chunks) + r;
                const int col = tn + 32 * (chunk % chunks) + 8 * (lane & 3);
                if (row >= g.M || col >= cols) continue;
                const uint32_t lo = sm0 + chunk * 4096 + unit_of(r, 2 * (lane & 3)) * 16, hi = sm0 + chunk * 4096 + unit_of(r, 2 * (lane & 3) + 1) * 16;
                float y[1][8] = {};
#pragma unroll 4
                for (int k = 0; k < g.cluster; ++k) {
                    const float4 a = cluster_load(cluster_address(lo, k)), b = cluster_load(cluster_address(hi, k));
                    y[0][0] += a.x; y[0][1] += a.y; y[0][2] += a.z; y[0][3] += a.w;
                    y[0][4] += b.x; y[0][5] += b.y; y[0][6] += b.z; y[0][7] += b.w;
                }
                if (kVectors && col + 8 <= cols) {
                    float b[8];
                    uint4 q[1] = {};
                    if (g.e.residual != nullptr && !g.e.out_f32) load_residuals<T, 1>(g.e, row, row + 1, col, q);
                    bias8(g.e, col, b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[0][j] += b[j];
                    emit_vectors<T, 1>(g.e, g.e.out, row, row + 1, col, y, q);
                } else {
                    float res[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        res[j] = col + j < cols ? residual1<T>(g.e, row, col + j) : 0.f;
                        if (col + j < cols) y[0][j] += bias1(g.e, col + j);
                    }
                    if (g.e.z != nullptr)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (col + j < cols) store_z1<T>(g.e, row, col + j, y[0][j]);
                    activate(y[0], g.e.act);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col + j < cols) store_y1<T>(g.e, g.e.out, row, col + j, y[0][j] + res[j]);
                }
            }
        __syncwarp();
        cluster_sync();  // nobody leaves while its shares are read
    }
    mlp::fence_before();
    __syncthreads();
    if (kPair) cluster_sync();  // nor while the pair's MMAs read its memory
    if (abort_flag != 0) {
        // Some role gave up (in a pair: of either block): copies and MMAs that the others did not wait for may still be under way.
        // A pair's copies are counted by the first block's barriers, in pairs. Where one block issued more of them, the other's
        // share is made up for: it will not come any more, or was not yet expected.
        if (warp == kOutWarps + 1 && rank == 0) {
            if (g.resident && kbs > 0) mlp::wait_parity(bfull, 0);
            const uint64_t mine = copies_issued;
            const uint64_t theirs = kPair ? cluster_load64(cluster_address((uint32_t)__cvta_generic_to_shared(&copies_issued), 1)) : mine;
            const uint64_t most = max(mine, theirs);
            if (kPair && lane == 0) {
                for (uint64_t c = mine; c < most; ++c) arrive_expect(full + 8 * (uint32_t)(c % g.stages), g.a.bytes + g.b.bytes);
                for (uint64_t c = theirs; c < most; ++c) count_copied(full + 8 * (uint32_t)(c % g.stages), g.a.bytes + g.b.bytes);
            }
            __syncwarp();
            for (uint64_t c = most - min(most, (uint64_t)g.stages); c < most; ++c)
                mlp::wait_parity(full + 8 * (uint32_t)(c % g.stages), (uint32_t)(c / g.stages) & 1u);
        } else if (warp == kOutWarps) {
            if (rank == 0 && elect_one()) {
                if (kPair) commit_pair(drain);  // both blocks' MMAs, reported to both
                else mlp::commit(drain);
            }
            mlp::wait_parity(drain, 0);
        }
        __syncthreads();
        if (kPair) cluster_sync();
    }
    mlp::fence_after();
    if (threadIdx.x == 0 && abort_flag != 0) report_given_up(g.status);
    __syncwarp();
    if (warp == 0) {
        if (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.tmem_columns) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.tmem_columns) : "memory");
    }
}

// Copies of arrays whose rows do not begin on 16-byte boundaries into rows that do (TMA copies no
// others): 16 bytes out a thread at a time, from the two aligned 16-byte units that hold them,
// shifted together; four such at once keep loads in flight.
struct Realign {
    const void* p;
    uint16_t* to;
    uint64_t bytes;        // extent of the source
    int64_t outer, ld, chunks;  // chunks of 8 elements of a row, rounded up
    int inner, role;
};
struct RealignList {
    Realign a[2];
    int64_t first;  // chunks of a[0]
    int64_t total;
};

// Eight elements of a row (zeros beyond its end).
struct Chunk {
    uint4 p, q;
    uint32_t shift;  // bytes
    int n;           // elements that are there
};

__device__ __forceinline__ void begin_chunk(const Realign& s, int64_t row, int col, Chunk& c) {
    c.p = c.q = make_uint4(0u, 0u, 0u, 0u);
    c.shift = 0;
    c.n = min(8, s.inner - col);
    const char* base = static_cast<const char*>(s.p);
    const uint64_t off = (uint64_t)(row * s.ld + col) * 2, lo = off & ~15ull;
    const uint32_t sh = (uint32_t)(off & 15u);
    const bool two = sh + 2 * c.n > 16;
    if (lo + (two ? 32 : 16) <= s.bytes) {
        c.shift = sh;
        if (in_bounds_role(s.role, base + lo, 16)) c.p = __ldg(reinterpret_cast<const uint4*>(base + lo));
        if (two && in_bounds_role(s.role, base + lo + 16, 16)) c.q = __ldg(reinterpret_cast<const uint4*>(base + lo + 16));
        return;
    }
    // the array's last bytes: one element at a time
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < c.n && in_bounds_role(s.role, base + off + 2 * j, 2))
            w[j >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(base + off + 2 * j) << (16 * (j & 1));
    c.p = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 finish_chunk(const Chunk& c) {
    uint32_t w[8] = {c.p.x, c.p.y, c.p.z, c.p.w, c.q.x, c.q.y, c.q.z, c.q.w};
    if (c.shift & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (c.shift & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = (c.shift & 2u) * 8u;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __funnelshift_r(w[i], w[i + 1], bits);
        if (2 * i + 1 >= c.n) v[i] = 2 * i < c.n ? v[i] & 0xffffu : 0u;
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void realign_block(const RealignList& l, int64_t block) {
    constexpr int kAtOnce = 4;
    const int64_t i0 = block * (256 * kAtOnce) + threadIdx.x;
    Chunk c[kAtOnce];
    const bool second = i0 >= l.first;  // a block whose chunks lie in both arrays tells them apart below
    const bool same = second == (i0 + 256 * (kAtOnce - 1) >= l.first) && i0 + 256 * (kAtOnce - 1) < l.total;
    const Realign s = l.a[second];
    const int64_t j0 = second ? i0 - l.first : i0;
    auto place = [](int64_t j, int64_t chunks, int64_t& row, int& col) {
        row = ((uint64_t)j >> 32) == 0 && chunks < (1 << 30) ? (int64_t)((uint32_t)j / (uint32_t)chunks) : j / chunks;
        col = (int)(j - row * chunks) * 8;
    };
    int64_t last_row;
    int last_col;
    place(j0 + 256 * (kAtOnce - 1), s.chunks, last_row, last_col);
    if (same && (((uint64_t)(last_row * s.ld + last_col) * 2) & ~15ull) + 32 <= s.bytes) {
        // both units of every chunk lie inside the array: loads without guards, all under way before the first is used
        const char* base = static_cast<const char*>(s.p);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            int64_t row;
            int col;
            place(j0 + 256 * u, s.chunks, row, col);
            const uint64_t off = (uint64_t)(row * s.ld + col) * 2, at = off & ~15ull;
            c[u].shift = (uint32_t)(off & 15u);
            c[u].n = min(8, s.inner - col);
            c[u].p = in_bounds_role(s.role, base + at, 16) ? __ldg(reinterpret_cast<const uint4*>(base + at)) : make_uint4(0u, 0u, 0u, 0u);
            c[u].q = in_bounds_role(s.role, base + at + 16, 16) ? __ldg(reinterpret_cast<const uint4*>(base + at + 16)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            uint16_t* to = s.to + 8 * (j0 + 256 * u);
            if (in_bounds<kChkWork>(to, 16)) *reinterpret_cast<uint4*>(to) = finish_chunk(c[u]);
        }
        return;
    }
    for (int u = 0; u < kAtOnce; ++u) {
        const int64_t i = i0 + 256 * u;
        if (i >= l.total) return;
        const Realign& a = l.a[i >= l.first];
        const int64_t j = i >= l.first ? i - l.first : i;
        int64_t row;
        int col;
        place(j, a.chunks, row, col);
        begin_chunk(a, row, col, c[0]);
        uint16_t* to = a.to + 8 * j;
        if (in_bounds<kChkWork>(to, 16)) *reinterpret_cast<uint4*>(to) = finish_chunk(c[0]);
    }
}

// ---------------------------------------------------------------------------------------
// The whole backward pass of a narrow layer in one pass over its rows (in, out up to 128, many
// rows: the layers of a head over a batch of points). Such a layer is bound by memory: dy, z and
// x are read once and dx is written once, 2 (2 out + 2 in) bytes a row, where separate products
// would move dz three more times and x once.
//
// Persistent blocks, one an SM, over tiles of 128 rows. TMA brings a tile of dy, z and x into a stage in
// the 128-byte-swizzled layout. Eight warps turn dy into dz in place (and keep db's sums in
// registers); behind a smooth activation dz is two numbers, the low one in z's place, and each product
// runs over both. That one copy of dz then serves both products: with rows of 64 outputs it is a k-major
// A operand of dx = dz W and, read the other way, an mn-major A operand of dW = dz^T x, as the tile of x
// is its mn-major B operand. W stays in shared memory. dx goes out as in the kernel above; dW
// gathers in tensor memory over kFlush tiles, and is then added to fp32 registers (the tensor cores'
// additions cut off: see kGather above). Each block writes its sums to the workspace, where
// sum_parts_kernel adds them in order.
//
// Warps: 0-7 write dx, 8 issues MMAs, 9 copies, 10-17 make dz and keep dW's and db's sums.
// ---------------------------------------------------------------------------------------
constexpr int kFlush = 6;
constexpr int kNarrowThreads = 32 * 18;
constexpr int kNarrowStages = 4;
constexpr int kBox = kBm * 128;  // bytes of a box of 128 rows x 64 columns

struct Narrow {
    CUtensorMap tdy, tz, tx, tw, tdx;
    int64_t rows;
    int in, out, act;
    int boxes_in, boxes_out, columns;  // 64-wide boxes of x and of dy (and z); columns from one accumulator to the next
    int pieces;                        // dz's: 2 where its low part takes z's place (or comes as z, without an activation)
    int stages, stage_bytes, w_bytes, k_out;  // k_out: out, rounded up to 16
    uint32_t id_dx, id_dw, tmem_columns;
    Epilogue e;                        // of dx; out NULL: not wanted
    float* parts;                      // [blocks][out * in + out]
    int want_db;
    int* status;
    Patience patience;
};

__host__ __device__ constexpr size_t narrow_smem(int stage_bytes_in_all, int w_bytes) {
    return 1024 + (size_t)stage_bytes_in_all + w_bytes + kStaging + 256 + 16;
}

template <typename T, int kChunks, bool kVectors>  // kChunks * 64 >= in; kVectors: dx leaves by TMA
__global__ void __launch_bounds__(kNarrowThreads, 1) narrow_backward_kernel(const __grid_constant__ Narrow g) {
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint8_t* ws = sm + (size_t)g.stages * g.stage_bytes;
    uint8_t* staging = ws + g.w_bytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStaging);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 32);
    __shared__ volatile int abort_flag;
    __shared__ int copies_issued;  // stages that the copying warp filled
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t sm0 = (uint32_t)__cvta_generic_to_shared(sm), w0 = (uint32_t)__cvta_generic_to_shared(ws);
    const uint32_t bar0 = (uint32_t)__cvta_generic_to_shared(bars);
    // barriers: stage copied [4], dz ready [4], stage free [4], dx done [2], dx room [2], dw done [2], dw room [2], W copied, drain
    const uint32_t full = bar0, ready = full + 32, empty = ready + 32, done = empty + 32, room = done + 16, wdone = room + 16, wroom = wdone + 16,
                   wfull = wroom + 16, drain = wfull + 8;
    const bool dx = g.e.out != nullptr;
    if (threadIdx.x == 32 * 9) {
        abort_flag = 0;
        for (int s = 0; s < g.stages; ++s) {
            mlp::mbar_init(full + 8 * s, 1);
            mlp::mbar_init(ready + 8 * s, 8);
            mlp::mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mlp::mbar_init(done + 8 * i, 1);
            mlp::mbar_init(room + 8 * i, 8);
            mlp::mbar_init(wdone + 8 * i, 1);
            mlp::mbar_init(wroom + 8 * i, 8);
        }
        mlp::mbar_init(wfull, 1);
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
    after_previous_kernel();
    const uint32_t tmem = *tslot;
    const int tiles = (int)((g.rows + kBm - 1) / kBm);
    const int mine = (tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1;  // at least one: the grid has no more blocks than tiles
    const bool second = g.act != kNoAct || g.pieces == 2;  // z, or dz's low part
    const int dy_bytes = g.boxes_out * kBox, z_at = dy_bytes, x_at = second ? 2 * dy_bytes : dy_bytes;

    if (warp == 9) {
        // ------------------------------- TMA copies -------------------------------
        const bool issues = elect_one();
        Waits waits(&abort_flag, g.patience, kCopies);
        bool ok = true;
        if (dx && issues) {
            arrive_expect(wfull, g.w_bytes);
            for (int j = 0; j < g.boxes_in; ++j) tma_load(w0 + j * g.k_out * 128, &g.tw, 64 * j, 0, wfull);
        }
        Ring r;
        int issued = 0;
        for (int i = 0; i < mine; ++i) {
            if (!(ok = warp_waits<false>(empty + 8 * r.stage, r.phase ^ 1u, waits))) break;
            const uint32_t bar = full + 8 * r.stage, s = sm0 + r.stage * g.stage_bytes;
            const int m0 = (int)(blockIdx.x + i * gridDim.x) * kBm;
            if (issues) {
                arrive_expect(bar, g.stage_bytes);
                for (int j = 0; j < g.boxes_out; ++j) tma_load(s + j * kBox, &g.tdy, 64 * j, m0, bar);
                if (second)
                    for (int j = 0; j < g.boxes_out; ++j) tma_load(s + z_at + j * kBox, &g.tz, 64 * j, m0, bar);
                for (int j = 0; j < g.boxes_in; ++j) tma_load(s + x_at + j * kBox, &g.tx, 64 * j, m0, bar);
            }
            r.next(g.stages);
            ++issued;
        }
        if (lane == 0) copies_issued = issued;
        // the block (and with it its barriers) stays until the MMAs' last reports of free stages have arrived
        Ring last = r;
        for (int i = 0; i < g.stages && ok; ++i, last.next(g.stages)) ok = warp_waits<false>(empty + 8 * last.stage, last.phase ^ 1u, waits);
    } else if (warp == 8) {
        // ---------------------------------- MMAs ----------------------------------
        const bool issues = elect_one();
        Waits waits(&abort_flag, g.patience, kMmas);
        Ring r;
        bool ok = !dx || warp_waits<false>(wfull, 0, waits);
        const uint32_t dw0 = tmem + 2 * g.columns, stage = g.stage_bytes >> 4;
        const uint64_t dz_k = swizzled_desc(sm0, 0), dz_mn = swizzled_desc(sm0, kBox), x_mn = swizzled_desc(sm0 + x_at, kBox),
                       w_mn = swizzled_desc(w0, g.k_out * 128);
        for (int i = 0; i < mine && ok; ++i) {
            const int b = i & 1, group = i / kFlush, f = group & 1;
            if (!(ok = warp_waits<false>(full + 8 * r.stage, r.phase, waits))) break;
            if (!(ok = warp_waits<false>(ready + 8 * r.stage, r.phase, waits))) break;
            if (dx && !(ok = warp_waits<false>(room + 8 * b, ((i >> 1) & 1u) ^ 1u, waits))) break;
            if (i % kFlush == 0 && !(ok = warp_waits<false>(wroom + 8 * f, ((group >> 1) & 1u) ^ 1u, waits))) break;
            mlp::fence_after();
            const uint32_t off = (uint32_t)r.stage * stage;
            if (dx) {
                for (int p = 0; p < g.pieces; ++p)
                    for (int k = 0; k < g.k_out / 16; ++k) {
                        const uint32_t ak = (p != 0 ? z_at >> 4 : 0) + (k >> 2) * (kBox >> 4) + (k & 3) * 2, bk = k * 128;
                        if (issues) mlp::mma(tmem + b * g.columns, dz_k + off + ak, w_mn + bk, g.id_dx, (p | k) != 0 ? 1u : 0u);
                    }
                if (issues) mlp::commit(done + 8 * b);
            }
            uint32_t acc = i % kFlush != 0 ? 1u : 0u;
            for (int p = 0; p < g.pieces; ++p, acc = 1u) {
                const uint32_t at = off + (p != 0 ? z_at >> 4 : 0);
#pragma unroll
                for (int k = 0; k < kBm / 16; ++k)
                    if (issues) mlp::mma(dw0 + f * g.columns, dz_mn + at + k * 128, x_mn + off + k * 128, g.id_dw, k != 0 ? 1u : acc);
            }
            if (issues) mlp::commit(empty + 8 * r.stage);
            if (issues && (i % kFlush == kFlush - 1 || i == mine - 1)) mlp::commit(wdone + 8 * f);
            r.next(g.stages);
        }
    } else if (warp < 8) {
        // ---------------------------------- dx -----------------------------------
        Waits waits(&abort_flag, g.patience, kOut);
        const int quarter = warp & 3, chunks = (g.in + 31) / 32;
        uint8_t* st = staging + warp * 4096;
        for (int i = 0; i < mine && dx; ++i) {
            const int b = i & 1;
            const int m0 = (int)(blockIdx.x + i * gridDim.x) * kBm + 32 * quarter;
            if (!warp_waits<false>(done + 8 * b, (i >> 1) & 1u, waits)) break;
            mlp::fence_after();
            for (int c = warp >> 2; c < chunks; c += 2) {
                uint32_t v[32];
                __syncwarp();
                tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + b * g.columns + 32 * c, v);
                float y[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(v[j]);
                if (!kVectors) {
                    float4* sq = reinterpret_cast<float4*>(st);
#pragma unroll
                    for (int u = 0; u < 8; ++u) sq[unit_of(lane, u)] = make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
                    __syncwarp();
                    const int rows = (int)min((int64_t)32, g.rows - m0);
                    if (32 * c + lane < g.in)
#pragma unroll 1
                        for (int r0 = 0; r0 < rows; r0 += 8) {
                            float s[8];
#pragma unroll
                            for (int p = 0; p < 8; ++p) s[p] = reinterpret_cast<const float*>(st)[unit_of(r0 + p, lane >> 2) * 4 + (lane & 3)];
                            if (rows - r0 >= 8) emit_column8<T, true>(g.e, g.e.out, m0 + r0, 8, 32 * c + lane, s);
                            else emit_column8<T, false>(g.e, g.e.out, m0 + r0, rows - r0, 32 * c + lane, s);
                        }
                    __syncwarp();
                    continue;
                }
                if (lane == 0) store_wait_read();  // the last chunk has left
                __syncwarp();
                if (g.e.out_f32) stage_row32(st, lane, y);
                else stage_row16<T>(st, lane, y);
                mlp::fence_async_smem();
                __syncwarp();
                if (lane == 0 && m0 < g.rows) {
                    tma_store(&g.tdx, (uint32_t)__cvta_generic_to_shared(st), 32 * c, m0, 0);
                    store_commit();
                }
            }
            mlp::fence_before();
            __syncwarp();
            if (lane == 0) mlp::mbar_arrive(room + 8 * b);
        }
        if (lane == 0) store_wait();
    } else {
        // --------------------------- dz, and dW's and db's sums ---------------------------
        Waits waits(&abort_flag, g.patience, kSlopes);
        const int tt = threadIdx.x - 32 * 10, quarter = warp & 3, half = (warp - 10) >> 2;
        // a thread keeps one 16-byte column chunk and takes every 256 / (8 boxes_out)-th row
        const int per_row = 8 * g.boxes_out, chunk = tt % per_row, row_step = 256 / per_row, row0 = tt / per_row;
        const int box_at = (chunk >> 3) * kBox, cc = chunk & 7;
        float sum[8] = {}, acc[kChunks][32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[c][j] = 0.f;
        bool ok = true;
        auto flush = [&](int group) {  // adds what a group of tiles gathered in tensor memory
            const int f = group & 1;
            if (!warp_waits<false>(wdone + 8 * f, (group >> 1) & 1u, waits)) return false;
            mlp::fence_after();
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (32 * quarter >= g.out || 32 * (2 * c + half) >= g.in) continue;
                uint32_t v[32];
                __syncwarp();
                tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + (2 + f) * g.columns + 32 * (2 * c + half), v);
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[c][j] += __uint_as_float(v[j]);
            }
            mlp::fence_before();
            __syncwarp();
            if (lane == 0) mlp::mbar_arrive(wroom + 8 * f);
            return true;
        };
        // dy becomes dz, of one number or two (kBoth)
        auto slopes = [&](uint8_t* s, auto both) {
            constexpr bool kBoth = decltype(both)::value;
#pragma unroll 2
            for (int row = row0; row < kBm; row += row_step) {
                uint4* at = reinterpret_cast<uint4*>(s + row * 128 + ((cc ^ (row & 7)) << 4));
                const uint4 q = *at;
                float d[8];
                const float2 d0 = unpack2<T>(q.x), d1 = unpack2<T>(q.y), d2 = unpack2<T>(q.z), d3 = unpack2<T>(q.w);
                d[0] = d0.x; d[1] = d0.y; d[2] = d1.x; d[3] = d1.y; d[4] = d2.x; d[5] = d2.y; d[6] = d3.x; d[7] = d3.y;
                if (kBoth || g.act != kNoAct) {
                    uint4* zat = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(at) + z_at);
                    const uint4 zq = *zat;
                    const float2 z0 = unpack2<T>(zq.x), z1 = unpack2<T>(zq.y), z2 = unpack2<T>(zq.z), z3 = unpack2<T>(zq.w);
                    const float z[8] = {z0.x, z0.y, z1.x, z1.y, z2.x, z2.y, z3.x, z3.y};
                    times_slope(d, z, g.act);
                    if constexpr (kBoth) *at = split8<T>(d, *zat);
                    else *at = pack8<T>(d);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += d[j];
            }
            mlp::fence_async_smem();
        };
        Ring r;
        for (int i = 0; i < mine && ok; ++i) {
            if (!(ok = warp_waits<false>(full + 8 * r.stage, r.phase, waits))) break;
            uint8_t* s = sm + r.stage * g.stage_bytes + box_at;
            if (g.act != kNoAct && g.pieces == 2) slopes(s, std::true_type());
            else if (g.act != kNoAct || g.want_db) slopes(s, std::false_type());
            __syncwarp();
            if (lane == 0) mlp::mbar_arrive(ready + 8 * r.stage);
            r.next(g.stages);
            // a group's sums are collected one tile after its last MMAs became ready: by then they are done, and nothing waits
            if (i % kFlush == 1 && i > kFlush) ok = flush(i / kFlush - 1);
        }
        if (ok && mine > kFlush && (mine - 1) % kFlush == 0) ok = flush((mine - 1) / kFlush - 1);
        if (ok) ok = flush((mine - 1) / kFlush);
        float* part = g.parts + (int64_t)blockIdx.x * ((int64_t)g.out * g.in + g.out);
        const int o = 32 * quarter + lane;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const int col = 32 * (2 * c + half) + j;
                float* p = part + (int64_t)o * g.in + col;
                if (o >= g.out || col >= g.in) continue;
                if (g.in % 4 == 0 && g.out % 4 == 0) {  // a block's sums are in * out + out floats
                    if (in_bounds<kChkWork>(p, 16)) *reinterpret_cast<float4*>(p) = make_float4(acc[c][j], acc[c][j + 1], acc[c][j + 2], acc[c][j + 3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (col + k < g.in && in_bounds<kChkWork>(p + k, 4)) p[k] = acc[c][j + k];
                }
            }
        // db: the threads of a column chunk in order, through the first stage (every MMA that read it is done)
        if (g.want_db) {
            float* shared = reinterpret_cast<float*>(sm);
#pragma unroll
            for (int j = 0; j < 8; ++j) shared[(row0 * per_row + chunk) * 8 + j] = sum[j];
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (tt < g.out) {
                float s = 0.f;
                for (int k = 0; k < row_step; ++k) s += shared[(k * per_row) * 8 + tt];
                float* p = part + (int64_t)g.out * g.in + tt;
                if (in_bounds<kChkWork>(p, 4)) *p = s;
            }
        }
    }
    __syncwarp();
    mlp::fence_before();
    __syncthreads();
    if (abort_flag != 0) {  // some role gave up: copies and MMAs that the others did not wait for may still be under way
        if (warp == 9) {
            if (dx) mlp::wait_parity(wfull, 0);
            for (int c = max(0, copies_issued - g.stages); c < copies_issued; ++c)
                mlp::wait_parity(full + 8 * (c % g.stages), (uint32_t)(c / g.stages) & 1u);
        } else if (warp == 8 && elect_one()) {
            mlp::commit(drain);
            mlp::wait_parity(drain, 0);
        }
        __syncthreads();
    }
    mlp::fence_after();
    if (threadIdx.x == 0 && abort_flag != 0) report_given_up(g.status);
    __syncwarp();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.tmem_columns) : "memory");
}

// dz = dy act'(z), rounded to T, into dz (NULL: not wanted), what the rounding left into low (NULL: nothing, or not
// wanted), and the sums of the unrounded dz over a block's share of the rows into sums[share][col] (NULL: not wanted). A block takes up to 64 columns,
// a thread eight neighbouring ones of every (256 / groups)-th row.
struct Slope {
    Realign dy, z;     // as sources
    int64_t rows, lddz;
    int cols, act;
    void* dz;
    void* low;
    float* sums;
    int role;          // CheckRole of sums
    int groups;        // column groups of eight in a block: 1, 2, 4 or 8
    int col_blocks, shares;
};

// kVectors: the rows of dy and z begin on 16-byte boundaries and cols is a multiple of 8. kLow: low is wanted (a kernel of its
// own, since it takes 110 registers instead of 80).
template <typename T, bool kVectors, bool kLow>
__device__ __forceinline__ void slope_block(const Slope& a, int block) {
    __shared__ float part[8][64];
    const T* dy = static_cast<const T*>(a.dy.p);
    const T* z = static_cast<const T*>(a.z.p);
    T* dz = static_cast<T*>(a.dz);
    [[maybe_unused]] T* low = static_cast<T*>(a.low);
    const int col_block = block % a.col_blocks, which = block / a.col_blocks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = col_block * 64 + 8 * (threadIdx.x % a.groups), r = threadIdx.x / a.groups, step = 256 / a.groups;
    const int64_t share = (a.rows + a.shares - 1) / a.shares, r0 = which * share, r1 = min(a.rows, r0 + share);
    const int n = min(8, a.cols - col);
    float s[8] = {};
    auto one = [&](int64_t row, uint4 q, uint4 zq) {
        const float2 d0 = unpack2<T>(q.x), d1 = unpack2<T>(q.y), d2 = unpack2<T>(q.z), d3 = unpack2<T>(q.w);
        float d[8] = {d0.x, d0.y, d1.x, d1.y, d2.x, d2.y, d3.x, d3.y};
        if (a.act != kNoAct) {
            const float2 z0 = unpack2<T>(zq.x), z1 = unpack2<T>(zq.y), z2 = unpack2<T>(zq.z), z3 = unpack2<T>(zq.w);
            const float v[8] = {z0.x, z0.y, z1.x, z1.y, z2.x, z2.y, z3.x, z3.y};
            times_slope(d, v, a.act);
        }
        // rows of dz are multiples of 8 wide: what lies between `cols` and that is zero
        if (dz != nullptr && in_bounds<kChkWork>(dz + row * a.lddz + col, 16)) {
            if constexpr (kLow) {
                uint4 rest;
                *reinterpret_cast<uint4*>(dz + row * a.lddz + col) = split8<T>(d, rest);
                if (in_bounds<kChkWork>(low + row * a.lddz + col, 16)) *reinterpret_cast<uint4*>(low + row * a.lddz + col) = rest;
            } else {
                *reinterpret_cast<uint4*>(dz + row * a.lddz + col) = pack8<T>(d);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += d[j];
    };
    const uint4 nothing = make_uint4(0u, 0u, 0u, 0u);
    int64_t row = n > 0 ? r0 + r : r1;
    if (kVectors) {
        auto load = [&](int64_t at, uint4& q, uint4& zq) {
            const T* p = dy + at * a.dy.ld + col;
            const T* pz = z + at * a.z.ld + col;
            q = in_bounds<kChkDout>(p, 16) ? __ldg(reinterpret_cast<const uint4*>(p)) : nothing;
            zq = a.act != kNoAct && in_bounds<kChkZ>(pz, 16) ? __ldg(reinterpret_cast<const uint4*>(pz)) : nothing;
        };
        for (; row + 3 * step < r1; row += 4 * step) {  // four rows' loads under way at a time
            uint4 q[4], zq[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) load(row + k * step, q[k], zq[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) one(row + k * step, q[k], zq[k]);
        }
        for (; row < r1; row += step) {
            uint4 q, zq;
            load(row, q, zq);
            one(row, q, zq);
        }
    } else {
        // Several rows at a time while both 16-byte units that hold their elements lie inside the arrays: those loads need no
        // guard, so that all of them are under way before the first is used.
        constexpr int kRows = 4;
        const char* by = static_cast<const char*>(a.dy.p);
        const char* bz = static_cast<const char*>(a.z.p);
        for (; row + (kRows - 1) * step < r1; row += kRows * step) {
            const int64_t last = row + (kRows - 1) * step;
            if ((((uint64_t)(last * a.dy.ld + col) * 2) & ~15ull) + 32 > a.dy.bytes ||
                (a.act != kNoAct && (((uint64_t)(last * a.z.ld + col) * 2) & ~15ull) + 32 > a.z.bytes))
                break;
            Chunk c[kRows], cz[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const uint64_t off = (uint64_t)((row + k * step) * a.dy.ld + col) * 2, at = off & ~15ull;
                c[k].shift = (uint32_t)(off & 15u);
                c[k].n = n;
                c[k].p = in_bounds<kChkDout>(by + at, 16) ? __ldg(reinterpret_cast<const uint4*>(by + at)) : nothing;
                c[k].q = in_bounds<kChkDout>(by + at + 16, 16) ? __ldg(reinterpret_cast<const uint4*>(by + at + 16)) : nothing;
            }
            if (a.act != kNoAct)
#pragma unroll
                for (int k = 0; k < kRows; ++k) {
                    const uint64_t off = (uint64_t)((row + k * step) * a.z.ld + col) * 2, at = off & ~15ull;
                    cz[k].shift = (uint32_t)(off & 15u);
                    cz[k].n = n;
                    cz[k].p = in_bounds<kChkZ>(bz + at, 16) ? __ldg(reinterpret_cast<const uint4*>(bz + at)) : nothing;
                    cz[k].q = in_bounds<kChkZ>(bz + at + 16, 16) ? __ldg(reinterpret_cast<const uint4*>(bz + at + 16)) : nothing;
                }
#pragma unroll
            for (int k = 0; k < kRows; ++k) one(row + k * step, finish_chunk(c[k]), a.act != kNoAct ? finish_chunk(cz[k]) : nothing);
        }
        for (; row < r1; row += step) {
            Chunk c, cz;
            begin_chunk(a.dy, row, col, c);
            if (a.act != kNoAct) begin_chunk(a.z, row, col, cz);
            one(row, finish_chunk(c), a.act != kNoAct ? finish_chunk(cz) : nothing);
        }
    }
    if (a.sums == nullptr) return;
    for (int o = 16; o >= a.groups; o >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
    if (lane < a.groups)
#pragma unroll
        for (int j = 0; j < 8; ++j) part[warp][8 * lane + j] = s[j];
    __syncthreads();
    const int c = col_block * 64 + threadIdx.x;
    if (threadIdx.x < 8 * a.groups && c < a.cols) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += part[w][threadIdx.x];
        float* p = a.sums + (int64_t)which * a.cols + c;
        if (in_bounds_role(a.role, p, 4)) *p = t;
    }
}

// What comes before the products, in one launch: dz and db's sums (the first blocks), and the copies of
// arrays that TMA cannot read as they are.
template <typename T, bool kVectors, bool kLow>
__global__ void __launch_bounds__(256, !kVectors ? 2 : kLow ? 1 : 3) prepare_kernel(const __grid_constant__ Slope slope, const __grid_constant__ RealignList copies, int slope_blocks) {
    after_previous_kernel();
    if ((int)blockIdx.x < slope_blocks) slope_block<T, kVectors, kLow>(slope, blockIdx.x);
    else realign_block(copies, blockIdx.x - slope_blocks);
}

// Sums of parts in order, of one or two arrays: out[i] = sum over p of parts[p * stride + i]. A block takes
// 32 neighbours of an array, each of its 8 warps every eighth part.
struct Sums {
    const float* parts;
    int64_t stride, n;
    int count, out_type;  // parts; 0 fp32, 1 T
    void* out;
    int role;
};
struct SumsList {
    Sums a[2];
    int blocks0;  // blocks of a[0]
};

template <typename T>
__global__ void __launch_bounds__(256) sum_parts_kernel(const __grid_constant__ SumsList l) {
    __shared__ float part[8][32];
    const bool second = (int)blockIdx.x >= l.blocks0;
    const Sums s = l.a[second];  // in registers
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)(second ? blockIdx.x - l.blocks0 : blockIdx.x) * 32 + lane;
    float v = 0.f;
    after_previous_kernel();
    if (i < s.n) {
        const float* at = s.parts + i + warp * s.stride;
        const int64_t step = 8 * s.stride;
        int p = warp;
        for (; p + 56 < s.count; p += 64, at += 8 * step) {  // eight loads under way at a time
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = in_bounds<kChkWork>(at + k * step, 4) ? __ldg(at + k * step) : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) v += x[k];
        }
        float x[8] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (p + 8 * k < s.count && in_bounds<kChkWork>(at + k * step, 4)) x[k] = __ldg(at + k * step);
#pragma unroll
        for (int k = 0; k < 8; ++k) v += x[k];
    }
    part[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || i >= s.n) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) v += part[w][lane];
    if (s.out_type == 0) {
        float* p = static_cast<float*>(s.out) + i;
        if (in_bounds_role(s.role, p, 4)) *p = v;
    } else {
        T* p = static_cast<T*>(s.out) + i;
        if (in_bounds_role(s.role, p, sizeof(T))) *p = from_float<T>(v);
    }
}

}  // namespace linear
}  // namespace hg
