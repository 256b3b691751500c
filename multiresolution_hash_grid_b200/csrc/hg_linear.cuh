// hg_linear.cuh -- linear layers with their gradients.
//
//   forward:  z = x W^T + b;  y = act(z) + residual
//   backward: dz = dy act'(z);  dx = dz W;  dW = dz^T x;  db = sum over rows of dz
//
// All three products are D[m][n] = sum_k A(m, k) B(n, k) with 16-bit operands, exact products
// and fp32 sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "hg_check.cuh"

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
};

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
        if (in_bounds<kChkOut>(p, 4)) *p = y;
    } else {
        if (e.residual != nullptr) {
            const T* r = static_cast<const T*>(e.residual) + row * e.ldr + col;
            if (in_bounds<kChkResidual>(r, sizeof(T))) y += to_float(*r);
        }
        T* p = static_cast<T*>(e.out) + row * e.ldo + col;
        if (in_bounds<kChkOut>(p, sizeof(T))) *p = from_float<T>(y);
    }
}

// An operand: element (i, k) at p[i * si + k * sk], i < rows of the product's side.
struct Operand {
    const void* p;
    int64_t si, sk;
};

constexpr int kTileM = 64, kTileN = 64, kTileK = 16;

// D in 64 x 64 tiles, 4 x 4 values a thread, operands staged as fp32.
template <typename T>
__global__ void __launch_bounds__(256) product_kernel(Operand A, Operand B, int64_t M, int64_t N, int64_t K, Epilogue e) {
    __shared__ float as[kTileK][kTileM + 4], bs[kTileK][kTileN + 4];
    const int64_t m0 = (int64_t)blockIdx.x * kTileM, n0 = (int64_t)blockIdx.y * kTileN;
    const int tm = (threadIdx.x >> 4) * 4, tn = (threadIdx.x & 15) * 4;
    const T* a = static_cast<const T*>(A.p);
    const T* b = static_cast<const T*>(B.p);
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += kTileK) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // neighbouring threads along the operand's contiguous axis
            const int t = threadIdx.x + 256 * j;
            int i = A.sk == 1 ? t >> 4 : t & 63, k = A.sk == 1 ? t & 15 : t >> 6;
            as[k][i] = m0 + i < M && k0 + k < K ? to_float(a[(m0 + i) * A.si + (k0 + k) * A.sk]) : 0.f;
            i = B.sk == 1 ? t >> 4 : t & 63, k = B.sk == 1 ? t & 15 : t >> 6;
            bs[k][i] = n0 + i < N && k0 + k < K ? to_float(b[(n0 + i) * B.si + (k0 + k) * B.sk]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTileK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][tm + i], bs[k][tn + j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (m0 + tm + i < M && n0 + tn + j < N) emit<T>(e, m0 + tm + i, n0 + tn + j, acc[i][j]);
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

// out[col] = sum over parts of sums[part][col], in order.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ sums, int parts, int cols, float* __restrict__ out) {
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= cols) return;
    float s = 0.f;
    for (int p = 0; p < parts; ++p) s += sums[(int64_t)p * cols + col];
    if (in_bounds<kChkBias>(out + col, 4)) out[col] = s;
}

}  // namespace linear
}  // namespace hg
