// epilogue.cuh -- the projection's epilogue outside the tensor-core kernel: bias, activation and
// residual of the fp32 path, and the backward's dZ = dY * act'(Z) with the bias gradient.
//
//   Z_i = X_i W + s_i (X_i A_i) B_i + b_i,   Y = act(Z) + R
//   dZ = dY * act'(Z),   db_i = sum of dZ over adapter i's rows,   dR = dY
//
// On the tensor-core path Y and Z are finished in the base GEMM's own epilogue (tc.cuh).
#pragma once
#include <cuda_bf16.h>
#include <type_traits>
#include "plan.cuh"
#include "simt.cuh"

namespace plora {

// plora_activation
enum : int32_t { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

constexpr float kInvSqrt2 = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kGeluCubic = 0.044715f;

template <int ACT> __device__ __forceinline__ float act_fwd(float z) {
    if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;   // a NaN stays a NaN
    if constexpr (ACT == kActGelu) return 0.5f * z * (1.f + erff(z * kInvSqrt2));
    if constexpr (ACT == kActGeluTanh) return 0.5f * z * (1.f + tanhf(kSqrt2OverPi * z * (1.f + kGeluCubic * z * z)));
    if constexpr (ACT == kActSilu) return z / (1.f + expf(-z));
    return z;
}

template <int ACT> __device__ __forceinline__ float act_bwd(float z) {
    if constexpr (ACT == kActRelu) return z <= 0.f ? 0.f : 1.f;
    if constexpr (ACT == kActGelu)
        return 0.5f * (1.f + erff(z * kInvSqrt2)) + z * kInvSqrt2Pi * expf(-0.5f * z * z);
    if constexpr (ACT == kActGeluTanh) {
        const float t = tanhf(kSqrt2OverPi * z * (1.f + kGeluCubic * z * z));
        return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z);
    }
    if constexpr (ACT == kActSilu) {
        const float s = 1.f / (1.f + expf(-z));
        return s * (1.f + z * (1.f - s));
    }
    return 1.f;
}

// Calls f with the activation as a compile-time constant.
template <typename F> __device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
        case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
        case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
        case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
        default: f(std::integral_constant<int, kActNone>{}); break;
    }
}

// Eight consecutive values of a row as floats (16-byte aligned in bf16, 32 bytes in fp32).
template <typename T> __device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
            v[2 * k] = f.x;
            v[2 * k + 1] = f.y;
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
}

constexpr int kEpiCols = 256;   // columns of one block of the elementwise kernels: 32 threads x 8

struct EpiArgs {
    int32_t act;
    int32_t n_adapters;
    int64_t d_out;
    const TokTile* tok;          // 128-row tiles of the adapters' tokens
    const void* const* bias;     // [n] device pointers (entries may be null), or null
    const void* residual;        // [T][d_out] or null
    void* Y;
    void* Z;                     // [T][d_out] or null
};

// Finishes the fp32 path's output in place: Y holds X W + s (X A) B.  grid (column blocks, tiles),
// block 32 x 8: a thread owns eight columns and every eighth row of the tile.  Memory bound.
template <typename T>
__global__ void __launch_bounds__(256) epilogue_kernel(const __grid_constant__ EpiArgs a) {
    const TokTile t = a.tok[blockIdx.y];
    const int64_t col = (int64_t)blockIdx.x * kEpiCols + (threadIdx.x & 31) * 8;
    if (col >= a.d_out) return;
    float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const T* bias = a.bias ? static_cast<const T*>(a.bias[t.adapter]) : nullptr;
    if (bias) load8<T>(bias + col, b);
    with_act(a.act, [&](auto ACT) {
        for (int r = threadIdx.x >> 5; r < t.rows; r += 8) {
            const int64_t at = (int64_t)(t.x_row + r) * a.d_out + col;
            float z[8], res[8];
            load8<T>(static_cast<const T*>(a.Y) + at, z);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] += b[k];
            if (a.Z) store8<T>(static_cast<T*>(a.Z) + at, z);
            if (a.residual) load8<T>(static_cast<const T*>(a.residual) + at, res);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                z[k] = act_fwd<ACT.value>(z[k]);
                if (a.residual) z[k] += res[k];
            }
            store8<T>(static_cast<T*>(a.Y) + at, z);
        }
    });
}

struct ActGradArgs {
    int32_t act;
    int32_t pad_;
    int64_t d_out;
    const TokTile* tok;
    const void* dY;
    const void* Z;               // null without an activation
    void* dZ;                    // null without an activation
    float* part;                 // [tiles][d_out] column sums of a tile's dZ, or null
};

// dZ = dY * act'(Z) over one 128-row tile x 256 columns, with the tile's column sums of dZ before its
// rounding (fp32: each thread sums 16 rows, the eight row groups then add up in a fixed order).
// Memory bound: reads dY and Z, writes dZ, 6 bytes per element in bf16; the partial sums add 4 bytes
// per 128 rows.
template <typename T>
__global__ void __launch_bounds__(256) act_grad_kernel(const __grid_constant__ ActGradArgs a) {
    __shared__ float sums[8][kEpiCols];
    const TokTile t = a.tok[blockIdx.y];
    const int lane = threadIdx.x & 31, rg = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * kEpiCols + lane * 8;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col < a.d_out) {
        with_act(a.act, [&](auto ACT) {
#pragma unroll 4
            for (int r = rg; r < t.rows; r += 8) {
                const int64_t at = (int64_t)(t.x_row + r) * a.d_out + col;
                float d[8];
                load8<T>(static_cast<const T*>(a.dY) + at, d);
                if constexpr (ACT.value != kActNone) {
                    float z[8];
                    load8<T>(static_cast<const T*>(a.Z) + at, z);
#pragma unroll
                    for (int k = 0; k < 8; ++k) d[k] *= act_bwd<ACT.value>(z[k]);
                    store8<T>(static_cast<T*>(a.dZ) + at, d);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] += d[k];
            }
        });
    }
    if (!a.part) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[rg][lane * 8 + k] = sum[k];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * kEpiCols + threadIdx.x;
    if (c >= a.d_out) return;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) s += sums[r][threadIdx.x];
    a.part[(int64_t)blockIdx.y * a.d_out + c] = s;
}

// db_i = the sum of adapter i's tile sums, in tile order (so it does not depend on what else is packed
// with it); zero for an adapter without tokens.  grid (column blocks, adapters).
__global__ void __launch_bounds__(256) bias_grad_kernel(const AdapterDev* __restrict__ ad, float* const* __restrict__ db,
                                                        const int32_t* __restrict__ tile0,
                                                        const float* __restrict__ part, int64_t d_out) {
    const int i = blockIdx.y;
    float* out = db[i];
    const int64_t c = (int64_t)blockIdx.x * kEpiCols + threadIdx.x;
    if (!out || c >= d_out) return;
    const int tiles = (ad[i].n + kTileM - 1) / kTileM;
    const float* src = part + (int64_t)tile0[i] * d_out + c;
    float s = 0.f;
#pragma unroll 8
    for (int t = 0; t < tiles; ++t) s += src[(int64_t)t * d_out];
    out[c] = s;
}

}  // namespace plora
