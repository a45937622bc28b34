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

// act(z) and act'(z) for results of type T.  fp32 uses CUDA's accurate functions.  bf16 results keep 9 of 24
// bits, so theirs use the fast exponential and division and no branch, whose 64
// divisions per thread and chunk would otherwise run one after another.  The exponential is off by 2 + 1.16 |x| units
// of its last place: a tail's relative error grows with |z|, but what a function is off by stays below 2^-21 of |z|
// (2^-19 for the derivatives, absolute):
//   tanh form: (1 + tanh y) / 2 = 1 / (1 + exp(-2 y))
//   erf form:  Abramowitz and Stegun 7.1.26, erfc(x) = t (a1 + ... + a5 t^4) exp(-x^2), t = 1 / (1 + p x), x >= 0,
//              absolute error 1.5e-7, and exp(-z^2/2) serves the derivative as well
// A quotient past 2^126 is 0 (values below 1e-36).
// The logistic function of z and of -z (their sum is 1), each to its own relative accuracy.
__device__ __forceinline__ void fast_logistic(float z, float& s, float& r) {
    const float e = __expf(-fabsf(z)), more = __fdividef(1.f, 1.f + e), less = e * more;
    s = z < 0.f ? less : more;
    r = z < 0.f ? more : less;
}
// Phi(z), the normal distribution, and e = exp(-z^2/2)
__device__ __forceinline__ float fast_normal(float z, float& e) {
    const float t = __fdividef(1.f, fmaf(0.3275911f * kInvSqrt2, fabsf(z), 1.f));
    e = __expf(-0.5f * z * z);
    float q = fmaf(t, 1.061405429f, -1.453152027f);
    q = fmaf(t, q, 1.421413741f);
    q = fmaf(t, q, -0.284496736f);
    q = fmaf(t, q, 0.254829592f);
    const float tail = 0.5f * t * q * e;
    return z < 0.f ? tail : 1.f - tail;
}
// y of gelu_tanh and dy/dz / y': past |z| = 100 the functions have their limits
__device__ __forceinline__ float gelu_square(float z) { return fminf(z * z, 1e4f); }

template <typename T, int ACT> __device__ __forceinline__ float act_fwd(float z) {
    constexpr bool kFast = sizeof(T) == 2;
    if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;   // a NaN stays a NaN
    if constexpr (ACT == kActGelu) {
        if constexpr (kFast) {
            float e;
            return z * fast_normal(z, e);
        } else {
            return 0.5f * z * (1.f + erff(z * kInvSqrt2));
        }
    }
    if constexpr (ACT == kActGeluTanh) {
        const float y = kSqrt2OverPi * z * fmaf(kGeluCubic, gelu_square(z), 1.f);
        return kFast ? __fdividef(z, 1.f + __expf(-2.f * y)) : 0.5f * z * (1.f + tanhf(y));
    }
    if constexpr (ACT == kActSilu) return kFast ? __fdividef(z, 1.f + __expf(-z)) : z / (1.f + expf(-z));
    return z;
}

template <typename T, int ACT> __device__ __forceinline__ float act_bwd(float z) {
    constexpr bool kFast = sizeof(T) == 2;
    if constexpr (ACT == kActRelu) return z <= 0.f ? 0.f : 1.f;
    if constexpr (ACT == kActGelu) {
        if constexpr (kFast) {
            float e;
            const float phi = fast_normal(z, e);
            return fmaf(z * kInvSqrt2Pi, e, phi);
        } else {
            return 0.5f * (1.f + erff(z * kInvSqrt2)) + z * kInvSqrt2Pi * expf(-0.5f * z * z);
        }
    }
    if constexpr (ACT == kActGeluTanh) {
        const float z2 = gelu_square(z), y = kSqrt2OverPi * z * fmaf(kGeluCubic, z2, 1.f);
        const float dy = kSqrt2OverPi * fmaf(3.f * kGeluCubic, z2, 1.f);
        if constexpr (kFast) {
            float s, r;
            fast_logistic(2.f * y, s, r);
            return fmaf(2.f * z * dy, s * r, s);
        } else {
            const float t = tanhf(y);
            return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * dy;
        }
    }
    if constexpr (ACT == kActSilu) {
        if constexpr (kFast) {
            float s, r;
            fast_logistic(z, s, r);
            return s * fmaf(z, r, 1.f);
        } else {
            const float s = 1.f / (1.f + expf(-z));
            return s * (1.f + z * (1.f - s));
        }
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

// Eight consecutive values of a row (16-byte aligned in bf16, 32 bytes in fp32), as they were read and as floats.
template <typename T> struct Raw8 {
    uint4 w[sizeof(T) == 2 ? 1 : 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) w[k] = reinterpret_cast<const uint4*>(p)[k];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (sizeof(T) == 2) {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[k]));
                    v[2 * k] = f.x;
                    v[2 * k + 1] = f.y;
                } else {
                    v[4 * i + k] = __uint_as_float(u[k]);
                }
            }
        }
    }
};
template <typename T> __device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    Raw8<T> r;
    r.load(p);
    r.get(v);
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
    int32_t pad_;
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
                z[k] = act_fwd<T, ACT.value>(z[k]);
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
// per 128 rows.  16384 x 14336, silu: 238 us, 5.9 TB/s (357 us with one row's loads at a time and the accurate
// functions).
template <typename T>
__global__ void __launch_bounds__(256) act_grad_kernel(const __grid_constant__ ActGradArgs a) {
    __shared__ float sums[8][kEpiCols];
    const TokTile t = a.tok[blockIdx.y];
    const int lane = threadIdx.x & 31, rg = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * kEpiCols + lane * 8;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col < a.d_out) {
        with_act(a.act, [&](auto ACT) {
            const int64_t at0 = (int64_t)t.x_row * a.d_out + col;
            if constexpr (ACT.value == kActNone) {
                const T* src = static_cast<const T*>(a.dY) + at0;
#pragma unroll 8
                for (int r = rg; r < t.rows; r += 8) {
                    float v[8];
                    load8<T>(src + (int64_t)r * a.d_out, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum[k] += v[k];
                }
                return;
            }
            // a batch's loads are requested before its first store (which the compiler would not move them over)
            constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
            for (int r0 = rg; r0 < t.rows; r0 += 8 * kBatch) {
                Raw8<T> d[kBatch], z[kBatch];
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const int64_t at = at0 + (int64_t)min(r0 + 8 * q, t.rows - 1) * a.d_out;
                    d[q].load(static_cast<const T*>(a.dY) + at);
                    z[q].load(static_cast<const T*>(a.Z) + at);
                }
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    if (r0 + 8 * q >= t.rows) break;
                    float v[8], x[8];
                    d[q].get(v);
                    z[q].get(x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] *= act_bwd<T, ACT.value>(x[k]);
                    store8<T>(static_cast<T*>(a.dZ) + at0 + (int64_t)(r0 + 8 * q) * a.d_out, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum[k] += v[k];
                }
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
