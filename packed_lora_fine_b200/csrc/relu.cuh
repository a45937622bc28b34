// relu.cuh -- the signs of relu's Z, for a training forward on the tensor cores.
//
//   Z = X W + s (X A) B + b;   the backward takes dZ = dY where Z > 0 and 0 elsewhere
//
// That derivative jumps with Z's sign, so an error of Z that is nothing to any other activation turns a gradient
// entry into another where |Z| is below it; and an adapter with few rows has no other entries to hide it in.  The
// tensor cores' sums over d_in drift: measured over 4096 x 4096 outputs of Gaussian, uniform, one-sided and outlier
// inputs, Z near 0 is off by up to 0.8 (0.15 rms) times 2^-24 (d_in / 16) |x| |w| / sqrt(d_in), 6 to 7 times what
// fp32 sums are, and 10 times as many signs are wrong (41 of 16.8 million at d_in = 10808, none to 5 with fp32).
//
// So the forward's Z is gone over once more, and where it is below a bound on its error it is computed anew:
//   |Z| < e (|x| |w| / sqrt(d_in) + |b| + (|h| + s |x| |A| / sqrt(d_in)) |B_c|) + 2^-16 |h| |B_c|
//       from X W in fp64 and the two bf16 parts of H';
//   that < e sum_j max(|h_j|, s |x| |a_j| / sqrt(d_in)) |B_cj| + 2^-16 sum_j |h_j B_cj|
//       from A too, eight products at a time in fp32 and their sums in fp64;
//   that < 2^-20 of the first sum
//       all in fp64.
// with e = 1.25 2^-24 ((d_in + 2 P rblk) / 16 + 16), 1.5 times the largest drift seen and 8 times its rms, |h| the
// norm of the row's H' and |A| Frobenius's.  (A row or column whose norm leaves fp32's range, entries past 10^18 or
// all below 10^-22, is left alone.)  The norms are kept behind the low parts in `saved`.
#pragma once
#include <cuda_bf16.h>
#include "epilogue.cuh"
#include "plan.cuh"

namespace plora {

struct ReluArgs {
    const __nv_bfloat16* X;      // [T][d_in]
    const __nv_bfloat16* W;      // [d_out][d_in]
    const __nv_bfloat16* H;      // H''s high parts, rows of RP
    int64_t low;                 // elements from a high part to its low part
    const AdapterDev* ad;
    const TokTile* tok;          // [tiles]
    const void* const* bias;     // [n] (entries may be null), or null
    __nv_bfloat16* Y;            // null with a residual: Y then keeps what the base GEMM's epilogue wrote
    __nv_bfloat16* Z;
    float* nx;                   // [T] |x| / sqrt(d_in)
    float* nh;                   // [T] |h|
    float* nw;                   // [d_out] |w|
    float* na;                   // [n][RP] |a_j|, A_i's row j
    float* nb;                   // [n][d_out] |B_i's row|
    int64_t d_in, d_out;
    int32_t n, RP, tiles, pad_;
    OutBlocks blocks;
};

__host__ __device__ __forceinline__ int64_t relu_norm_items(const ReluArgs& a) {
    return (int64_t)a.tiles * kTileM + a.d_out + (int64_t)a.n * a.RP + (a.n * a.d_out + 7) / 8;
}

__device__ __forceinline__ float relu_warp_sum(float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// |v|^2 of k elements (a multiple of 8, 16-byte aligned), a warp's.
__device__ __forceinline__ float relu_square(const __nv_bfloat16* v, int64_t k) {
    float s = 0.f;
#pragma unroll 4
    for (int64_t e = (threadIdx.x & 31) * 8; e < k; e += 256) {
        float x[8];
        load8<__nv_bfloat16>(v + e, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) s = fmaf(x[q], x[q], s);
    }
    return relu_warp_sum(s);
}

// A warp per item: a token's X and H' rows, a row of W, a row of an A_i, eight rows of the B_i.
__global__ void __launch_bounds__(256) relu_norms_kernel(const __grid_constant__ ReluArgs a) {
    const int lane = threadIdx.x & 31;
    int64_t k = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (k < (int64_t)a.tiles * kTileM) {
        const TokTile t = a.tok[k / kTileM];
        const int row = (int)(k % kTileM);
        if (row >= t.rows) return;
        const float x = sqrtf(relu_square(a.X + (int64_t)(t.x_row + row) * a.d_in, a.d_in) / (float)a.d_in);
        const float h = sqrtf(relu_square(a.H + (int64_t)(t.h_row + row) * a.RP, a.RP));
        if (lane == 0) {
            a.nx[t.x_row + row] = x;
            a.nh[t.x_row + row] = h;
        }
        return;
    }
    k -= (int64_t)a.tiles * kTileM;
    if (k < a.d_out) {
        const float w = sqrtf(relu_square(a.W + k * a.d_in, a.d_in));
        if (lane == 0) a.nw[k] = w;
        return;
    }
    k -= a.d_out;
    if (k < (int64_t)a.n * a.RP) {
        const AdapterDev& ad = a.ad[k / a.RP];
        const int j = (int)(k % a.RP);
        if (j >= a.blocks.n * ad.rank) return;
        const float v = sqrtf(relu_square(static_cast<const __nv_bfloat16*>(ad.A) + j * a.d_in, a.d_in));
        if (lane == 0) a.na[k] = v;
        return;
    }
    k = (k - (int64_t)a.n * a.RP) * 8 + (lane >> 2);
    float s = 0.f;
    const bool in = k < a.n * a.d_out;
    if (in) {
        const AdapterDev& ad = a.ad[k / a.d_out];
        const __nv_bfloat16* const B = static_cast<const __nv_bfloat16*>(ad.B) + k % a.d_out * ad.rank;
        for (int j = lane & 3; j < ad.rank; j += 4) {
            const float v = __bfloat162float(B[j]);
            s = fmaf(v, v, s);
        }
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (in && (lane & 3) == 0) a.nb[k] = sqrtf(s);
}

__device__ __forceinline__ double relu_warp_sum(double v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// This lane's share of coef[j] u v_j, N vectors v_j of k elements `pitch` apart: in fp64 (the products are exact in
// fp32), or eight at a time in fp32.
template <bool EXACT, int N>
__device__ __forceinline__ double relu_dots(const __nv_bfloat16* u, const __nv_bfloat16* v, int64_t pitch, int64_t k,
                                            const double (&coef)[N]) {
    double s[N] = {};
#pragma unroll (N == 1 ? 4 : 2)
    for (int64_t e = (threadIdx.x & 31) * 8; e < k; e += 256) {
        Raw8<__nv_bfloat16> ru, rv[N];
        ru.load(u + e);
#pragma unroll
        for (int j = 0; j < N; ++j) rv[j].load(v + j * pitch + e);
        float x[8];
        ru.get(x);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float y[8];
            rv[j].get(y);
            if constexpr (EXACT) {
#pragma unroll
                for (int q = 0; q < 8; ++q) s[j] += (double)(x[q] * y[q]);
            } else {
                float p = 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q) p = fmaf(x[q], y[q], p);
                s[j] += (double)p;
            }
        }
    }
    double r = 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j) r += coef[j] * s[j];
    return r;
}

// One element of a tile: where its operands are.
struct ReluAt {
    const __nv_bfloat16 *x, *w, *h, *A, *B;
    const float* na;
    int64_t z;            // its place in Z and Y
    float bias, xs;       // s |x| / sqrt(d_in)
};

// Goes over one 128-row tile x 256 columns of Z: first every element against its bound (a thread has eight columns
// and every eighth row, as in act_grad_kernel), then a warp for each one below it, then the block for each that A
// decides.  Each element's value depends on its own row and column alone.
// 16384 x 4096 -> 14336, ranks 8 to 128: 344 us and 64 for the norms, next to 1450 for the forward; 8192 x 14336 -> 4096
// 280 and 67, next to 720 (the bytes of Z alone: 72 and 10).  What is left waits for the second look's rows of A, in a few
// blocks: one warp's dot products in turn took 1109 and 1966, the block's one by one 366 and 412.
__global__ void __launch_bounds__(256, 3) relu_signs_kernel(const __grid_constant__ ReluArgs a) {
    __shared__ uint32_t below[kTileM * 8], again[kTileM * 8];      // a bit per element: eight words per row
    __shared__ float norm_a;
    __shared__ double sums[8];
    const TokTile t = a.tok[blockIdx.y];
    const AdapterDev ad = a.ad[t.adapter];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col0 = (int64_t)blockIdx.x * kEpiCols, col = col0 + lane * 8;
    const __nv_bfloat16* const bias = a.bias ? static_cast<const __nv_bfloat16*>(a.bias[t.adapter]) : nullptr;
    const float scale = fabsf(ad.scale);
    if (warp == 0) {
        float s = 0.f;
        for (int j = lane; j < a.blocks.n * ad.rank; j += 32) {
            const float v = a.na[(int64_t)t.adapter * a.RP + j];
            s = fmaf(v, v, s);
        }
        s = relu_warp_sum(s);
        if (lane == 0) norm_a = sqrtf(s);
    }
    __syncthreads();
    const float eps = 7.4505806e-8f * ((float)(a.d_in + 2 * ad.rp16) * 0.0625f + 16.f), parts = 1.52587890625e-5f;
    uint8_t* const bytes = reinterpret_cast<uint8_t*>(below);
    bool any = false;
    {
        float w[8] = {}, b[8] = {}, fixed[8] = {};
        if (col < a.d_out) {
            load8<float>(a.nw + col, w);
            load8<float>(a.nb + (int64_t)t.adapter * a.d_out + col, b);
            if (bias) load8<__nv_bfloat16>(bias + col, fixed);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            w[k] *= eps;
            fixed[k] = fabsf(fixed[k]) * eps;
        }
        const float sa = eps * scale * norm_a;
        constexpr int kBatch = 4;
#pragma unroll
        for (int r0 = 0; r0 < kTileM; r0 += 8 * kBatch) {
            Raw8<__nv_bfloat16> raw[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int r = r0 + 8 * q + warp;
                if (col < a.d_out && r < t.rows) raw[q].load(a.Z + (int64_t)(t.x_row + r) * a.d_out + col);
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int r = r0 + 8 * q + warp;
                uint32_t bits = 0;
                if (col < a.d_out && r < t.rows) {
                    const float x = a.nx[t.x_row + r], h = a.nh[t.x_row + r];
                    const float low = fmaf(h, eps + parts, sa * x);
                    float z[8];
                    raw[q].get(z);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float bound = fmaf(x, w[k], fmaf(low, b[k], fixed[k]));
                        bits |= fabsf(z[k]) < bound && bound < 3e38f ? 1u << k : 0u;
                    }
                }
                bytes[r * 32 + lane] = (uint8_t)bits;
                any = any || bits;
            }
        }
    }
    for (int e = threadIdx.x; e < kTileM * 8; e += 256) again[e] = 0;
    if (!__syncthreads_or(any)) return;
    // f(word, bit) for every bit set in `set`, in order
    auto each = [&](const uint32_t* set, auto&& f) {
        for (int i = 0; i < kTileM * 8 / 32; ++i) {
            const uint32_t mine = set[i * 32 + lane];
            for (uint32_t left = __ballot_sync(0xffffffffu, mine != 0); left; left &= left - 1) {
                const int src = __ffs((int)left) - 1;
                for (uint32_t v = __shfl_sync(0xffffffffu, mine, src); v; v &= v - 1) f(i * 32 + src, __ffs((int)v) - 1);
            }
        }
    };
    auto at = [&](int word, int bit) {
        const int r = word >> 3;
        const int64_t c = col0 + (word & 7) * 32 + bit, row = t.x_row + r;
        int blk = 0;
        while (blk + 1 < a.blocks.n && c >= a.blocks.end[blk]) ++blk;
        ReluAt p;
        p.x = a.X + row * a.d_in;
        p.w = a.W + c * a.d_in;
        p.h = a.H + (int64_t)(t.h_row + r) * a.RP + blk * ad.rblk;
        p.A = static_cast<const __nv_bfloat16*>(ad.A) + (int64_t)blk * ad.rank * a.d_in;
        p.B = static_cast<const __nv_bfloat16*>(ad.B) + c * ad.rank;
        p.na = a.na + (int64_t)t.adapter * a.RP + blk * ad.rank;
        p.z = row * a.d_out + c;
        p.bias = bias ? __bfloat162float(bias[c]) : 0.f;
        p.xs = scale * a.nx[row];
        return p;
    };
    // sum_j max(|h_j|, s |x| |a_j| / sqrt(d_in)) |B_cj|, and sum_j |h_j B_cj|
    auto size_of = [&](const ReluAt& p, float& held) {
        float most = 0.f;
        held = 0.f;
        for (int j = lane; j < ad.rank; j += 32) {
            const float h = fabsf(__bfloat162float(p.h[j])), b = fabsf(__bfloat162float(p.B[j]));
            most = fmaf(fmaxf(h, p.xs * p.na[j]), b, most);
            held = fmaf(h, b, held);
        }
        held = relu_warp_sum(held);
        return relu_warp_sum(most);
    };
    auto put = [&](const ReluAt& p, double z) {
        const float f = (float)z;
        a.Z[p.z] = __float2bfloat16_rn(f);
        if (a.Y) a.Y[p.z] = __float2bfloat16_rn(act_fwd<__nv_bfloat16, kActRelu>(f));
    };
    int turn = 0;                                // the warps take the elements in turn
    each(below, [&](int word, int bit) {
        if ((turn++ & 7) != warp) return;
        const ReluAt p = at(word, bit);
        double z = relu_dots<true, 1>(p.x, p.w, 0, a.d_in, {1.0});
        for (int j = lane; j < ad.rank; j += 32)
            z += ((double)__bfloat162float(p.h[j]) + (double)__bfloat162float(p.h[a.low + j])) * (double)__bfloat162float(p.B[j]);
        z = relu_warp_sum(z) + (double)p.bias;
        float held;
        const float most = size_of(p, held);
        if (lane != 0) return;
        if (fabs(z) < (double)(eps * most + parts * held)) atomicOr(&again[word], 1u << bit);
        else put(p, z);
    });
    __syncthreads();
    each(again, [&](int word, int bit) {
        const ReluAt p = at(word, bit);
        float held;
        const double sure = (double)(9.5367431640625e-7f * size_of(p, held));      // 2^-20
        double z = 0.0;
        for (int exact = 0; exact < 2; ++exact) {
            double v = 0.0;
            // the warps share the rank's products, four at a time and the rest one by one, and X W's
            const int whole = ad.rank & ~3;
            auto coef = [&](int j) { return (double)ad.scale * (double)__bfloat162float(p.B[j]); };
            for (int j = 4 * warp; j < whole; j += 32) {
                const double c[4] = {coef(j), coef(j + 1), coef(j + 2), coef(j + 3)};
                const __nv_bfloat16* const A = p.A + j * a.d_in;
                v += exact ? relu_dots<true, 4>(p.x, A, a.d_in, a.d_in, c) : relu_dots<false, 4>(p.x, A, a.d_in, a.d_in, c);
            }
            if (whole + warp < ad.rank) {
                const double c[1] = {coef(whole + warp)};
                const __nv_bfloat16* const A = p.A + (whole + warp) * a.d_in;
                v += exact ? relu_dots<true, 1>(p.x, A, 0, a.d_in, c) : relu_dots<false, 1>(p.x, A, 0, a.d_in, c);
            }
            if (warp == 7) v += relu_dots<true, 1>(p.x, p.w, 0, a.d_in, {1.0});
            v = relu_warp_sum(v);
            __syncthreads();
            if (lane == 0) sums[warp] = v;
            __syncthreads();
            z = (double)p.bias;
            for (int q = 0; q < 8; ++q) z += sums[q];
            if (!(fabs(z) < sure)) break;
        }
        if (threadIdx.x == 0) put(p, z);
    });
}

}  // namespace plora
