// few.cuh -- the projection with its epilogue over a few tokens, for inference (nothing kept for a backward).
//
//   H = s_i X_i A_i,   Z = X W + H B_i + b_i,   Y = act(Z) + R,   at most kFewTokens rows in all
//
// Bound by the one reading of W (and of A_i and B_i), so two streaming kernels take the place of the 256-row
// tensor-core tiles, of which a few tokens would fill a small part and a layer's columns too few blocks: for
// 3584 x 3584 14 blocks, which read W at 0.5 TB/s.  Eight tokens of eight adapters of rank 32: 9.9 us (the
// bytes' floor 4.5; 76 through the training kernels), 14336 x 4096, rank 64: 29 (21; 240).  At 32 tokens 20 us
// against 76, and 62 against 240; past that the tiles fill up and their kernels take over.
//
// A block computes 16 rows of the streamed matrix (W's, or A_i's) times the tokens.  Its eight warps take the 64-
// element slices of K in turn; a lane reads 16 consecutive bytes of a row, two rows and two halves of a slice at a
// time.  The products are mma.m16n8k16: K's order within a slice is free, so a lane's eight elements are its
// operands of two products, the tokens' likewise, and nothing passes through shared memory but the warps' sums.
// Every sum's order depends on K alone: a token's result does not depend on what else is in the call.
#pragma once
#include <cuda_bf16.h>
#include "epilogue.cuh"
#include "plan.cuh"
#include "ptx.cuh"

namespace plora {

constexpr int kFewTokens = 32;
constexpr int kFewRows = 16;       // rows of the streamed matrix per block

struct FewAdapter {                // an adapter with tokens
    const __nv_bfloat16* A;        // [P rank][d_in]
    const __nv_bfloat16* B;        // [d_out][rank]
    const __nv_bfloat16* bias;     // [d_out] or null
    float scale;
    int32_t rank;
    int32_t x_row, n;
    int32_t tile0;                 // its first block of the shrink
    int32_t pad_;
};
struct FewArgs {
    const __nv_bfloat16* X;        // [T][d_in]
    const __nv_bfloat16* W;        // [d_out][d_in]
    const __nv_bfloat16* residual; // [T][d_out] or null (may be Y)
    __nv_bfloat16* Y;
    float* H;                      // [T][RP]: column b rank + k of output block b
    int64_t d_in, d_out;
    int32_t T, RP, n, act;
    OutBlocks blocks;
    uint8_t owner[kFewTokens];     // the adapter of each token
    FewAdapter ad[kFewTokens];
};

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// sums[warp][16 rows][8 NT tokens] = this warp's share of (`rows` <= 16 rows at M) x (`tokens` rows at X), K each.
// Up to eight tokens the next slices' loads are requested before a slice's products (14336 x 4096, one token: 24 us
// against 44 without); for more the tokens' own loads, from L2, are the larger part (32 rows per block, which halves
// them, took 16.7 us for 12.4 at 3584 x 3584, 16 tokens, and 71 for 80 at 4096 x 14336, 32 tokens: not kept).
template <int NT>
__device__ __forceinline__ void few_product(const __nv_bfloat16* M, int rows, const __nv_bfloat16* X, int tokens, int64_t K,
                                            float* sums) {
    constexpr int U = 2, BUFS = NT == 1 ? 2 : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int64_t step = 8 * 64 * U, kl = (lane & 3) * 8;
    float acc[NT][4] = {};
    uint4 a[BUFS][U][2][2], x[BUFS][U][2][NT];
    auto fetch = [&](int64_t k0, int buf) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = k0 + kl + u * 512 + h * 32;
                const bool in = k < K;
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    a[buf][u][h][r] = in && 8 * r + g < rows ? __ldg(reinterpret_cast<const uint4*>(M + (8 * r + g) * K + k)) : zero;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    x[buf][u][h][t] = in && 8 * t + g < tokens ? __ldg(reinterpret_cast<const uint4*>(X + (8 * t + g) * K + k)) : zero;
            }
    };
    auto multiply = [&](int buf) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 &p = a[buf][u][h][0], &q = a[buf][u][h][1], &y = x[buf][u][h][t];
                    mma_16x8x16(acc[t], p.x, q.x, p.y, q.y, y.x, y.y);
                    mma_16x8x16(acc[t], p.z, q.z, p.w, q.w, y.z, y.w);
                }
    };
    int64_t k0 = warp * 64;
    if constexpr (BUFS == 2) {
        fetch(k0, 0);
        while (k0 < K) {
            fetch(k0 + step, 1);
            multiply(0);
            k0 += step;
            if (k0 >= K) break;
            fetch(k0 + step, 0);
            multiply(1);
            k0 += step;
        }
    } else {
        for (; k0 < K; k0 += step) {
            fetch(k0, 0);
            multiply(0);
        }
    }
    float* const mine = sums + warp * (kFewRows * 8 * NT);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(g + (i >> 1) * 8) * (8 * NT) + 8 * t + (lane & 3) * 2 + (i & 1)] = acc[t][i];
    __syncthreads();
}
template <int NT> __device__ __forceinline__ float few_sum(const float* sums, int row, int token) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sums[(w * kFewRows + row) * (8 * NT) + token];
    return v;
}

// H of 16 of an adapter's rank rows.
template <int NT>
__global__ void __launch_bounds__(256) few_shrink_kernel(const __grid_constant__ FewArgs a) {
    __shared__ float sums[8 * kFewRows * 8 * NT];
    ptx::grid_launch_dependents();
    int i = 0;
    while (i + 1 < a.n && (int)blockIdx.x >= a.ad[i + 1].tile0) ++i;
    const FewAdapter& ad = a.ad[i];
    const int row0 = ((int)blockIdx.x - ad.tile0) * kFewRows;
    few_product<NT>(ad.A + row0 * a.d_in, min(kFewRows, a.blocks.n * ad.rank - row0), a.X + ad.x_row * a.d_in, ad.n, a.d_in,
                    sums);
    for (int e = threadIdx.x; e < kFewRows * ad.n; e += 256) {
        const int row = e & (kFewRows - 1), t = e / kFewRows;
        if (row0 + row < a.blocks.n * ad.rank)
            a.H[(int64_t)(ad.x_row + t) * a.RP + row0 + row] = ad.scale * few_sum<NT>(sums, row, t);
    }
}

// 16 columns of Y.  W's products do not wait for the shrink; four lanes share an output's low-rank sum.
template <int NT>
__global__ void __launch_bounds__(256, 2) few_base_kernel(const __grid_constant__ FewArgs a) {
    __shared__ float sums[8 * kFewRows * 8 * NT];
    const int64_t col0 = (int64_t)blockIdx.x * kFewRows;
    const int cols = (int)min((int64_t)kFewRows, a.d_out - col0), part = threadIdx.x & 3;
    few_product<NT>(a.W + col0 * a.d_in, cols, a.X, a.T, a.d_in, sums);
    ptx::grid_wait();
    for (int o = threadIdx.x >> 2; o < kFewRows * a.T; o += 64) {      // (a warp's eight outputs: all or none)
        const int c = o & (kFewRows - 1), t = o / kFewRows;
        const bool in = c < cols;
        const int64_t col = col0 + (in ? c : 0);
        const FewAdapter& ad = a.ad[a.owner[t]];
        int b = 0;
        while (b + 1 < a.blocks.n && col >= a.blocks.end[b]) ++b;
        const float* const h = a.H + (int64_t)t * a.RP + b * ad.rank;
        const __nv_bfloat16* const B = ad.B + col * ad.rank;
        float low = 0.f;
        if ((ad.rank & 7) == 0) {
#pragma unroll 4
            for (int k = part * 8; k < ad.rank; k += 32) {
                float w[8], v[8];
                load8<__nv_bfloat16>(B + k, w);
                *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(h + k));
                *reinterpret_cast<float4*>(v + 4) = __ldcg(reinterpret_cast<const float4*>(h + k + 4));
#pragma unroll
                for (int q = 0; q < 8; ++q) low = fmaf(v[q], w[q], low);
            }
        } else {
            for (int k = part; k < ad.rank; k += 4) low = fmaf(__ldcg(h + k), __bfloat162float(B[k]), low);
        }
        low += __shfl_xor_sync(0xffffffffu, low, 1);
        low += __shfl_xor_sync(0xffffffffu, low, 2);
        if (part || !in) continue;
        float z = few_sum<NT>(sums, c, t) + low;
        if (ad.bias) z += __bfloat162float(ad.bias[col]);
        const int64_t at = t * a.d_out + col;
        with_act(a.act, [&](auto ACT) { z = act_fwd<__nv_bfloat16, ACT.value>(z); });
        if (a.residual) z += __bfloat162float(a.residual[at]);
        a.Y[at] = __float2bfloat16(z);
    }
}

}  // namespace plora
