// muon.cuh -- one Muon step for every adapter of a packed job.
//
// Per matrix M (an adapter's A or B, one per output block):
//   m <- mu m + g,   u = g + mu m (Nesterov) or m,   X_0 = u / (|u|_F + eps)
//   X_{k+1} = (a I + b X_k X_k^T + c (X_k X_k^T)^2) X_k        (Newton-Schulz, on the short side)
//   p <- p (1 - lr wd) - lr k X_n
// Every iterate is a polynomial in the Gram matrix of u times u.  So, with s the short side and L the
// long one, the step is one pass that forms G = u u^T (s x s), the iteration on s x s matrices
//   P_k = a I + b G_k + c G_k^2,   Q_{k+1} = P_k Q_k,   G_{k+1} = P_k G_k P_k,
// and one pass that applies O = Q_n X_0 and updates p and m: two passes over u instead of two for each
// of the n steps.  G squares the condition of u, so it and the iteration are kept in 64 bits: small
// singular values grow by a per step, and rounding G to 32 bits would grow by a^2 with them (at ten
// percent of the singular values' range the 32-bit form was 50 to 100 times further from the formula
// than iterating on X itself; the 64-bit form is nearer).
//
// The first pass reads g and m without writing, so that several blocks may read the same element; the
// second pass owns its columns and writes m.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

namespace plora {

constexpr int kMuonChunk = 1024;    // long-side extent of one Gram partial
constexpr int kMuonTile = 64;       // Gram tile (rows and columns) of a block
constexpr int kMuonApply = 32;      // long-side extent of an apply block
constexpr int kMuonNsTile = 32;     // product tile of the iteration
constexpr int kMuonCluster = 8;     // blocks per matrix in the iteration

// One matrix of the step.  Element (c, l), c on the short side: c * L + l if !tall, l * s + c if tall.
struct MuonMat {
    const float* g;
    float* m;
    float* p;
    __nv_bfloat16* out;   // the layer's bf16 copy, or nullptr when p is the parameter
    double* part;         // [nchunks][s][s] Gram partials
    double* ns;           // four [s][s] matrices of the iteration
    float* Q;             // [s][s], then 1 / (|u|_F + eps)
    int32_t s, L;
    int32_t tall, nesterov;
    int32_t steps, nchunks;
    int32_t gram0;        // first block of this matrix in the Gram launch
    int32_t apply0;       // first block in the apply launch
    float mu, decay;      // decay = 1 - lr wd
    float step, eps;      // step = lr k
    float a, b, c;
    int32_t pad_;
};
static_assert(sizeof(MuonMat) % 8 == 0, "MuonMat layout");

__device__ __forceinline__ int64_t muon_at(const MuonMat& M, int c, int l) {
    return M.tall ? (int64_t)l * M.s + c : (int64_t)c * M.L + l;
}
__device__ __forceinline__ float muon_m(const MuonMat& M, float m, float g) { return fmaf(M.mu, m, g); }
__device__ __forceinline__ float muon_u(const MuonMat& M, float m_new, float g) {
    return M.nesterov ? fmaf(M.mu, m_new, g) : m_new;
}
// u of one element, from the momentum before the step
__device__ __forceinline__ float muon_load_u(const MuonMat& M, int64_t e) {
    const float g = M.g[e];
    return muon_u(M, muon_m(M, M.m[e], g), g);
}

// The matrix whose blocks hold block `b` (begin: the prefix each matrix records).
template <typename F> __device__ __forceinline__ int muon_find(int n, int b, F&& begin) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (begin(mid) <= b) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Gram partial of one chunk, one 64 x 64 tile (ti <= tj) per block, 4 x 4 sums per thread in fp64.
__global__ void __launch_bounds__(256) muon_gram_kernel(const MuonMat* __restrict__ mats, int n) {
    __shared__ float us[2][16][kMuonTile + 1];
    const int mi = muon_find(n, blockIdx.x, [&](int k) { return mats[k].gram0; });
    const MuonMat M = mats[mi];
    const int nt = (M.s + kMuonTile - 1) / kMuonTile, pairs = nt * (nt + 1) / 2;
    const int b = blockIdx.x - M.gram0;
    const int chunk = b / pairs;
    int t = b - chunk * pairs, ti = 0;
    while (t >= nt - ti) { t -= nt - ti; ++ti; }
    const int tj = ti + t;
    const int l0 = chunk * kMuonChunk, l1 = min(M.L, l0 + kMuonChunk);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    double acc[4][4] = {};
    for (int l = l0; l < l1; l += 16) {
        for (int e = threadIdx.x; e < 2 * 16 * kMuonTile; e += 256) {
            const int w = e / (16 * kMuonTile), f = e - w * 16 * kMuonTile;
            int cc, ll;   // consecutive threads on consecutive addresses
            if (M.tall) { cc = f & 63; ll = f >> 6; } else { ll = f & 15; cc = f >> 4; }
            const int c = (w ? tj : ti) * kMuonTile + cc;
            us[w][ll][cc] = (c < M.s && l + ll < l1) ? muon_load_u(M, muon_at(M, c, l + ll)) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            double x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { x[i] = us[0][k][ty + 16 * i]; y[i] = us[1][k][tx + 16 * i]; }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fma(x[i], y[j], acc[i][j]);
        }
        __syncthreads();
    }
    double* out = M.part + (int64_t)chunk * M.s * M.s;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = ti * kMuonTile + ty + 16 * i, c = tj * kMuonTile + tx + 16 * j;
            if (r < M.s && c < M.s) {
                out[(int64_t)r * M.s + c] = acc[i][j];
                if (ti != tj) out[(int64_t)c * M.s + r] = acc[i][j];
            }
        }
}

// C = A B for symmetric s x s matrices that commute (so C is symmetric and B's rows serve as its
// columns), tiles dealt over the cluster's blocks; out(r, c, v) takes each element.  256 threads: four
// slices of K, each 8 x 8 threads of 4 x 4 sums over a 32 x 32 tile.
template <typename F>
__device__ __forceinline__ void ns_product(const double* A, const double* B, int s, int rank, double* sm, F&& out) {
    constexpr int T = kMuonNsTile, K = 32;
    double* as = sm;                 // [K][T + 1]
    double* bs = sm + K * (T + 1);
    double* red = bs + K * (T + 1);  // [3][T * T]
    const int nt = (s + T - 1) / T;
    const int slice = threadIdx.x >> 6, th = threadIdx.x & 63, tx = th & 7, ty = th >> 3;
    for (int t = rank; t < nt * nt; t += kMuonCluster) {
        const int r0 = (t / nt) * T, c0 = (t % nt) * T;
        double acc[4][4] = {};
        for (int k0 = 0; k0 < s; k0 += K) {
            for (int e = threadIdx.x; e < T * K; e += 256) {
                const int k = e & (K - 1), x = e / K;
                as[k * (T + 1) + x] = (r0 + x < s && k0 + k < s) ? __ldcg(A + (int64_t)(r0 + x) * s + k0 + k) : 0.0;
                bs[k * (T + 1) + x] = (c0 + x < s && k0 + k < s) ? __ldcg(B + (int64_t)(c0 + x) * s + k0 + k) : 0.0;
            }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < K / 4; ++kk) {
                const int k = slice * (K / 4) + kk;
                double x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) { x[i] = as[k * (T + 1) + ty + 8 * i]; y[i] = bs[k * (T + 1) + tx + 8 * i]; }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fma(x[i], y[j], acc[i][j]);
            }
            __syncthreads();
        }
        if (slice > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) red[(slice - 1) * T * T + (ty + 8 * i) * T + tx + 8 * j] = acc[i][j];
        }
        __syncthreads();
        if (slice == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = (ty + 8 * i) * T + tx + 8 * j;
                    const double v = ((acc[i][j] + red[at]) + red[T * T + at]) + red[2 * T * T + at];
                    const int r = r0 + ty + 8 * i, c = c0 + tx + 8 * j;
                    if (r < s && c < s) out(r, c, v);
                }
        }
        __syncthreads();
    }
}

constexpr int kMuonNsSmem = (2 * 32 * (kMuonNsTile + 1) + 3 * kMuonNsTile * kMuonNsTile) * 8;

// The iteration on one matrix's s x s Gram matrix: a cluster of eight blocks per matrix, the matrices
// in L2, one cluster barrier after each product.
__global__ void __cluster_dims__(kMuonCluster, 1, 1) __launch_bounds__(256)
muon_ns_kernel(const MuonMat* __restrict__ mats) {
    extern __shared__ double sm[];
    __shared__ double norm_part[8];
    const MuonMat M = mats[blockIdx.x / kMuonCluster];
    const int rank = (int)ptx::cluster_ctarank();
    const int s = M.s;
    const int64_t n2 = (int64_t)s * s;
    double* G = M.ns;
    double* P = G + n2;
    double* R = P + n2;
    double* Q = R + n2;
    // |u|_F^2 = the trace of G, summed by every block in the same order
    double tr = 0.0;
    for (int e = threadIdx.x; e < s * M.nchunks; e += 256) {
        const int d = e % s, ch = e / s;
        tr += M.part[(int64_t)ch * n2 + (int64_t)d * s + d];
    }
    for (int o = 16; o > 0; o >>= 1) tr += __shfl_xor_sync(0xffffffffu, tr, o);
    if ((threadIdx.x & 31) == 0) norm_part[threadIdx.x >> 5] = tr;
    __syncthreads();
    tr = 0.0;
    for (int w = 0; w < 8; ++w) tr += norm_part[w];
    const double inv = 1.0 / (sqrt(tr) + (double)M.eps);
    if (rank == 0 && threadIdx.x == 0) M.Q[n2] = (float)inv;
    for (int64_t e = rank * 256 + threadIdx.x; e < n2; e += 256 * kMuonCluster) {
        double g = 0.0;
        for (int ch = 0; ch < M.nchunks; ++ch) g += M.part[(int64_t)ch * n2 + e];
        G[e] = (g * inv) * inv;
    }
    auto sync = [] {
        __threadfence();
        ptx::cluster_sync();
    };
    sync();
    const double a = M.a, b = M.b, c = M.c;
    for (int k = 0; k < M.steps; ++k) {
        const bool last = k + 1 == M.steps;
        // P = a I + b G + c G^2 (the first step's P is Q_1)
        ns_product(G, G, s, rank, sm, [&](int i, int j, double v) {
            const int64_t e = (int64_t)i * s + j;
            const double p = (i == j ? a : 0.0) + b * __ldcg(G + e) + c * v;
            P[e] = p;
            if (k == 0) Q[e] = p;
            if (k == 0 && last) M.Q[e] = (float)p;
        });
        sync();
        if (last && k == 0) break;
        if (k > 0) {
            ns_product(P, Q, s, rank, sm, [&](int i, int j, double v) {
                const int64_t e = (int64_t)i * s + j;
                if (last) M.Q[e] = (float)v;
                else R[e] = v;
            });
            if (last) break;
            sync();
            double* t = Q; Q = R; R = t;
        }
        ns_product(P, G, s, rank, sm, [&](int i, int j, double v) { R[(int64_t)i * s + j] = v; });
        sync();
        ns_product(P, R, s, rank, sm, [&](int i, int j, double v) { G[(int64_t)i * s + j] = v; });
        sync();
    }
}

// O = Q X_0 over 32 columns of the long side, then the update of p, its bf16 copy and m.  A block owns
// its columns: u comes from the old momentum, which it then replaces.
__global__ void __launch_bounds__(256) muon_apply_kernel(const MuonMat* __restrict__ mats, int n) {
    extern __shared__ float fs[];
    const int mi = muon_find(n, blockIdx.x, [&](int k) { return mats[k].apply0; });
    const MuonMat M = mats[mi];
    constexpr int T = kMuonApply, LD = T + 1;
    const int l0 = (blockIdx.x - M.apply0) * T, cols = min(T, M.L - l0);
    float* x = fs;                 // [s][LD] X_0
    float* o = fs + M.s * LD;      // [s][LD] O
    const float inv = M.Q[(int64_t)M.s * M.s];
    for (int e = threadIdx.x; e < M.s * cols; e += 256) {
        const int c = M.tall ? e % M.s : e / cols, l = M.tall ? e / M.s : e % cols;
        const int64_t at = muon_at(M, c, l0 + l);
        const float g = M.g[at], mn = muon_m(M, M.m[at], g);
        M.m[at] = mn;
        x[c * LD + l] = muon_u(M, mn, g) * inv;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int c0 = (threadIdx.x >> 5) * 4; c0 < M.s; c0 += 32) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        const float* q = M.Q + (int64_t)c0 * M.s;
        for (int k = 0; k < M.s; ++k) {
            const float v = lane < cols ? x[k * LD + lane] : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + i < M.s) acc[i] = fmaf(q[(int64_t)i * M.s + k], v, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c0 + i < M.s && lane < cols) o[(c0 + i) * LD + lane] = acc[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < M.s * cols; e += 256) {
        const int c = M.tall ? e % M.s : e / cols, l = M.tall ? e / M.s : e % cols;
        const int64_t at = muon_at(M, c, l0 + l);
        const float p = fmaf(-M.step, o[c * LD + l], M.p[at] * M.decay);
        M.p[at] = p;
        if (M.out) M.out[at] = __float2bfloat16_rn(p);
    }
}

}  // namespace plora
