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
// of the n steps.
//
// Precision.  G squares the condition of u: its small eigenvalues grow by a^2 per step next to a
// rounding relative to its largest, so a Gram matrix in plain 32-bit sums ends 10 to 100 times further
// from the formula than iterating on X (simulated over decaying spectra).  G is therefore formed to about
// 2^-27 and the iteration runs in fp64.  The tensor cores reach that with operands split into three fp16
// parts, v = x0 + x1 + x2: x0 is v rounded to an integer of at most 8 bits in units of the largest
// |v| / 256 (or 128), so that the sums of x0 x0 are integers below 2^24 and exact in their fp32
// accumulator, and x1, x2 are the next 11 bits each.  The seven products of a lower order
// (x0 x1, x1 x0, x1 x1, x0 x2, x2 x0, x1 x2, x2 x1) share a second accumulator, whose roundings are
// relative to its own, 2^-8 smaller, sums.
//
// Tiles.  Both passes work on tiles of 128 rows m x 64 columns l'.  For s > 64 a row is a short-side
// index c; for s <= 64, J = floor(128 / s) long-side blocks are stacked, m = (j, c), so that a tile holds
// the same work for every s: the Gram pass then sums the J diagonal s x s blocks of its 128 x 128
// result, and the apply pass multiplies by the block-diagonal matrix of J copies of Q.
//   l contiguous (!tall):  l = 64 J tile + 64 j + l'        rows of 64 consecutive elements
//   c contiguous (tall):   l = J (64 tile + l') + j         columns of J s consecutive elements
// Either way elements go to shared memory in their order in memory and the matrix descriptors
// (K-major or MN-major) do the transposition.
//
// The first pass reads g and m without writing; the second owns its elements and writes m.
#pragma once
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

namespace plora {

constexpr int kMuonTileL = 64;        // columns l' of a tile
constexpr int kMuonGramTiles = 16;    // tiles of one Gram item
constexpr int kMuonPlane = 128 * kMuonTileL * 2;   // bytes of one fp16 part of a tile (16 KB)
constexpr int kMuonNsTile = 32;       // product tile of the iteration
constexpr int kMuonCluster = 8;       // blocks per matrix in the iteration
constexpr int kMuonBigS = 128;        // above: two 128-row halves per tile in the apply pass

// One matrix of the step.  Element (c, l), c on the short side: c * L + l if !tall, l * s + c if tall.
struct MuonMat {
    const float* g;
    float* m;
    float* p;
    __nv_bfloat16* out;   // the layer's bf16 copy, or nullptr when p is the parameter
    double* part;         // [nchunks][s][s] Gram partials
    double* ns;           // four [sp][sp] matrices of the iteration, sp = s rounded up to 8
    uint8_t* q;           // Q's fp16 parts as the apply pass stages them (muon_q_at)
    float* hdr;           // x scale, output scale, max|u| of each Gram item, max|Q| of each block
    int32_t s, L;
    int32_t tall, nesterov;
    int32_t steps;
    int32_t J;            // long-side blocks stacked in a tile's rows (1 for s > 64)
    int32_t tiles;        // tiles of 64 J long-side indices
    int32_t nchunks, npairs;   // Gram items: chunks of kMuonGramTiles tiles x pairs of 64-row groups
    int32_t gram0;        // first item of this matrix in the Gram launch
    int32_t apply0;       // first tile in its apply launch
    float mu, decay;      // decay = 1 - lr wd
    float step, eps;      // step = lr k
    float a, b, c;
};
static_assert(sizeof(MuonMat) % 8 == 0, "MuonMat layout");

__device__ __forceinline__ float muon_m(const MuonMat& M, float m, float g) { return fmaf(M.mu, m, g); }
__device__ __forceinline__ float muon_u(const MuonMat& M, float m_new, float g) {
    return M.nesterov ? fmaf(M.mu, m_new, g) : m_new;
}

// Copies matrix k's record to shared memory (kept there rather than in 30 registers of each thread); the
// caller synchronises.
__device__ __forceinline__ void muon_fetch(MuonMat* dst, const MuonMat* src) {
    if (threadIdx.x < sizeof(MuonMat) / 8)
        reinterpret_cast<uint64_t*>(dst)[threadIdx.x] = reinterpret_cast<const uint64_t*>(src)[threadIdx.x];
}

// The matrix whose items hold item `b` (begin: the prefix each matrix records).
template <typename F> __device__ __forceinline__ int muon_find(int lo, int hi, int b, F&& begin) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (begin(mid) <= b) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Four consecutive elements of a tile: `e` the first one's index in the matrix, n (0..4) how many exist.
struct MuonQuad {
    int32_t e;            // (a matrix has at most 65536 x 256 elements)
    int n;
};
// Quad (row, x): row m and columns 4x.. of a tile if !tall, column l' = row and rows 4x.. if tall.  lo64,
// hi64: the short-side index of tile rows 0 and 64 (0 and 64, or a pair of 64-row groups).
__device__ __forceinline__ MuonQuad muon_quad(const MuonMat& M, int tile, int row, int x, int lo64, int hi64) {
    MuonQuad q{0, 0};
    if (!M.tall) {
        int c, l = tile * kMuonTileL * M.J + 4 * x;
        if (M.J > 1) {
            const int j = row / M.s;
            if (j >= M.J) return q;
            c = row - j * M.s;
            l += j * kMuonTileL;
        } else {
            c = row + (row < 64 ? lo64 : hi64 - 64);
            if (c >= M.s) return q;
        }
        q.n = min(4, M.L - l);
        q.e = c * M.L + l;
    } else if (M.J > 1) {
        const int w = M.J * M.s, m = 4 * x;
        q.e = (tile * kMuonTileL + row) * w + m;
        q.n = min(min(4, w - m), M.L * M.s - q.e);
    } else {
        const int l = tile * kMuonTileL + row, c = 4 * x + (4 * x < 64 ? lo64 : hi64 - 64);
        if (l >= M.L) return q;
        q.n = min(4, M.s - c);
        q.e = l * M.s + c;
    }
    if (q.n < 0) q.n = 0;
    return q;
}
// Whether every quad of the matrix starts at a multiple of four elements and is whole or empty.
__device__ __forceinline__ bool muon_aligned(const MuonMat& M) {
    return ((M.tall ? M.J * M.s : M.L) & 3) == 0;
}
__device__ __forceinline__ void muon_load4(const float* p, const MuonQuad& q, bool vec, float (&v)[4]) {
    if (vec && q.n == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p + q.e);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = k < q.n ? p[q.e + k] : 0.f;
    }
}

// v = x0 + x1 + x2 (see the top of the file), four at a time, into the three parts of a tile at `at`.
__device__ __forceinline__ void muon_split4(const float (&v)[4], uint32_t at, uint32_t plane) {
    __half h[3][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float x0 = rintf(v[k]), r = v[k] - x0;
        h[0][k] = __float2half_rn(x0);
        h[1][k] = __float2half_rn(r);
        h[2][k] = __float2half_rn(r - __half2float(h[1][k]));
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __half2 a = __halves2half2(h[i][0], h[i][1]), b = __halves2half2(h[i][2], h[i][3]);
        ptx::st_shared_v2(at + i * plane, *reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}
// Byte offset of quad (row, x) in one part of a tile, 128-byte swizzled: rows of 64 elements; in a tall
// matrix's tile, 64-row groups of m (x / 16) of 64 columns each.
__device__ __forceinline__ uint32_t muon_quad_at(bool tall, int row, int x) {
    const uint32_t group = tall ? (uint32_t)(x >> 4) * 8192u : 0u, y = (uint32_t)x & 15u;
    return group + (uint32_t)row * 128u + (((y >> 1) ^ ((uint32_t)row & 7u)) << 4) + (y & 1u) * 8u;
}

// D0 += a0 b0, D1 += the products of a lower order, over one K step; the parts of an operand lie
// `astep` / `bstep` (in descriptor units of 16 bytes) apart.
__device__ __forceinline__ void muon_mma(uint32_t d0, uint32_t d1, uint64_t a, uint64_t b, uint64_t astep, uint64_t bstep,
                                         uint32_t idesc, bool first) {
    ptx::tc_mma_f16(d0, a, b, idesc, first ? 0u : 1u);
    ptx::tc_mma_f16(d1, a, b + bstep, idesc, first ? 0u : 1u);
    ptx::tc_mma_f16(d1, a + astep, b, idesc, 1u);
    ptx::tc_mma_f16(d1, a + astep, b + bstep, idesc, 1u);
    ptx::tc_mma_f16(d1, a, b + 2 * bstep, idesc, 1u);
    ptx::tc_mma_f16(d1, a + 2 * astep, b, idesc, 1u);
    ptx::tc_mma_f16(d1, a + astep, b + 2 * bstep, idesc, 1u);
    ptx::tc_mma_f16(d1, a + 2 * astep, b + bstep, idesc, 1u);
}

// ---------------------------------------------------------------------------------------------- Gram
constexpr int kGramThreads = 256;
constexpr int kGramStage = 3 * kMuonPlane;
constexpr int kGramSmem = 2 * kGramStage + 1024;

// One item: the partial Gram matrix of up to 16 tiles over one pair of 64-row groups (the only pair for
// s <= 128).  The next tile's g and m are requested before this one is split, and its products run while
// the next tile is loaded and split (two stages); two blocks per SM.
// The scale of the split is a power of two above the first tile's largest |u|.  A tile that exceeds it
// takes the sums out of the accumulators and starts them anew at its own scale.
__global__ void __launch_bounds__(kGramThreads, 2)
muon_gram_kernel(const MuonMat* __restrict__ mats, int n, int* err_flag, uint64_t timeout_ns) {
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t done[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ float red[kGramThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ MuonMat record;
    muon_fetch(&record, mats + muon_find(0, n - 1, blockIdx.x, [&](int k) { return mats[k].gram0; }));
    __syncthreads();
    const MuonMat& M = record;
    const int item = blockIdx.x - M.gram0;
    const int chunk = item / M.npairs;
    int ga = 0, gb = 1;
    const int ng = (M.s + 63) / 64;
    for (int k = item - chunk * M.npairs; k > 0; --k)
        if (++gb >= ng) { ++ga; gb = ga + 1; }
    const int t0 = chunk * kMuonGramTiles, t1 = min(M.tiles, t0 + kMuonGramTiles);
    const bool vec = muon_aligned(M);

    if (tid == 0) {
        ptx::mbar_init(&done[0], 1);
        ptx::mbar_init(&done[1], 1);
        abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 0) {
        ptx::tmem_alloc<256>(&tmem_slot);
        ptx::tmem_relinquish();
    }
    // rows past the matrix's stay zero (their products reach no output, but must not be NaN)
    for (int e = tid; e < 2 * kGramStage / 16; e += kGramThreads) reinterpret_cast<uint4*>(smem)[e] = make_uint4(0, 0, 0, 0);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t s0 = ptx::smem_u32(smem);
    const uint32_t idesc = ptx::idesc_f16_f32(128, 128, M.tall != 0, M.tall != 0);
    // this thread's quads: row + i * rstep, x
    const int row = M.tall ? tid >> 5 : tid >> 4, x = M.tall ? tid & 31 : tid & 15, rstep = M.tall ? 8 : 16;

    float g[8][4], m[8][4];
    auto load = [&](int tile) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const MuonQuad q = muon_quad(M, tile, row + i * rstep, x, ga * 64, gb * 64);
            muon_load4(M.g, q, vec, g[i]);
            muon_load4(M.m, q, vec, m[i]);
        }
    };
    uint32_t used = 0;      // uses of each stage so far (bits 0, 1: parity of its next completion)
    int pending = -1;       // stage of the last products issued
    auto wait_stage = [&](int st) {
        ptx::mbar_wait(&done[st], ((used >> st) & 1u) ^ 1u, &abort_flag, timeout_ns, err_flag);
        ptx::tc_fence_after();
    };
    float scale = 0.f, unscale = 0.f;
    bool stored = false;
    float item_max = 0.f;
    bool bad = false;

    // Adds the accumulators, in units of unscale^2, to the item's partial.
    auto drain = [&]() {
        wait_stage(pending);
        double* out = M.part + (int64_t)chunk * M.s * M.s;
        const double us = (double)unscale * (double)unscale;
        const int r = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        double* stack = reinterpret_cast<double*>(smem);   // [128][s], the diagonal blocks' rows
        if (M.J > 1) __syncthreads();                      // every warp has seen the products complete
        for (int c0 = half * 64; c0 < half * 64 + 64; c0 += 16) {
            uint32_t hi[16], lo[16];
            ptx::tmem_ld16(t_row + c0, hi);
            ptx::tmem_ld16(t_row + 128 + c0, lo);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int c = c0 + k;
                const double v = ((double)__uint_as_float(hi[k]) + (double)__uint_as_float(lo[k])) * us;
                if (M.J > 1) {
                    const int j = r / M.s;
                    if (j < M.J && c >= j * M.s && c < (j + 1) * M.s) stack[(int64_t)r * M.s + (c - j * M.s)] = v;
                } else {
                    const int gr = r < 64 ? ga : gb, gc = c < 64 ? ga : gb;
                    const int rr = gr * 64 + (r & 63), cc = gc * 64 + (c & 63);
                    // a diagonal block is in several pairs: the pair with the next group writes it (the last
                    // group's, the pair with the one before)
                    const bool own = gr != gc || (gr == ga ? gb == ga + 1 : ga == ng - 2) || ng == 1;
                    if (own && rr < M.s && cc < M.s) {
                        double* o = out + (int64_t)rr * M.s + cc;
                        *o = stored ? *o + v : v;
                    }
                }
            }
        }
        if (M.J > 1) {
            __syncthreads();
            for (int e = tid; e < M.s * M.s; e += kGramThreads) {
                double v = 0.0;
                for (int j = 0; j < M.J; ++j) v += stack[(int64_t)j * M.s * M.s + e];
                out[e] = stored ? out[e] + v : v;
            }
            __syncthreads();
            // the stages held sums: clear their rows again
            for (int e = tid; e < 2 * kGramStage / 16; e += kGramThreads)
                reinterpret_cast<uint4*>(smem)[e] = make_uint4(0, 0, 0, 0);
            __syncthreads();
        }
        ptx::tc_fence_before();
        stored = true;
        pending = -1;
    };

    load(t0);
    for (int t = t0; t < t1; ++t) {
        float u[8][4];
        float big = 0.f;
        bool over = false;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                u[i][k] = muon_u(M, muon_m(M, m[i][k], g[i][k]), g[i][k]);
                const float a = fabsf(u[i][k]);
                over = over || !(a * scale <= 128.f);      // also a NaN
                big = fmaxf(big, a);
            }
        if (t + 1 < t1) load(t + 1);
        item_max = fmaxf(item_max, big);
        // the first tile has no scale yet; a first tile of zeros leaves it to the next
        if (__syncthreads_or(over || scale == 0.f)) {
            if (pending >= 0) drain();
            float w = big;
            bool nan = over && !(big * 0.f == 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) nan = nan || !(u[i][k] * 0.f == 0.f);
            for (int o = 16; o > 0; o >>= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
            if (lane == 0) red[warp] = w;
            bad = __syncthreads_or(nan) || bad;
            w = 0.f;
            for (int k = 0; k < kGramThreads / 32; ++k) w = fmaxf(w, red[k]);
            if (!bad && w > 0.f) {
                const int e = max(ilogbf(w) + 1, -100);    // w < 2^e
                scale = scalbnf(1.f, 7 - e);
                unscale = scalbnf(1.f, e - 7);
            }
            __syncthreads();
        }
        if (bad) break;                     // a NaN or an infinity: the whole matrix becomes NaN
        if (scale == 0.f) continue;         // nothing but zeros so far
        const int st = t & 1;
        const uint32_t base = s0 + st * kGramStage;
        if ((used >> (2 + st)) & 1u) wait_stage(st);       // the products that last read this stage
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = u[i][k] * scale;
            muon_split4(v, base + muon_quad_at(M.tall, row + i * rstep, x), kMuonPlane);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncthreads();
        ptx::tc_fence_after();
        if (tid == 0) {
            const uint64_t d = M.tall ? ptx::smem_desc_sw128(base, 8192, 1024) : ptx::smem_desc_sw128(base, 16, 1024);
            const uint64_t kstep = M.tall ? 2048 / 16 : 32 / 16;
            for (int ks = 0; ks < kMuonTileL / 16; ++ks)
                muon_mma(tmem, tmem + 128, d + ks * kstep, d + ks * kstep, kMuonPlane / 16, kMuonPlane / 16, idesc,
                         pending < 0 && ks == 0);
            ptx::tc_commit(&done[st]);
        }
        used ^= 1u << st;
        used |= 4u << st;
        pending = st;
    }
    if (pending >= 0) drain();
    // nothing but zeros, or a NaN or an infinity somewhere in the item
    if (!stored || bad) {
        __syncthreads();
        double* out = M.part + (int64_t)chunk * M.s * M.s;
        const double v = bad ? __longlong_as_double(0x7ff8000000000000ll) : 0.0;
        for (int e = tid; e < M.s * M.s; e += kGramThreads) {
            const int r = e / M.s, c = e - r * M.s, gr = r >> 6, gc = c >> 6;
            if (M.npairs == 1 || ((gr == ga || gr == gb) && (gc == ga || gc == gb) &&
                                  (gr != gc || (gr == ga ? gb == ga + 1 : ga == ng - 2))))
                out[e] = v;
        }
    }
    for (int o = 16; o > 0; o >>= 1) item_max = fmaxf(item_max, __shfl_xor_sync(0xffffffffu, item_max, o));
    if (lane == 0) red[warp] = item_max;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (tid == 0) {
        float w = 0.f;
        for (int k = 0; k < kGramThreads / 32; ++k) w = fmaxf(w, red[k]);
        M.hdr[2 + item] = w;
    }
    if (warp == 0) ptx::tmem_dealloc<256>(tmem);
}

// ----------------------------------------------------------------------------------------- iteration
constexpr int kNsK = 64;                               // K extent of one stage
constexpr int kNsPitch = kNsK + 4;                     // doubles; rows shift by 4 so that fragment loads spread
constexpr int kNsStages = 3;
constexpr int kNsStageD = 2 * kMuonNsTile * kNsPitch;  // doubles of one stage: the A rows, then the B rows
constexpr int kMuonNsSmem = (kNsStages * kNsStageD + 4 * 32 * 8) * 8;

__device__ __forceinline__ void dmma_16x8x8(double (&d)[4], const double (&a)[4], const double (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f64.f64.f64.f64 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+d"(d[0]), "+d"(d[1]), "+d"(d[2]), "+d"(d[3])
        : "d"(a[0]), "d"(a[1]), "d"(a[2]), "d"(a[3]), "d"(b[0]), "d"(b[1]));
}

// C = A B for symmetric sp x sp matrices that commute (so C is symmetric and B's rows serve as its
// columns): the 32 x 32 tiles of C's lower half, dealt over the cluster's blocks, each with its K in
// stages of 64 that run ahead across tiles.  out(r, c, v) takes each element with c <= r.  Eight warps: 2 x 2
// blocks of 16 x 16, two halves of each stage's K, joined in a fixed order.
template <typename F>
__device__ __forceinline__ void ns_product(const double* A, const double* B, int sp, int rank, double* sm, F&& out) {
    constexpr int T = kMuonNsTile;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wr = (warp & 1) * 16, wc = ((warp >> 1) & 1) * 16, kh = warp >> 2;
    const int nt = (sp + T - 1) / T, tiles = nt * (nt + 1) / 2, nk = (sp + kNsK - 1) / kNsK;
    const int mine = tiles > rank ? (tiles - rank + kMuonCluster - 1) / kMuonCluster : 0;
    const int steps = mine * nk;
    auto tile_of = [&](int k, int& ti, int& tj) {
        int t = rank + (k / nk) * kMuonCluster;
        ti = 0;
        while (t > ti) { t -= ti + 1; ++ti; }
        tj = t;
    };
    auto fetch = [&](int k) {
        if (k < steps) {
            int ti, tj;
            tile_of(k, ti, tj);
            const int k0 = (k % nk) * kNsK;
            double* st = sm + (k % kNsStages) * kNsStageD;
#pragma unroll
            for (int e0 = 0; e0 < 2 * T * kNsK / 2; e0 += 256) {
                const int e = e0 + tid, half = e >> 10, r = (e >> 5) & 31, c = (e & 31) * 2;
                const int gr = (half ? tj : ti) * T + r, gc = k0 + c;
                const bool ok = gr < sp && gc < sp;
                const double* src = (half ? B : A) + (ok ? (int64_t)gr * sp + gc : 0);
                ptx::cp_async16(st + (half * T + r) * kNsPitch + c, src, ok ? 16 : 0);
            }
        }
        ptx::cp_async_commit();
    };
    double acc[2][4] = {};
    for (int k = 0; k < kNsStages - 1; ++k) fetch(k);
    for (int k = 0; k < steps; ++k) {
        ptx::cp_async_wait<kNsStages - 2>();
        __syncthreads();
        fetch(k + kNsStages - 1);
        const double* as = sm + (k % kNsStages) * kNsStageD + (wr + (lane >> 2)) * kNsPitch + (lane & 3) + kh * (kNsK / 2);
        const double* bs = sm + (k % kNsStages) * kNsStageD + (T + wc + (lane >> 2)) * kNsPitch + (lane & 3) + kh * (kNsK / 2);
#pragma unroll
        for (int kk = 0; kk < kNsK / 2; kk += 8) {
            const double a[4] = {as[kk], as[kk + 8 * kNsPitch], as[kk + 4], as[kk + 8 * kNsPitch + 4]};
            const double b0[2] = {bs[kk], bs[kk + 4]};
            const double b1[2] = {bs[kk + 8 * kNsPitch], bs[kk + 8 * kNsPitch + 4]};
            dmma_16x8x8(acc[0], a, b0);
            dmma_16x8x8(acc[1], a, b1);
        }
        if (k % nk == nk - 1) {   // the tile is complete
            int ti, tj;
            tile_of(k, ti, tj);
            double* red = sm + kNsStages * kNsStageD + ((warp & 3) * 32 + lane) * 8;
            if (kh) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) red[4 * j + i] = acc[j][i];
            }
            __syncthreads();
            if (!kh) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = ti * T + wr + (lane >> 2) + (i >> 1) * 8, c = tj * T + wc + j * 8 + (lane & 3) * 2 + (i & 1);
                        // (a diagonal tile's upper half would mirror onto its lower one)
                        if (r < sp && c <= r) out(r, c, acc[j][i] + red[4 * j + i]);
                    }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.0;
        }
    }
    ptx::cp_async_wait<0>();
    __syncthreads();
}

// Byte offset of the eight-element chunk (row, 8 k8 ..) of part `part` of Q as the apply pass stages it:
// blocks of 128 rows x 64 columns, 128-byte swizzled, ordered (row half, column block, part).
__host__ __device__ __forceinline__ int64_t muon_q_at(int kblocks, int row, int k8, int part) {
    const int64_t block = ((int64_t)(row >> 7) * kblocks + (k8 >> 3)) * 3 + part;
    const int r = row & 127;
    return block * kMuonPlane + r * 128 + (((k8 & 7) ^ (r & 7)) << 4);
}

// The iteration on one matrix's Gram matrix in fp64 on the fp64 tensor cores: a cluster of eight blocks
// per matrix, the matrices in L2, one cluster barrier after each product.  Then Q's three fp16 parts for
// the apply pass (block-diagonal over the stacked blocks) and the scales.
__global__ void __cluster_dims__(kMuonCluster, 1, 1) __launch_bounds__(256)
muon_ns_kernel(const MuonMat* __restrict__ mats) {
    extern __shared__ __align__(16) double sm[];
    __shared__ double redd[8];
    __shared__ float redf[8];
    const MuonMat M = mats[blockIdx.x / kMuonCluster];
    const int rank = (int)ptx::cluster_ctarank();
    const int tid = threadIdx.x, s = M.s, sp = (s + 7) & ~7;
    const int64_t s2 = (int64_t)s * s, n2 = (int64_t)sp * sp;
    double* G = M.ns;
    double* P = G + n2;
    double* R = P + n2;
    double* Q = R + n2;
    // |u|_F^2, the trace of G, and max |u|: by every block in the same order
    double tr = 0.0;
    for (int e = tid; e < s * M.nchunks; e += 256) {
        const int d = e % s, ch = e / s;
        tr += M.part[ch * s2 + (int64_t)d * (s + 1)];
    }
    float big = 0.f;
    for (int e = tid; e < M.nchunks * M.npairs; e += 256) big = fmaxf(big, M.hdr[2 + e]);
    for (int o = 16; o > 0; o >>= 1) {
        tr += __shfl_xor_sync(0xffffffffu, tr, o);
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    }
    if ((tid & 31) == 0) { redd[tid >> 5] = tr; redf[tid >> 5] = big; }
    __syncthreads();
    tr = 0.0;
    big = 0.f;
    for (int w = 0; w < 8; ++w) { tr += redd[w]; big = fmaxf(big, redf[w]); }
    const double inv = 1.0 / (sqrt(tr) + (double)M.eps);
    for (int64_t e = rank * 256 + tid; e < n2; e += 256 * kMuonCluster) {
        const int r = (int)(e / sp), c = (int)(e - (int64_t)r * sp);
        double g = 0.0;
        if (r < s && c < s)
            for (int ch = 0; ch < M.nchunks; ++ch) g += M.part[ch * s2 + (int64_t)r * s + c];
        G[e] = (g * inv) * inv;
    }
    auto sync = [] {
        __threadfence();
        ptx::cluster_sync();
    };
    sync();
    const double a = M.a, b = M.b, c = M.c;
    auto both = [&](double* C, int i, int j, double v) {
        C[(int64_t)i * sp + j] = v;
        C[(int64_t)j * sp + i] = v;
    };
    for (int k = 0; k < M.steps; ++k) {
        const bool last = k + 1 == M.steps;
        // P = a I + b G + c G^2 (the first step's P is Q_1)
        ns_product(G, G, sp, rank, sm, [&](int i, int j, double v) {
            const double p = (i == j && i < s ? a : 0.0) + b * __ldcg(G + (int64_t)i * sp + j) + c * v;
            both(P, i, j, p);
            if (k == 0) both(Q, i, j, p);
        });
        sync();
        if (k > 0) {
            ns_product(P, Q, sp, rank, sm, [&](int i, int j, double v) { both(R, i, j, v); });
            sync();
            double* t = Q; Q = R; R = t;
        }
        if (last) break;
        ns_product(P, G, sp, rank, sm, [&](int i, int j, double v) { both(R, i, j, v); });
        sync();
        ns_product(P, R, sp, rank, sm, [&](int i, int j, double v) { both(G, i, j, v); });
        sync();
    }
    // max |Q|: each block's share, then the eight of them
    float* const qpart = M.hdr + 2 + M.nchunks * M.npairs;
    float qmax = 0.f;
    for (int64_t e = rank * 256 + tid; e < n2; e += 256 * kMuonCluster) qmax = fmaxf(qmax, (float)fabs(__ldcg(Q + e)));
    for (int o = 16; o > 0; o >>= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, o));
    __syncthreads();
    if ((tid & 31) == 0) redf[tid >> 5] = qmax;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < 8; ++w) qmax = fmaxf(qmax, redf[w]);
        qpart[rank] = qmax;
    }
    sync();
    qmax = 0.f;
    for (int k = 0; k < kMuonCluster; ++k) qmax = fmaxf(qmax, __ldcg(qpart + k));
    const int eq = qmax > 0.f && qmax < 3e38f ? ilogbf(qmax) + 1 : 0, eu = max(big > 0.f ? ilogbf(big) + 1 : -100, -100);
    const double qs = scalbn(1.0, 8 - eq);
    if (rank == 0 && tid == 0) {
        M.hdr[0] = scalbnf(1.f, 8 - eu);                                      // x = u hdr[0], |x| < 256
        // a NaN or an infinity in u makes the whole of O a NaN
        const bool fine = tr * 0.0 == 0.0 && qmax < 3e38f && qmax == qmax;
        M.hdr[1] = fine ? (float)(inv * scalbn(1.0, eu - 8 + eq - 8)) : __int_as_float(0x7fc00000);
    }
    const int w = s > kMuonBigS ? 256 : 128, kblocks = w / 64;
    for (int e = rank * 256 + tid; e < w * (w / 8); e += 256 * kMuonCluster) {
        const int r = e / (w / 8), k8 = e - r * (w / 8);
        const int jr = r / s, cr = r - jr * s;
        __align__(16) __half h[3][8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int kk = k8 * 8 + k, jk = kk / s, ck = kk - jk * s;
            const double v = jr < M.J && jr == jk ? __ldcg(Q + (int64_t)cr * sp + ck) * qs : 0.0;
            const double x0 = rint(v);
            h[0][k] = __double2half(x0);
            h[1][k] = __double2half(v - x0);
            h[2][k] = __double2half((v - x0) - (double)__half2float(h[1][k]));
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
            *reinterpret_cast<uint4*>(M.q + muon_q_at(kblocks, r, k8, i)) = *reinterpret_cast<const uint4*>(h[i]);
    }
}

// --------------------------------------------------------------------------------------------- apply
constexpr int kApplyThreads = 512;
constexpr int kApplyQ = 6 * kMuonPlane;               // Q of s <= 128, or two (half, column block) stages
constexpr int kApplyV = 6 * kMuonPlane;               // two tiles of 128 rows, or one of 256
constexpr int kApplyWarpStage = 32 * 16 * 4;          // a warp's 32 x 16 block of O
constexpr int kApplySmem = kApplyQ + kApplyV + (kApplyThreads / 32) * kApplyWarpStage + 1024;
static_assert(kApplySmem + 128 <= 232448, "shared memory per CTA");

// O = Q X_0 tile by tile, then p, its bf16 copy and m.  One block per SM over a contiguous run of tiles
// (all matrices' tiles in one list, so the blocks finish together); Q stays in shared memory while the
// matrix does.  Per tile: u is formed from the loaded g and m, the new m stored, u split into its parts;
// the products of this tile run while the previous tile's O is turned into its update and the next
// tile's g and m arrive.
// BIG (s > 128): tiles of 256 rows, Q's (half, column block) pieces streamed from L2 through two stages.
template <bool BIG>
__global__ void __launch_bounds__(kApplyThreads, 1)
muon_apply_kernel(const MuonMat* __restrict__ mats, int first, int last, int tiles, int* err_flag, uint64_t timeout_ns) {
    constexpr int NQ = BIG ? 8 : 4;                    // quads per thread
    constexpr int PLANE = BIG ? 2 * kMuonPlane : kMuonPlane;
    constexpr int HALVES = BIG ? 2 : 1;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = smem;
    uint8_t* sv = smem + kApplyQ;
    __shared__ __align__(8) uint64_t done[2], qfull[2], qfree[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ MuonMat record[4];   // matrix k's record in slot k & 3: at most three are in use at once
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float* stage = reinterpret_cast<float*>(smem + kApplyQ + kApplyV + warp * kApplyWarpStage);
    const int u0 = (int)((int64_t)tiles * blockIdx.x / gridDim.x), u1 = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
    if (tid == 0) {
        for (int k = 0; k < 2; ++k) {
            ptx::mbar_init(&done[k], 1);
            ptx::mbar_init(&qfull[k], 1);
            ptx::mbar_init(&qfree[k], 1);
        }
        abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 0) {
        ptx::tmem_alloc<512>(&tmem_slot);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t sq0 = ptx::smem_u32(sq), sv0 = ptx::smem_u32(sv);
    auto wait = [&](uint64_t* bar, uint32_t parity) { ptx::mbar_wait(bar, parity, &abort_flag, timeout_ns, err_flag); };

    // state of the tile being loaded, of the one being multiplied and of the one being finished
    int mi = muon_find(first, last - 1, u0, [&](int k) { return mats[k].apply0; });
    int row, x, rstep;
    bool vec;
    auto enter = [&]() {      // makes matrix mi the one whose tiles are loaded
        muon_fetch(&record[mi & 3], mats + mi);
        __syncthreads();
        const MuonMat& M = record[mi & 3];
        const int per = BIG ? 64 : 32;                 // quads of a tall tile's column
        row = M.tall ? tid / per : tid >> 4;
        x = M.tall ? tid % per : tid & 15;
        rstep = M.tall ? kApplyThreads / per : kApplyThreads / 16;
        vec = muon_aligned(M);
    };
    // rows 128 and up of a 256-row tile are short-side indices too
    auto quad = [&](const MuonMat& Z, int tile, int i) {
        if (!BIG) return muon_quad(Z, tile, row + i * rstep, x, 0, 64);
        MuonQuad q{0, 0};
        if (!Z.tall) {
            const int c = row + i * rstep, l = tile * kMuonTileL + 4 * x;
            if (c < Z.s) { q.n = max(0, min(4, Z.L - l)); q.e = c * Z.L + l; }
        } else {
            const int l = tile * kMuonTileL + row + i * rstep, c = 4 * x;
            if (l < Z.L) { q.n = max(0, min(4, Z.s - c)); q.e = l * Z.s + c; }
        }
        return q;
    };
    float g[NQ][4], m[NQ][4];
    auto load = [&](int u) {
        const MuonMat& M = record[mi & 3];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const MuonQuad q = quad(M, u - M.apply0, i);
            muon_load4(M.g, q, vec, g[i]);
            muon_load4(M.m, q, vec, m[i]);
        }
    };
    int fin_mi = 0, fin_tile = 0;   // the finished tile
    bool have = false;
    uint32_t n_done = 0;        // tiles multiplied so far (buffer and parity of `done`)
    uint32_t n_q = 0;           // Q pieces (BIG) or whole Qs loaded so far
    const int quarter = warp & 3, cg = warp >> 2;       // this warp's accumulator rows and 16 columns

    // the update of the finished tile from accumulator buffer `buf`
    auto finish = [&](uint32_t buf) {
        const MuonMat& fin = record[fin_mi & 3];
        const float osc = fin.hdr[1];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            const int m0 = h * 128 + quarter * 32;      // first tile row of this warp
            float p[16];
            int at[16];
            if (!fin.tall) {
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int mr = m0 + 2 * k + (lane >> 4);
                    const int j = fin.J > 1 ? mr / fin.s : 0, c = mr - j * fin.s;
                    const int l = (fin_tile * fin.J + j) * kMuonTileL + cg * 16 + (lane & 15);
                    at[k] = (j < fin.J && c < fin.s && l < fin.L) ? c * fin.L + l : -1;
                }
            } else {
                const int w = fin.J * fin.s, mr = m0 + lane;
                const int total = fin.L * fin.s;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int e = (fin_tile * kMuonTileL + cg * 16 + k) * w + mr;
                    at[k] = mr < w && e < total ? e : -1;
                }
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) p[k] = at[k] >= 0 ? fin.p[at[k]] : 0.f;
            if (h == 0) {
                wait(&done[buf & 1], (buf >> 1) & 1u);
                ptx::tc_fence_after();
            }
            const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16) + (buf & 1) * 256 + h * 128 + cg * 16;
            uint32_t hi[16], lo[16];
            __syncwarp();
            ptx::tmem_ld16(t_row, hi);
            ptx::tmem_ld16(t_row + 64, lo);
            ptx::tmem_ld_wait();
            float o[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = (__uint_as_float(hi[k]) + __uint_as_float(lo[k])) * osc;
            if (!fin.tall) {
                // rows of 16 consecutive elements: through shared memory, two rows per instruction
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 16; ++k) stage[lane * 16 + (k ^ ((lane >> 1) & 15))] = o[k];
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int r = 2 * k + (lane >> 4);
                    o[k] = stage[r * 16 + ((lane & 15) ^ ((r >> 1) & 15))];
                }
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (at[k] < 0) continue;
                const float v = fmaf(-fin.step, o[k], p[k] * fin.decay);
                fin.p[at[k]] = v;
                if (fin.out) fin.out[at[k]] = __float2bfloat16_rn(v);
            }
        }
        ptx::tc_fence_before();
    };

    enter();
    load(u0);
    int mq = -1;                 // the matrix whose Q is in shared memory (or streamed)
    for (int u = u0; u < u1; ++u) {
        const int ci = mi;
        const MuonMat& C = record[ci & 3];     // this tile's matrix
        const int tile = u - C.apply0;
        float xv[NQ][4];
        const float xs = C.hdr[0];
        const bool fresh = mq != mi;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const MuonQuad q = quad(C, tile, i);
            float mn[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                mn[k] = muon_m(C, m[i][k], g[i][k]);
                xv[i][k] = muon_u(C, mn[k], g[i][k]) * xs;
            }
            if (vec && q.n == 4) {
                *reinterpret_cast<float4*>(C.m + q.e) = make_float4(mn[0], mn[1], mn[2], mn[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < q.n) C.m[q.e + k] = mn[k];
            }
        }
        const int crow = row, cx = x, crstep = rstep;
        // BIG: one tile buffer; otherwise the products that read this one ended before the previous finish
        if (fresh || BIG) {
            if (have) wait(&done[(n_done - 1) & 1], ((n_done - 1) >> 1) & 1u);
            ptx::tc_fence_after();
            __syncthreads();
        }
        if (fresh) {
            if (!BIG && tid == 0) {
                ptx::mbar_arrive_expect_tx(&qfull[0], kApplyQ);
                ptx::bulk_load(sq, C.q, kApplyQ, &qfull[0]);
            }
            // rows past the matrix's are zero: their products reach no output, but must not be NaN
            for (int e = tid; e < kApplyV / 16; e += kApplyThreads) reinterpret_cast<uint4*>(sv)[e] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            mq = mi;
        }
        const uint32_t vbase = sv0 + (BIG ? 0u : (n_done & 1u) * (uint32_t)(3 * kMuonPlane));
#pragma unroll
        for (int i = 0; i < NQ; ++i)
            muon_split4(xv[i], vbase + muon_quad_at(C.tall, crow + i * crstep, cx), PLANE);
        // the next tile's g and m
        if (u + 1 < u1) {
            if (u + 1 >= C.apply0 + C.tiles) {
                ++mi;
                enter();
            }
            load(u + 1);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncthreads();
        ptx::tc_fence_after();
        const uint32_t buf = n_done;
        if (tid == 0) {
            const uint32_t d0 = tmem + (buf & 1) * 256;
            const uint32_t idesc = ptx::idesc_f16_f32(128, 64, false, !C.tall);
            const int ksteps = (min(C.J * C.s, HALVES * 128) + 15) / 16;
            // K step ks of the tile: its rows 16 ks ..
            auto vdesc = [&](int ks) {
                return C.tall ? ptx::smem_desc_sw128(vbase + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024)
                              : ptx::smem_desc_sw128(vbase + ks * 2048, 8192, 1024);
            };
            if constexpr (!BIG) {
                if (fresh) {
                    wait(&qfull[0], n_q & 1u);
                }
                for (int ks = 0; ks < ksteps; ++ks)
                    muon_mma(d0, d0 + 64, ptx::smem_desc_sw128(sq0 + (ks >> 2) * 3 * kMuonPlane + (ks & 3) * 32, 16, 1024),
                             vdesc(ks), kMuonPlane / 16, PLANE / 16, idesc, ks == 0);
            } else {
                const int kb = (ksteps + 3) / 4, pieces = 2 * kb;
                auto fetch = [&](int k) {   // piece k: row half k / kb, column block k % kb
                    const uint32_t nq = n_q + k;
                    if (nq >= 2) wait(&qfree[nq & 1], ((nq >> 1) & 1u) ^ 1u);
                    ptx::mbar_arrive_expect_tx(&qfull[nq & 1], 3 * kMuonPlane);
                    ptx::bulk_load(sq + (nq & 1) * 3 * kMuonPlane, C.q + ((int64_t)(k / kb) * 4 + k % kb) * 3 * kMuonPlane,
                                   3 * kMuonPlane, &qfull[nq & 1]);
                };
                fetch(0);
                for (int k = 0; k < pieces; ++k) {
                    if (k + 1 < pieces) fetch(k + 1);
                    const uint32_t nq = n_q + k;
                    wait(&qfull[nq & 1], (nq >> 1) & 1u);
                    const int h = k / kb, b = k % kb;
                    for (int ks = 0; ks < 4 && b * 4 + ks < ksteps; ++ks)
                        muon_mma(d0 + h * 128, d0 + h * 128 + 64,
                                 ptx::smem_desc_sw128(sq0 + (nq & 1) * 3 * kMuonPlane + ks * 32, 16, 1024), vdesc(b * 4 + ks),
                                 kMuonPlane / 16, PLANE / 16, idesc, b == 0 && ks == 0);
                    ptx::tc_commit(&qfree[nq & 1]);
                }
                n_q += pieces;
            }
            ptx::tc_commit(&done[buf & 1]);
        }
        if (!BIG && fresh) ++n_q;
        __syncwarp();
        ++n_done;
        if (have) finish(buf - 1);
        fin_mi = ci;
        fin_tile = tile;
        have = true;
    }
    if (have) finish(n_done - 1);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 0) ptx::tmem_dealloc<512>(tmem);
}

}  // namespace plora
