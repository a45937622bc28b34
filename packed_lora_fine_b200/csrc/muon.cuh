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
// from the formula than iterating on X (simulated over decaying spectra).  G is therefore formed beyond 32 bits
// and the iteration runs in fp64.  The tensor cores reach that with operands split into three fp16
// parts, v = x0 + x1 + x2: x0 is v rounded to an integer of at most 8 bits in units of the largest
// |v| / 256 (or 128), so that the sums of x0 x0 are integers below 2^24 and exact in their fp32
// accumulator, and x1, x2 are the next 11 bits each, floating: an element far below the largest keeps 22 bits.
// An accumulator rounds, by up to 2^-23 per step, next to its own sum, so the Gram pass has one for each order of
// products: x0 x0 | x0 x1, x1 x0 | x1 x1, x0 x2, x2 x0 | x1 x2, x2 x1.  Where a few columns of u dominate (an
// outlier feature), the rest of u has no x0, its products stand alone in the third, and what the outliers put
// into the first two is exact; one accumulator for all the lower orders lost the rest in the outliers' roundings (a
// column 1000 times the others, 128 x 4096: O off by 5e-5, now 1e-6; 32-bit iteration 5e-7).  For the lower parts to
// keep their bits in fp16 they are scaled by 2^6 and 2^12 there.  Q X_0 takes all products but x2 x2 in two
// accumulators, x0 x0 and the rest.
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
#include <type_traits>
#include "ptx.cuh"

namespace plora {

constexpr int kMuonTileL = 64;        // columns l' of a tile
constexpr int kMuonPlane = 128 * kMuonTileL * 2;   // bytes of one fp16 part of a tile (16 KB)
constexpr int kMuonBigS = 128;        // above: two 128-row halves per tile in the apply pass

// One matrix of the step.  Element (c, l), c on the short side: c * L + l if !tall, l * s + c if tall.
struct MuonMat {
    const float* g;
    float* m;
    float* p;
    __nv_bfloat16* out;   // the layer's bf16 copy, or nullptr when p is the parameter
    double* part;         // [nchunks][s][s] Gram partials
    double* ns;           // G, P and Q, [sp][sp], sp = s rounded up to 8 (s > 128)
    uint8_t* q;           // Q's fp16 parts as the apply pass stages them (muon_q_at)
    float* hdr;           // x scale, output scale, max|u| of each Gram item
    int32_t s, L;
    int32_t tall, nesterov;
    int32_t steps;
    int32_t J;            // long-side blocks stacked in a tile's rows (1 for s > 64)
    int32_t tiles;        // tiles of 64 J long-side indices
    int32_t nchunks, npairs;   // Gram items: chunks of per_chunk tiles x pairs of 64-row groups
    int32_t per_chunk, pad_;
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

// Byte offset of element (row, y) in one part of a tile, 128-byte swizzled: rows of 64 elements (y < 64);
// in a tall matrix's tile the row is the column l' and y the row m, in 64-row groups of 64 columns each.
__device__ __forceinline__ uint32_t muon_elem_at(int row, int y) {
    return (uint32_t)(y >> 6) * 8192u + (uint32_t)row * 128u + ((((uint32_t)y >> 3 & 7u) ^ ((uint32_t)row & 7u)) << 4) +
           (uint32_t)(y & 7) * 2u;
}

// scale * v = x0 + x1 / UP + x2 / UP^2 (see the top of the file), two values at a time.  |scale v| <= 256, so adding
// 1.5 2^23 rounds to an integer; scale and UP are powers of two, so the products are exact.
template <int UP>
__device__ __forceinline__ void muon_split2(uint64_t v, uint64_t scale, uint32_t (&h)[3]) {
    constexpr float kRound = 12582912.f, kUp = (float)UP;
    const uint64_t round = ptx::f32x2(kRound, kRound), neg = ptx::f32x2(-1.f, -1.f);
    const uint64_t t = ptx::f32x2_fma(v, scale, round);             // x0 + 1.5 2^23
    const uint64_t n0 = ptx::f32x2_fma(t, ptx::f32x2(-kUp, -kUp), ptx::f32x2(kUp * kRound, kUp * kRound));      // -UP x0
    const uint64_t r = ptx::f32x2_fma(v, UP == 1 ? scale : ptx::f32x2_mul(scale, ptx::f32x2(kUp, kUp)), n0);
    const float2 x0 = ptx::f32x2_get(ptx::f32x2_add(t, ptx::f32x2(-kRound, -kRound))), rr = ptx::f32x2_get(r);
    const __half2 h0 = __floats2half2_rn(x0.x, x0.y), h1 = __floats2half2_rn(rr.x, rr.y);
    const float2 f1 = __half22float2(h1);
    const uint64_t left = ptx::f32x2_fma(ptx::f32x2(f1.x, f1.y), neg, r);
    const float2 x2 = ptx::f32x2_get(UP == 1 ? left : ptx::f32x2_mul(left, ptx::f32x2(kUp, kUp)));
    const __half2 h2 = __floats2half2_rn(x2.x, x2.y);
    h[0] = *reinterpret_cast<const uint32_t*>(&h0);
    h[1] = *reinterpret_cast<const uint32_t*>(&h1);
    h[2] = *reinterpret_cast<const uint32_t*>(&h2);
}

// How T threads hold a step of TL columns of a tile of ROWS rows, 4 NQ elements each, in the order of memory:
//   kRows    not tall, L % 4 == 0: quads of 4 columns of a row
//   kFlat    tall, w = J s a multiple of 4: quads of the step's TL w consecutive elements
//   kPairs   tall, other w: pairs of consecutive rows m of a column l'
//   kQuads   what is left (a tall pair of 64-row groups of s > 128, an odd L): quads, each checked
// col0: the step's first column in its tile.
template <int T, int TL, int ROWS>
struct MuonTile {
    enum { kRows, kFlat, kPairs, kQuads };
    static constexpr int NQ = ROWS * TL / 4 / T;
    static constexpr int kPairCols = T / (ROWS / 2);   // columns l' that the threads' pairs cover at once
    static constexpr int kRowStep = T / (TL / 4);      // rows that the threads' quads cover at once (not tall)
    static constexpr int kColStep = T / (ROWS / 4);    // columns that the threads' quads cover at once (tall)
    static_assert(kRowStep % 8 == 0, "the swizzle repeats every eight rows");
    int mode, row, x, lo64, hi64;
    int meta[NQ];      // kRows: the quad's first element in tile 0; kFlat: its place in the tile; -1: none

    // whole: the tile's rows are the whole short side (J stacked blocks of it); otherwise rows 0 and 64 are the
    // short-side indices lo and hi.
    __device__ __forceinline__ void enter(const MuonMat& M, int tid, bool whole, int lo, int hi) {
        const int w = M.J * M.s;
        lo64 = lo;
        hi64 = hi;
        mode = M.tall ? (!whole ? kQuads : (w & 3) ? kPairs : kFlat) : (M.L & 3) ? kQuads : kRows;
        const int per = mode == kPairs ? ROWS / 2 : M.tall ? ROWS / 4 : TL / 4;
        row = mode == kFlat ? tid : tid / per;
        x = mode == kFlat ? 0 : (tid - row * per) * (mode == kPairs ? 2 : 4);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            meta[i] = -1;
            if (mode == kFlat) {
                const int f = 4 * (tid + i * T), l = f / w, m = f - l * w;
                if (l < TL) meta[i] = (int)muon_elem_at(l, m);
            } else if (mode == kRows) {
                const int r = row + i * kRowStep;
                int j = 0, c = r;
                if (M.J > 1) { j = r / M.s; c = r - j * M.s; }
                else if (ROWS == 128) c = r + (r < 64 ? lo64 : hi64 - 64);
                if (j < M.J && c < M.s) meta[i] = c * M.L + j * kMuonTileL + x;
            }
        }
    }
    // Quad i where each is checked: its first element, and how many exist.
    __device__ __forceinline__ int quad(const MuonMat& M, int tile, int col0, int i, int& n) const {
        if (!M.tall) {
            const int r = row + i * kRowStep;
            int j = 0, c = r;
            if (M.J > 1) { j = r / M.s; c = r - j * M.s; }
            else if (ROWS == 128) c = r + (r < 64 ? lo64 : hi64 - 64);
            const int l = (tile * M.J + j) * kMuonTileL + col0 + x;
            n = j < M.J && c < M.s ? max(0, min(4, M.L - l)) : 0;
            return c * M.L + l;
        }
        const int l = tile * kMuonTileL + col0 + row + i * kColStep;      // (a tall pair of groups: J = 1)
        const int c = x + (x < 64 ? lo64 : hi64 - 64);
        n = l < M.L ? max(0, min(4, M.s - c)) : 0;
        return l * M.s + c;
    }
    static __device__ __forceinline__ void set4(float (&v)[4], float4 f) { v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w; }
    static __device__ __forceinline__ float4 get4(const float* p, int e, bool ok) {
        return ok ? *reinterpret_cast<const float4*>(p + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }

    // g and m of a step (zeros for what does not exist)
    __device__ __forceinline__ void load(const MuonMat& M, int tile, int col0, float (&g)[NQ][4], float (&m)[NQ][4]) const {
        const float *pg = M.g, *pm = M.m;
        if (mode == kRows && tile + 1 < M.tiles) {
            const int t0 = tile * kMuonTileL * M.J + col0;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                set4(g[i], get4(pg, meta[i] + t0, meta[i] >= 0));
                set4(m[i], get4(pm, meta[i] + t0, meta[i] >= 0));
            }
        } else if (mode == kFlat) {
            const int e0 = (tile * kMuonTileL + col0) * M.J * M.s + 4 * row, total = M.L * M.s;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const bool ok = meta[i] >= 0 && e0 + 4 * T * i < total;
                set4(g[i], get4(pg, e0 + 4 * T * i, ok));
                set4(m[i], get4(pm, e0 + 4 * T * i, ok));
            }
        } else if (mode == kPairs) {
            const int w = M.J * M.s, total = M.L * M.s, e0 = (tile * kMuonTileL + col0 + row) * w + x;
#pragma unroll
            for (int p = 0; p < 2 * NQ; ++p) {
                const int e = e0 + p * kPairCols * w;
                const bool a = x < w && e < total, b = x + 1 < w && e + 1 < total;
                g[p >> 1][(p & 1) * 2] = a ? pg[e] : 0.f;
                g[p >> 1][(p & 1) * 2 + 1] = b ? pg[e + 1] : 0.f;
                m[p >> 1][(p & 1) * 2] = a ? pm[e] : 0.f;
                m[p >> 1][(p & 1) * 2 + 1] = b ? pm[e + 1] : 0.f;
            }
        } else {
            const bool vec = ((M.tall ? M.s : M.L) & 3) == 0;      // whole quads or none
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                int n;
                const int e = quad(M, tile, col0, i, n);
                if (vec) {
                    set4(g[i], get4(pg, e, n > 0));
                    set4(m[i], get4(pm, e, n > 0));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        g[i][k] = k < n ? pg[e + k] : 0.f;
                        m[i][k] = k < n ? pm[e + k] : 0.f;
                    }
                }
            }
        }
    }
    // The same into this thread's own 16-byte cells at `raw` (g's NQ, then m's, T cells apart), asynchronously.
    __device__ __forceinline__ void fetch(const MuonMat& M, int tile, int col0, uint8_t* raw) const {
        const float *pg = M.g, *pm = M.m;
        uint8_t* const rm = raw + NQ * T * 16;
        auto quads = [&](int i, int e, bool ok) {
            ptx::cp_async16(ptx::smem_u32(raw) + i * T * 16, ok ? pg + e : pg, ok ? 16 : 0);
            ptx::cp_async16(ptx::smem_u32(rm) + i * T * 16, ok ? pm + e : pm, ok ? 16 : 0);
        };
        auto single = [&](int i, int k, int e, bool ok) {
            ptx::cp_async4(ptx::smem_u32(raw) + i * T * 16 + k * 4, ok ? pg + e : pg, ok ? 4 : 0);
            ptx::cp_async4(ptx::smem_u32(rm) + i * T * 16 + k * 4, ok ? pm + e : pm, ok ? 4 : 0);
        };
        if (mode == kRows && tile + 1 < M.tiles) {
            const int t0 = tile * kMuonTileL * M.J + col0;
#pragma unroll
            for (int i = 0; i < NQ; ++i) quads(i, meta[i] + t0, meta[i] >= 0);
        } else if (mode == kFlat || mode == kPairs) {
            // the step's TL w elements as they lie in memory (kPairs: for read_pairs)
            const int n = TL * M.J * M.s, e0 = (tile * kMuonTileL + col0) * M.J * M.s, total = M.L * M.s - e0;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const int f = 4 * ((int)threadIdx.x + i * T);
                quads(i, e0 + f, f < n && f < total);
            }
        } else {
            const bool vec = ((M.tall ? M.s : M.L) & 3) == 0;      // whole quads or none
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                int n;
                const int e = quad(M, tile, col0, i, n);
                if (vec) {
                    quads(i, e, n > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) single(i, k, e + k, k < n);
                }
            }
        }
    }
    static __device__ __forceinline__ void read(const uint8_t* raw, float (&g)[NQ][4], float (&m)[NQ][4]) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            set4(g[i], *reinterpret_cast<const float4*>(raw + i * T * 16));
            set4(m[i], *reinterpret_cast<const float4*>(raw + (NQ + i) * T * 16));
        }
    }
    // kPairs: this thread's pairs out of a step that the block's threads have fetched to `raw` (its first cell)
    __device__ __forceinline__ void read_pairs(const MuonMat& M, const uint8_t* raw, float (&g)[NQ][4], float (&m)[NQ][4]) const {
        const int w = M.J * M.s;
        const float* const pg = reinterpret_cast<const float*>(raw) + row * w + x;
        const float* const pm = pg + NQ * T * 4;
        const bool a = x < w, b = x + 1 < w;
#pragma unroll
        for (int p = 0; p < 2 * NQ; ++p) {
            const int e = p * kPairCols * w;
            g[p >> 1][(p & 1) * 2] = a ? pg[e] : 0.f;
            g[p >> 1][(p & 1) * 2 + 1] = b ? pg[e + 1] : 0.f;
            m[p >> 1][(p & 1) * 2] = a ? pm[e] : 0.f;
            m[p >> 1][(p & 1) * 2 + 1] = b ? pm[e + 1] : 0.f;
        }
    }
    // stores v to where load() took it from in `dst`
    __device__ __forceinline__ void store(const MuonMat& M, float* dst, int tile, int col0, const float (&v)[NQ][4]) const {
        if (mode == kRows && tile + 1 < M.tiles) {
            const int t0 = tile * kMuonTileL * M.J + col0;
#pragma unroll
            for (int i = 0; i < NQ; ++i)
                if (meta[i] >= 0)
                    *reinterpret_cast<float4*>(dst + meta[i] + t0) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        } else if (mode == kFlat) {
            const int e0 = (tile * kMuonTileL + col0) * M.J * M.s + 4 * row, total = M.L * M.s;
#pragma unroll
            for (int i = 0; i < NQ; ++i)
                if (meta[i] >= 0 && e0 + 4 * T * i < total)
                    *reinterpret_cast<float4*>(dst + e0 + 4 * T * i) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        } else if (mode == kPairs) {
            const int w = M.J * M.s, total = M.L * M.s, e0 = (tile * kMuonTileL + col0 + row) * w + x;
#pragma unroll
            for (int p = 0; p < 2 * NQ; ++p) {
                const int e = e0 + p * kPairCols * w;
                if (x < w && e < total) dst[e] = v[p >> 1][(p & 1) * 2];
                if (x + 1 < w && e + 1 < total) dst[e + 1] = v[p >> 1][(p & 1) * 2 + 1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                int n;
                const int e = quad(M, tile, col0, i, n);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < n) dst[e + k] = v[i][k];
            }
        }
    }
    // The three parts of scale * v (scaled by 1, UP and UP^2) into the tile at `base`.  Elements of the tile past the matrix's end are
    // zeros; rows past the matrix's are left alone.
    template <int UP>
    __device__ __forceinline__ void put(const MuonMat& M, uint32_t base, uint32_t plane, int col0, float scale,
                                        const float (&v)[NQ][4]) const {
        const uint64_t scale2 = ptx::f32x2(scale, scale);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            uint32_t a[3], b[3];
            muon_split2<UP>(ptx::f32x2(v[i][0], v[i][1]), scale2, a);
            muon_split2<UP>(ptx::f32x2(v[i][2], v[i][3]), scale2, b);
            if (mode == kPairs) {
                if (x < M.J * M.s) {
                    const uint32_t aa = base + muon_elem_at(col0 + row + 2 * i * kPairCols, x);
                    const uint32_t bb = base + muon_elem_at(col0 + row + (2 * i + 1) * kPairCols, x);
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        ptx::st_shared_u32(aa + p * plane, a[p]);
                        ptx::st_shared_u32(bb + p * plane, b[p]);
                    }
                }
                continue;
            }
            uint32_t at;
            bool ok = true;
            if (mode == kFlat) { at = base + (uint32_t)(meta[i] + col0 * 128); ok = meta[i] >= 0; }
            else if (mode == kRows) { at = base + muon_elem_at(row, col0 + x) + (uint32_t)(i * kRowStep) * 128u; ok = meta[i] >= 0; }
            else if (!M.tall) at = base + muon_elem_at(row + i * kRowStep, col0 + x);
            else at = base + muon_elem_at(col0 + row + i * kColStep, x);
            if (ok) {
#pragma unroll
                for (int p = 0; p < 3; ++p) ptx::st_shared_v2(at + p * plane, a[p], b[p]);
            }
        }
    }
};

struct MuonDesc {
    uint32_t lo, hi;
    __device__ __forceinline__ MuonDesc(uint64_t d) : lo((uint32_t)d), hi((uint32_t)(d >> 32)) {}
};
// D0 += a0 b0, D1 += the products of a lower order (but a2 b2) over one K step; the parts of an operand lie `astep` / `bstep` (in descriptor units of 16 bytes) apart.  FIRST: the products start
// the accumulators.
template <bool FIRST>
__device__ __forceinline__ void muon_mma(uint32_t d0, uint32_t d1, MuonDesc a, MuonDesc b, uint32_t astep, uint32_t bstep,
                                         uint32_t idesc) {
    ptx::tc_mma_f16_lo<!FIRST>(d0, a.lo, a.hi, b.lo, b.hi, idesc);
    ptx::tc_mma_f16_lo<!FIRST>(d1, a.lo, a.hi, b.lo + bstep, b.hi, idesc);
    ptx::tc_mma_f16_lo<true>(d1, a.lo + astep, a.hi, b.lo, b.hi, idesc);
    ptx::tc_mma_f16_lo<true>(d1, a.lo + astep, a.hi, b.lo + bstep, b.hi, idesc);
    ptx::tc_mma_f16_lo<true>(d1, a.lo, a.hi, b.lo + 2 * bstep, b.hi, idesc);
    ptx::tc_mma_f16_lo<true>(d1, a.lo + 2 * astep, a.hi, b.lo, b.hi, idesc);
    ptx::tc_mma_f16_lo<true>(d1, a.lo + astep, a.hi, b.lo + 2 * bstep, b.hi, idesc);
    ptx::tc_mma_f16_lo<true>(d1, a.lo + 2 * astep, a.hi, b.lo + bstep, b.hi, idesc);
}
// The Gram pass's, a tile with itself: four accumulators of 128 columns (see the top of the file).
template <bool FIRST>
__device__ __forceinline__ void muon_gram_mma(uint32_t d, MuonDesc a, uint32_t step, uint32_t idesc) {
    auto mma = [&](auto first, int acc, uint32_t i, uint32_t j) {
        ptx::tc_mma_f16_lo<!decltype(first)::value>(d + acc * 128, a.lo + i * step, a.hi, a.lo + j * step, a.hi, idesc);
    };
    constexpr std::integral_constant<bool, FIRST> first{};
    constexpr std::false_type more{};
    mma(first, 0, 0, 0);
    mma(first, 1, 0, 1);
    mma(more, 1, 1, 0);
    mma(first, 2, 1, 1);
    mma(more, 2, 0, 2);
    mma(more, 2, 2, 0);
    mma(first, 3, 1, 2);
    mma(more, 3, 2, 1);
}

// ---------------------------------------------------------------------------------------------- Gram
// x 2^k as a double, from the bits of a finite x (a conversion instruction is several times slower than
// these four); what is below the smallest normal float becomes 0.
__device__ __forceinline__ double muon_to_double(float x, int k) {
    const uint32_t b = __float_as_uint(x), mag = b & 0x7fffffffu;
    const uint32_t hi = (b & 0x80000000u) | ((mag >> 3) + ((uint32_t)(1023 - 127 + k) << 20));
    return mag < 0x00800000u ? 0.0 : __hiloint2double((int)hi, (int)(b << 29));
}

constexpr int kGramLoad = 512;          // threads that load and split, warps 0 .. 15
constexpr int kGramThreads = kGramLoad + 32;   // and a warp that issues the products
constexpr int kGramStage = 3 * kMuonPlane;
constexpr int kGramRaw = 128 * kMuonTileL * 8; // a tile's g and m
constexpr int kGramSmem = 2 * kGramStage + 2 * kGramRaw + 1024;
static_assert(kGramSmem + 1024 <= 232448, "shared memory per CTA");
constexpr int kGramUp = 64;             // the lower parts' factor: the accumulators are in units of 1, 2^-6, 2^-12 and 2^-18
constexpr int kGramExactTiles = 16;     // tiles whose x0 x0 sums stay below 2^24 (|x0| <= 128, 64 columns each)

// One item: the partial Gram matrix (of its two equal halves the elements [c][r], c <= r) of a run of tiles
// over one pair of 64-row groups (the only pair for s <= 128).  Sixteen warps copy a tile's g and m to shared memory
// (two tiles ahead, every thread its own elements) and split u into one of two places; a further warp issues a place's products.
// The scale of the split is a power of two, 1.5 to 3 times the first tile's largest |u|.  A tile that exceeds it
// takes the sums out of the accumulators and starts them anew at its own scale, and so does every 16th tile.
// 8 bytes per element: 32 adapters of rank 8 to 128 at 4096 -> 14336 (40 M elements) take 191 us for the bytes' 49, 3.5
// us per tile (1.1 of them the products') and 7 per item to begin and to take the sums out; what bounds a tile is the
// chain from its copies through the split and the proxy fence to its products, one tile at a time over the block.
__global__ void __launch_bounds__(kGramThreads, 1)
muon_gram_kernel(const MuonMat* __restrict__ mats, int n, int* err_flag, uint64_t timeout_ns) {
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    enum { kAdd, kStart, kStop };                 // what the products of a place do to the accumulators
    __shared__ __align__(8) uint64_t full[2], done[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ volatile int what[2];
    __shared__ int which;
    __shared__ float red[kGramLoad / 32];
    __shared__ MuonMat record;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the item's matrix, found by all threads at once (a search would wait for six loads in turn)
    for (int k = tid; k < n; k += kGramThreads)
        if (mats[k].gram0 <= (int)blockIdx.x && (k + 1 == n || mats[k + 1].gram0 > (int)blockIdx.x)) which = k;
    if (tid == 0) {
        for (int k = 0; k < 2; ++k) {
            ptx::mbar_init(&full[k], kGramLoad / 32);
            ptx::mbar_init(&done[k], 1);
        }
        abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == kGramLoad / 32) {
        ptx::tmem_alloc<512>(&tmem_slot);
        ptx::tmem_relinquish();
    }
    // rows past the matrix's stay zero (their products reach no output, but must not be NaN)
    for (int e = tid; e < 2 * kGramStage / 16; e += kGramThreads) reinterpret_cast<uint4*>(smem)[e] = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    muon_fetch(&record, mats + which);
    __syncthreads();
    const MuonMat& M = record;
    const int item = blockIdx.x - M.gram0;
    const int chunk = item / M.npairs;
    int ga = 0, gb = 1;
    const int ng = (M.s + 63) / 64;
    for (int k = item - chunk * M.npairs; k > 0; --k)
        if (++gb >= ng) { ++ga; gb = ga + 1; }
    const int t0 = chunk * M.per_chunk, t1 = min(M.tiles, t0 + M.per_chunk);
    const uint32_t tmem = tmem_slot;
    const uint32_t s0 = ptx::smem_u32(smem);

    if (warp < kGramLoad / 32) {
        using Tile = MuonTile<kGramLoad, kMuonTileL, 128>;
        Tile T;
        T.enter(M, tid, M.npairs == 1, ga * 64, gb * 64);
        uint8_t* const raw_cells = smem + 2 * kGramStage + tid * 16;
        T.fetch(M, t0, 0, raw_cells);
        ptx::cp_async_commit();
        if (t0 + 1 < t1) T.fetch(M, t0 + 1, 0, raw_cells + kGramRaw);
        ptx::cp_async_commit();
        const uint64_t mu2 = ptx::f32x2(M.mu, M.mu);
        const bool nesterov = M.nesterov != 0, pairs = T.mode == Tile::kPairs;
        uint32_t count = 0;     // tiles handed over: the k-th went to place k & 1
        int since = 0;          // tiles in the accumulators
        float scale = 0.f;      // 2^-unit
        int unit = 0;
        bool stored = false, bad = false;
        float item_max = 0.f;
        // the products of the k-th tile have ended
        auto wait_step = [&](uint32_t k) {
            ptx::mbar_wait_many(&done[k & 1], (k >> 1) & 1u, &abort_flag, timeout_ns, err_flag);
            ptx::tc_fence_after();
        };
        auto sync = [&] { ptx::named_bar_sync(1, kGramLoad); };

        // Adds the accumulators, in units of 2^(2 unit), to the item's partial.
        auto drain = [&]() {
            wait_step(count - 1);
            double* out = M.part + (int64_t)chunk * M.s * M.s;
            const int k2 = 2 * unit;
            const int r = (warp & 3) * 32 + lane, part = warp >> 2;
            const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            double* stack = reinterpret_cast<double*>(smem);   // [s][128], the diagonal blocks' columns
            const int j = M.J > 1 ? r / M.s : 0;
            if (M.J > 1) sync();                               // every warp has seen the products end
            for (int c0 = part * 16; c0 < 128; c0 += 64) {     // the four warps of these rows take turns
                // only columns up to the warp's last row are needed
                if (c0 > (warp & 3) * 32 + 31) break;
                // a diagonal block is in several pairs: the pair with the next group writes it (the last group's, the
                // pair with the one before)
                const int gr = r < 64 ? ga : gb, gc = c0 < 64 ? ga : gb, rr = gr * 64 + (r & 63);
                const bool own = (gr != gc || (gr == ga ? gb == ga + 1 : ga == ng - 2)) && rr < M.s;
                double* const o = out + (gc * 64 + (c0 & 63)) * M.s + rr;      // lanes on consecutive addresses
                const int cols = min(16, M.s - (gc * 64 + (c0 & 63)));
#pragma unroll 1
                for (int k0 = 0; k0 < 16; k0 += 8) {
                    uint32_t d[4][8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) ptx::tmem_ld8(t_row + q * 128 + c0 + k0, d[q]);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int c = c0 + k0 + k;
                        if (c > r) continue;
                        const float low = fmaf(__uint_as_float(d[3][k]), 1.f / kGramUp, __uint_as_float(d[2][k]));
                        const double v = muon_to_double(__uint_as_float(d[0][k]), k2) + (muon_to_double(__uint_as_float(d[1][k]), k2 - 6) +
                                                                                        muon_to_double(low, k2 - 12));
                        if (M.J > 1) {
                            if (j < M.J && c >= j * M.s) stack[(c - j * M.s) * 128 + r] = v;
                        } else if (own && k0 + k < cols) {
                            o[(k0 + k) * M.s] = stored ? o[(k0 + k) * M.s] + v : v;
                        }
                    }
                }
            }
            if (M.J > 1) {
                sync();
                const int s2 = M.s * M.s;
                for (int e = tid; e < s2; e += kGramLoad) {
                    const int cc = e / M.s, rr = e - cc * M.s;
                    if (cc > rr) continue;
                    double v = 0.0;
                    for (int q = 0; q < M.J; ++q) v += stack[cc * 128 + q * M.s + rr];
                    out[e] = stored ? out[e] + v : v;
                }
                sync();
                // the stages held sums: clear their rows again
                for (int e = tid; e < 2 * kGramStage / 16; e += kGramLoad)
                    reinterpret_cast<uint4*>(smem)[e] = make_uint4(0, 0, 0, 0);
            }
            ptx::tc_fence_before();
            sync();
            stored = true;
            since = 0;
        };
        // hands a place to the issuing warp
        auto hand_over = [&](int todo) {
            if (tid == 0) what[count & 1] = todo;
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&full[count & 1]);
            ++count;
        };

        for (int t = t0; t < t1; ++t) {
            float u[Tile::NQ][4];
            {
                float g[Tile::NQ][4], m[Tile::NQ][4];
                uint8_t* const cells = raw_cells + ((t - t0) & 1) * kGramRaw;
                ptx::cp_async_wait<1>();
                if (pairs) {
                    sync();                             // other threads' copies are read
                    T.read_pairs(M, cells - tid * 16, g, m);
                } else {
                    Tile::read(cells, g, m);
                }
#pragma unroll
                for (int i = 0; i < Tile::NQ; ++i)
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const uint64_t gg = ptx::f32x2(g[i][k], g[i][k + 1]);
                        const uint64_t a = ptx::f32x2_fma(mu2, ptx::f32x2(m[i][k], m[i][k + 1]), gg);
                        const float2 c = ptx::f32x2_get(nesterov ? ptx::f32x2_fma(mu2, a, gg) : a);
                        u[i][k] = c.x;
                        u[i][k + 1] = c.y;
                    }
                if (!pairs) {
                    if (t + 2 < t1) T.fetch(M, t + 2, 0, cells);
                    ptx::cp_async_commit();
                }
            }
            float big = 0.f;
#pragma unroll
            for (int i = 0; i < Tile::NQ; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) big = ptx::max_nan(big, fabsf(u[i][k]));
            item_max = fmaxf(item_max, big);
            bool over = scale == 0.f || !(big * scale <= 128.f);      // also a NaN
            // (the first tile has no scale yet; a first tile of zeros leaves it to the next)
            over = ptx::named_bar_or(1, kGramLoad, over);
            if (pairs) {                                // every thread has read the cells
                if (t + 2 < t1) T.fetch(M, t + 2, 0, raw_cells + ((t - t0) & 1) * kGramRaw);
                ptx::cp_async_commit();
            }
            if (over || since == kGramExactTiles) {
                if (since > 0) drain();
                if (over) {
                    float w = big;
                    const bool nan = !(big * 0.f == 0.f);      // or an infinity
                    for (int o = 16; o > 0; o >>= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
                    if (lane == 0) red[warp] = w;
                    bad = ptx::named_bar_or(1, kGramLoad, nan) || bad;
                    w = 0.f;
                    for (int k = 0; k < kGramLoad / 32; ++k) w = fmaxf(w, red[k]);
                    if (!bad && w > 0.f) {
                        // a power of two at least 1.5 times the largest, so that the next steps' seldom exceed it
                        // (1.5 w itself may be past the largest float)
                        unit = max(ilogbf(0.75f * w) + 2, -100) - 7;
                        scale = scalbnf(1.f, -unit);
                    }
                    sync();
                }
            }
            if (bad) break;                     // a NaN or an infinity: the whole matrix becomes NaN
            if (scale == 0.f) continue;         // nothing but zeros so far
            if (count >= 2) wait_step(count - 2);              // the products that last read this place
            T.put<kGramUp>(M, s0 + (count & 1) * kGramStage, kMuonPlane, 0, scale, u);
            hand_over(since == 0 ? kStart : kAdd);
            ++since;
        }
        if (since > 0) drain();
        if (count >= 2) wait_step(count - 2);
        hand_over(kStop);
        // nothing but zeros, or a NaN or an infinity somewhere in the item
        if (!stored || bad) {
            sync();
            double* out = M.part + (int64_t)chunk * M.s * M.s;
            const double v = bad ? __longlong_as_double(0x7ff8000000000000ll) : 0.0;
            for (int e = tid; e < M.s * M.s; e += kGramLoad) {
                const int r = e / M.s, c = e - r * M.s, gr = r >> 6, gc = c >> 6;
                if (M.npairs == 1 || ((gr == ga || gr == gb) && (gc == ga || gc == gb) &&
                                      (gr != gc || (gr == ga ? gb == ga + 1 : ga == ng - 2))))
                    out[e] = v;
            }
        }
        for (int o = 16; o > 0; o >>= 1) item_max = fmaxf(item_max, __shfl_xor_sync(0xffffffffu, item_max, o));
        if (lane == 0) red[warp] = item_max;
        sync();
        if (tid == 0) {
            float w = 0.f;
            for (int k = 0; k < kGramLoad / 32; ++k) w = fmaxf(w, red[k]);
            M.hdr[2 + item] = w;
        }
    } else {
        // (the whole warp runs this, so that addresses stay in uniform registers; one lane issues)
        const bool one = ptx::elect_one();
        const bool tall = M.tall != 0;
        const uint32_t idesc = ptx::idesc_f16_f32(128, 128, tall, tall);
        for (uint32_t k = 0;; ++k) {
            const int place = k & 1;
            if (!ptx::mbar_wait_many(&full[place], (k >> 1) & 1u, &abort_flag, timeout_ns, err_flag)) break;
            const int todo = what[place];
            if (todo == kStop) break;
            ptx::tc_fence_after();
            const uint32_t base = s0 + place * kGramStage;
            const uint32_t kstep = tall ? 2048 / 16 : 32 / 16;
            const MuonDesc d0 = tall ? ptx::smem_desc_sw128(base, 8192, 1024) : ptx::smem_desc_sw128(base, 16, 1024);
            if (one) {
                MuonDesc d = d0;
                if (todo == kStart) muon_gram_mma<true>(tmem, d, kMuonPlane / 16, idesc);
                else muon_gram_mma<false>(tmem, d, kMuonPlane / 16, idesc);
#pragma unroll
                for (int q = 1; q < kMuonTileL / 16; ++q) {
                    d.lo += kstep;
                    muon_gram_mma<false>(tmem, d, kMuonPlane / 16, idesc);
                }
                ptx::tc_commit(&done[place]);
            }
            __syncwarp();
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kGramLoad / 32) ptx::tmem_dealloc<512>(tmem);
}

// ----------------------------------------------------------------------------------------- iteration
// Three forms, by s, all on the fp64 tensor cores (64 multiply-adds per clock and SM):
//   s <= 64    one block, G, P and Q in shared memory, the lower halves of the products
//   s <= 128   a cluster of four blocks, each with 32 rows of G and Q and a copy of the whole matrix that is the
//              right-hand operand: first G (for P = a I + b G + c G^2), then P.  With P at hand a block's rows of
//              Q P, of R = G P and of the new G = R P need nothing of the others', so a step takes two exchanges,
//              each block copying its rows into every block's matrix
//   s <= 256   a cluster of eight blocks with 32 rows each.  The matrices are in L2, where they come from in
//              stages; a block computes the blocks of its rows on and after the diagonal, half of them, cyclically,
//              and writes them to both places.
// (Products of symmetric matrices that commute are symmetric: B's rows serve as its columns.)
// Five steps, with the sum of the partials: one matrix of 16 27 us, of 64 64, of 128 137, of 256 357; 64 of 8 to 128
// (ranks of 32 adapters) 186; fifteen of 256 366, sixteen 546 (15 clusters of eight have an SM per block; two blocks of
// an SM share its pipe).  Bound by the fp64 pipe and, nearly as much again, by the short products' barriers and loads:
// a step at 128 takes 25 us, 17 of them the pipe's, at 256 73 of which 43.  Clusters of eight with 16 rows each were
// faster for one matrix of 128 (92 us) but with their 186 KB only 15 are resident at once, and the up mix took 274;
// products dealt over eight blocks from L2, with two barriers more per step, 218 and (sixteen of 256) 890.
constexpr int kNsRows = 32;                            // rows of a cluster's block
constexpr int kNsPitch = 64 + 4;                       // doubles; rows shift by 4 so that fragment loads spread
constexpr int kNsSmallS = 64;
constexpr int kNsMidS = 128, kNsMidPitch = kNsMidS + 4, kNsMidCluster = kNsMidS / kNsRows;
constexpr int kNsBigPitch = 256 + 4, kNsBigCluster = 256 / kNsRows;
constexpr int kNsK = 64, kNsStages = 2, kNsStage = kNsRows * (kNsK + 4);   // doubles of one stage of the streamed operand
constexpr int kNsSmallSmem = 3 * kNsSmallS * kNsPitch * 8;
constexpr int kNsMidSmem = (kNsMidS + 2 * kNsRows) * kNsMidPitch * 8;
constexpr int kNsBigSmem = (kNsRows * kNsBigPitch + kNsStages * kNsStage) * 8;
static_assert(kNsSmallSmem <= kNsMidSmem && kNsMidSmem + 2048 <= 232448, "shared memory per CTA");
static_assert(2 * (kNsBigSmem + 2048) <= 232448, "two CTAs per SM");

__device__ __forceinline__ void dmma_16x8x8(double (&d)[4], const double (&a)[4], const double (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f64.f64.f64.f64 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+d"(d[0]), "+d"(d[1]), "+d"(d[2]), "+d"(d[3])
        : "d"(a[0]), "d"(a[1]), "d"(a[2]), "d"(a[3]), "d"(b[0]), "d"(b[1]));
}
// acc (16 R x 8 N) += the 16 R rows at `a` times the 8 N rows at `b`, over k8 steps of eight.
template <int R, int N>
__device__ __forceinline__ void dmma_block(double (&acc)[R][N][4], const double* a, int ap, const double* b, int bp, int k8) {
    const int lane = threadIdx.x & 31;
    const double* as = a + (lane >> 2) * ap + (lane & 3);
    const double* bs = b + (lane >> 2) * bp + (lane & 3);
#pragma unroll 4
    for (int k = 0; k < k8; ++k, as += 8, bs += 8) {
        double x[R][4], y[N][2];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const double* p = as + 16 * i * ap;
            x[i][0] = p[0];
            x[i][1] = p[8 * ap];
            x[i][2] = p[4];
            x[i][3] = p[8 * ap + 4];
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            y[j][0] = bs[8 * j * bp];
            y[j][1] = bs[8 * j * bp + 4];
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) dmma_16x8x8(acc[i][j], x[i], y[j]);
    }
}
// That block's elements of this lane, two neighbours at a time: f(row, column, value, its right neighbour).
template <int R, int N, typename F> __device__ __forceinline__ void dmma_each(const double (&acc)[R][N][4], F&& f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                f(16 * i + (lane >> 2) + 8 * h, 8 * j + (lane & 3) * 2, acc[i][j][2 * h], acc[i][j][2 * h + 1]);
}

// A product for s <= 64 on one block with its matrices in shared memory (pitch kNsPitch): the 10 blocks of
// 16 x 16 of the lower half over the eight warps, their results kept in registers until every warp has
// read its operands, so that C may be A or B.
template <typename F>
__device__ __forceinline__ void ns_product_small(const double* A, const double* B, int sp, F&& out) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nt = (sp + 15) / 16, tiles = nt * (nt + 1) / 2;
    double acc[2][2][4] = {};
    auto tile_of = [](int t, int& ti, int& tj) {
        ti = 0;
        while (t > ti) { t -= ti + 1; ++ti; }
        tj = t;
    };
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int t = warp + 8 * w;
        if (t >= tiles) continue;
        int ti, tj;
        tile_of(t, ti, tj);
        const double* as = A + (ti * 16 + (lane >> 2)) * kNsPitch + (lane & 3);
        const double* bs = B + (tj * 16 + (lane >> 2)) * kNsPitch + (lane & 3);
#pragma unroll 2
        for (int kk = 0; kk < sp; kk += 8) {
            const double a[4] = {as[kk], as[kk + 8 * kNsPitch], as[kk + 4], as[kk + 8 * kNsPitch + 4]};
            const double b0[2] = {bs[kk], bs[kk + 4]};
            const double b1[2] = {bs[kk + 8 * kNsPitch], bs[kk + 8 * kNsPitch + 4]};
            dmma_16x8x8(acc[w][0], a, b0);
            dmma_16x8x8(acc[w][1], a, b1);
        }
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int t = warp + 8 * w;
        if (t >= tiles) continue;
        int ti, tj;
        tile_of(t, ti, tj);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ti * 16 + (lane >> 2) + (i >> 1) * 8, c = tj * 16 + j * 8 + (lane & 3) * 2 + (i & 1);
                if (r < sp && c <= r) out(r, c, acc[w][j][i]);
            }
    }
    __syncthreads();
}

// Byte offset of the eight-element chunk (row, 8 k8 ..) of part `part` of Q as the apply pass stages it:
// blocks of 128 rows x 64 columns, 128-byte swizzled, ordered (row half, column block, part).
__host__ __device__ __forceinline__ int64_t muon_q_at(int kblocks, int row, int k8, int part) {
    const int64_t block = ((int64_t)(row >> 7) * kblocks + (k8 >> 3)) * 3 + part;
    const int r = row & 127;
    return block * kMuonPlane + r * 128 + (((k8 & 7) ^ (r & 7)) << 4);
}

// Where the Gram matrix stands, sp x sp with zeros past s, for the iteration to scale.
__device__ __forceinline__ double* muon_gram_at(const MuonMat& M) {
    const int64_t sp = (M.s + 7) & ~7;
    return M.ns + (M.s > kNsMidS ? 4 * sp * sp : 0);
}
// The sum of the Gram partials (their halves [c][r], r >= c, in the chunks' order), to both halves.  kSumBlocks
// blocks per matrix, a warp per row at a time: 16 loads of 8 bytes in flight per thread.  (Summed by the iteration's
// few blocks instead, 64 partials of 128 x 128 took 200 us of its 316.)
constexpr int kSumBlocks = 32;
__global__ void __launch_bounds__(256) muon_sum_kernel(const MuonMat* __restrict__ mats) {
    const MuonMat& M = mats[blockIdx.x / kSumBlocks];
    const int s = M.s, sp = (s + 7) & ~7, s2 = s * s, chunks = M.nchunks, lane = threadIdx.x & 31;
    double* const G = muon_gram_at(M);
    const double* const part = M.part;
    for (int c = (blockIdx.x % kSumBlocks) * 8 + (threadIdx.x >> 5); c < sp; c += kSumBlocks * 8)
        for (int r0 = (c & ~31) + lane; r0 < sp; r0 += 128) {
            double g[4] = {};
            bool ok[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) ok[q] = c < s && r0 + 32 * q >= c && r0 + 32 * q < s;
            const double* p = part + (int64_t)c * s + r0;
            int ch = 0;
            for (; ch + 4 <= chunks; ch += 4, p += 4 * (int64_t)s2) {
                double v[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[k][q] = ok[q] ? p[k * (int64_t)s2 + 32 * q] : 0.0;
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int q = 0; q < 4; ++q) g[q] += v[k][q];
            }
            for (; ch < chunks; ++ch, p += s2)
#pragma unroll
                for (int q = 0; q < 4; ++q) g[q] += ok[q] ? p[32 * q] : 0.0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = r0 + 32 * q;
                if (r < c || r >= sp) continue;
                G[c * sp + r] = g[q];
                G[r * sp + c] = g[q];
            }
        }
}

// The iteration on the matrices' Gram matrices, then Q's three fp16 parts for the apply pass (block-diagonal over
// the stacked blocks) and the scales.  order: n matrices, BIG: those with s > 128, a cluster of eight each; else
// n_mid of s > 64, a cluster of four each, and then those that take a block each.
template <bool BIG>
__global__ void __launch_bounds__(256)
muon_ns_kernel(const MuonMat* __restrict__ mats, const int32_t* __restrict__ order, int n_mid, int n, int* err_flag,
               uint64_t timeout_ns) {
    constexpr int CLUSTER = BIG ? kNsBigCluster : kNsMidCluster;
    extern __shared__ __align__(16) double sm[];
    __shared__ double redd[8];
    __shared__ float redf[8], qmaxes[CLUSTER];
    __shared__ MuonMat record;
    __shared__ __align__(8) uint64_t arrived;
    __shared__ int abort_flag;
    const bool small = !BIG && blockIdx.x >= (unsigned)n_mid * CLUSTER;
    const int which = small ? n_mid + (int)blockIdx.x - n_mid * CLUSTER : (int)blockIdx.x / CLUSTER;
    if (which >= n) return;      // the last cluster's spare blocks (their cluster holds small matrices only)
    muon_fetch(&record, mats + order[which]);
    if (threadIdx.x == 0) {
        ptx::mbar_init(&arrived, 1);
        abort_flag = 0;
        ptx::fence_barrier_init();
    }
    __syncthreads();
    const MuonMat& M = record;
    const int rank = small ? 0 : (int)ptx::cluster_ctarank();
    const int tid = threadIdx.x, warp = tid >> 5, s = M.s, sp = (s + 7) & ~7, k8 = sp / 8;
    // Blocks past the matrix's rows leave: the cluster's barrier waits for threads that have not ended, and nobody
    // copies or stores into theirs.  (Sixteen matrices of 200: 403 us, 435 with them in every barrier.)
    const int active = small ? 1 : (s + kNsRows - 1) / kNsRows;
    if (rank >= active) return;
    // this block's rows of G and Q (from row r0 of the matrix on), and its own copies' pitch
    const int nr = small ? s : kNsRows, r0 = rank * kNsRows;
    const int pitch = BIG ? kNsBigPitch : small ? kNsPitch : kNsMidPitch;
    // small: G, P, Q; mid: the matrix, then the block's rows of G and Q; big: the rows of the left operand, stages
    double* const G = BIG || small ? sm : sm + kNsMidS * kNsMidPitch;
    double* const Q = BIG ? sm : small ? G + 2 * kNsSmallS * kNsPitch : G + kNsRows * kNsMidPitch;
    auto sync = [&] {
        if (small) __syncthreads();
        else ptx::cluster_sync();
    };
    // |u|_F^2, the trace of G, and max |u|: by every block in the same order
    const double* const raw = muon_gram_at(M);
    double tr = 0.0;
    for (int e = tid; e < s; e += 256) tr += raw[e * (sp + 1)];
    float umax = 0.f;
    for (int e = tid; e < M.nchunks * M.npairs; e += 256) umax = fmaxf(umax, M.hdr[2 + e]);
    auto block_sum = [&](double v) {
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        __syncthreads();
        if ((tid & 31) == 0) redd[warp] = v;
        __syncthreads();
        v = 0.0;
        for (int w = 0; w < 8; ++w) v += redd[w];
        return v;
    };
    auto block_max = [&](float v) {
        for (int o = 16; o > 0; o >>= 1) v = ptx::max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
        __syncthreads();
        if ((tid & 31) == 0) redf[warp] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < 8; ++w) v = ptx::max_nan(v, redf[w]);
        return v;
    };
    tr = block_sum(tr);
    umax = block_max(umax);
    const double inv = 1.0 / (sqrt(tr) + (double)M.eps);
    // zeros past s, and the scaled G: its own rows, and as the first right-hand operand
    {
        const int cells = BIG ? kNsRows * kNsBigPitch : (small ? kNsSmallSmem : kNsMidSmem) / 8;
        for (int e = tid; e < cells / 2; e += 256) reinterpret_cast<double2*>(sm)[e] = make_double2(0.0, 0.0);
        __syncthreads();
        const int h = sp / 2, rows = BIG ? min(kNsRows, sp - r0) : sp;
#pragma unroll 4
        for (int e = tid; e < rows * h; e += 256) {
            const int r = e / h, c2 = e - r * h;
            double2 v = reinterpret_cast<const double2*>(raw)[(BIG ? r0 + r : r) * h + c2];
            v.x = (v.x * inv) * inv;
            v.y = (v.y * inv) * inv;
            *reinterpret_cast<double2*>(sm + r * pitch + 2 * c2) = v;
            if (BIG) reinterpret_cast<double2*>(M.ns)[(r0 + r) * h + c2] = v;
            if (!BIG && !small && r >= r0 && r < r0 + kNsRows) *reinterpret_cast<double2*>(G + (r - r0) * pitch + 2 * c2) = v;
        }
    }
    sync();
    const double a = M.a, b = M.b, c = M.c;
    if constexpr (BIG) {
        double* gG = M.ns;
        double *gP = gG + sp * sp, *gQ = gP + sp * sp, *gR = gQ + sp * sp, *gS = gR + sp * sp;
        double* const stages = sm + kNsRows * kNsBigPitch;
        const int n = active;                             // blocks of 32 rows, and of 32 columns
        // rows of `X` for the left operand
        auto rows_of = [&](const double* X) {
            __syncthreads();
            for (int e = tid; e < kNsRows * (sp / 2); e += 256) {
                const int r = e / (sp / 2), c = (e - r * (sp / 2)) * 2;
                const bool ok = r0 + r < sp;
                ptx::cp_async16(ptx::smem_u32(G + r * kNsBigPitch + c), ok ? X + (r0 + r) * sp + c : X, ok ? 16 : 0);
            }
            ptx::cp_async_commit();               // (product waits for it with its first stage)
        };
        // C = f(those rows times X): the blocks (rank, rank + d mod n), 32 x 32 each, a warp's share 16 x 8
        const int wr = (warp & 1) * 16, wc = (warp >> 1) * 8;
        const int lane = tid & 31;
        const double* const as0 = G + (wr + (lane >> 2)) * kNsBigPitch + (lane & 3);
        const double* const bs0 = stages + (wc + (lane >> 2)) * (kNsK + 4) + (lane & 3);
        auto product = [&](const double* X, double* C, auto&& f) {
            const int nk = (sp + kNsK - 1) / kNsK, steps = (n / 2 + 1) * nk;
            const int fr = tid >> 5, fc = lane * 2;            // this thread's pieces of a stage: rows fr + 8 i
            const uint32_t dst0 = ptx::smem_u32(stages + fr * (kNsK + 4) + fc);
            int fd = 0, fk = 0, ck = 0, cd = 0, rows = 0;
            const double* src = X;
            auto fetch = [&](int k) {
                if (k < steps) {
                    if (fk == 0) {
                        int col = rank + fd;
                        if (col >= n) col -= n;
                        rows = sp - (col * kNsRows + fr);
                        src = X + (col * kNsRows + fr) * sp + fc;
                    }
                    const uint32_t dst = dst0 + (k & 1) * kNsStage * 8;
                    const bool in = fk * kNsK + fc < sp;
#pragma unroll
                    for (int i = 0; i < kNsRows / 8; ++i) {
                        const bool ok = in && 8 * i < rows;
                        ptx::cp_async16(dst + 8 * i * (kNsK + 4) * 8, ok ? src + 8 * i * sp : X, ok ? 16 : 0);
                    }
                    src += kNsK;
                    if (++fk == nk) { fk = 0; ++fd; }
                }
                ptx::cp_async_commit();
            };
            double acc[2][1][1][4] = {};          // even and odd steps of eight: two chains of products
            fetch(0);
            for (int k = 0; k < steps; ++k) {
                ptx::cp_async_wait<0>();
                __syncthreads();                  // the stage is there, and every warp has left the other one
                fetch(k + 1);
                const double* const as = as0 + ck * kNsK;
                const double* const bs = bs0 + (k & 1) * kNsStage;
                auto multiply = [&](int q) {
                    const double x[4] = {as[8 * q], as[8 * q + 8 * kNsBigPitch], as[8 * q + 4], as[8 * q + 8 * kNsBigPitch + 4]};
                    const double y[2] = {bs[8 * q], bs[8 * q + 4]};
                    dmma_16x8x8(acc[q & 1][0][0], x, y);
                };
                const int kn = k8 - ck * (kNsK / 8);
                if (kn >= kNsK / 8) {
#pragma unroll
                    for (int q = 0; q < kNsK / 8; ++q) multiply(q);
                } else {
#pragma unroll
                    for (int q = 0; q < kNsK / 8; ++q)
                        if (q < kn) multiply(q);
                }
                if (++ck < nk) continue;
                int col = rank + cd;
                if (col >= n) col -= n;
                // (the diagonal blocks and those half way round come from both sides: each writes its own)
                const bool mirror = cd > 0 && 2 * cd != n;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[0][0][0][i] += acc[1][0][0][i];
                dmma_each(acc[0], [&](int r, int q, double x, double y) {
                    const int i = r0 + wr + r, j = col * kNsRows + wc + q;
                    if (i >= sp || j >= sp) return;
                    x = f(i, j, x);
                    y = f(i, j + 1, y);
                    *reinterpret_cast<double2*>(C + i * sp + j) = make_double2(x, y);
                    if (mirror) {
                        C[j * sp + i] = x;
                        C[(j + 1) * sp + i] = y;
                    }
                });
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[0][0][0][i] = acc[1][0][0][i] = 0.0;
                ck = 0;
                ++cd;
            }
            ptx::cp_async_wait<0>();
            __syncthreads();
        };
        auto plain = [](int, int, double v) { return v; };
        for (int k = 0; k < M.steps; ++k) {
            const bool last = k + 1 == M.steps;
            double* const P = k == 0 ? gQ : gP;   // (the first step's P is Q_1)
            if (k > 0) rows_of(gG);
            product(gG, P, [&](int i, int j, double v) {
                return (i == j && i < s ? a : 0.0) + b * G[(i - r0) * kNsBigPitch + j] + c * v;
            });
            sync();
            if (!last) product(P, gR, plain);
            if (k > 0) {
                rows_of(gQ);
                product(P, gS, plain);
            }
            if (k + 1 < M.steps || k > 0) sync();
            if (!last) {
                rows_of(gR);
                product(P, gG, plain);
            }
            if (k > 0) {
                double* const t = gQ;
                gQ = gS;
                gS = t;
            }
            if (last) break;
            sync();
        }
        rows_of(gQ);
        ptx::cp_async_wait<0>();
        __syncthreads();
    } else if (small) {
        double* const P = G + kNsSmallS * kNsPitch;
        auto both = [&](double* C, int i, int j, double v) {
            C[i * kNsPitch + j] = v;
            C[j * kNsPitch + i] = v;
        };
        for (int k = 0; k < M.steps; ++k) {
            // P = a I + b G + c G^2 (the first step's P is Q_1)
            ns_product_small(G, G, sp, [&](int i, int j, double v) {
                const double p = (i == j && i < s ? a : 0.0) + b * G[i * kNsPitch + j] + c * v;
                both(P, i, j, p);
                if (k == 0) both(Q, i, j, p);
            });
            if (k > 0) ns_product_small(P, Q, sp, [&](int i, int j, double v) { both(Q, i, j, v); });
            if (k + 1 == M.steps) break;
            ns_product_small(P, G, sp, [&](int i, int j, double v) { both(G, i, j, v); });
            ns_product_small(P, G, sp, [&](int i, int j, double v) { both(G, i, j, v); });
        }
    } else {
        const int c0 = warp * 16;                 // this warp's columns
        const bool work = c0 < s;
        // The blocks send their rows, as they lie in their own copy, to each other's.
        constexpr uint32_t kRowsBytes = kNsRows * kNsMidPitch * 8;
        constexpr int p = kNsMidPitch;
        double* const F = sm;
        double* const own = F + r0 * p;
        uint32_t parity = 0;
        auto exchange = [&]() {
            ptx::fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0) {
                ptx::mbar_arrive_expect_tx(&arrived, (uint32_t)(active - 1) * kRowsBytes);
                for (int k = 1; k < active; ++k) {
                    const uint32_t peer = (uint32_t)((rank + k) % active);
                    ptx::bulk_copy_cluster(ptx::cluster_addr(own, peer), own, kRowsBytes, ptx::cluster_addr(&arrived, peer));
                }
            }
            ptx::mbar_wait_many(&arrived, parity, &abort_flag, timeout_ns, err_flag);
            parity ^= 1u;
        };
        auto put = [&](double* C, const double (&v)[2][2][4]) {
            dmma_each(v, [&](int r, int q, double x, double y) {
                *reinterpret_cast<double2*>(C + r * p + c0 + q) = make_double2(x, y);
            });
        };
        for (int k = 0; k < M.steps; ++k) {
            const bool last = k + 1 == M.steps;
            double acc[2][2][4] = {};
            if (work) dmma_block(acc, G, p, F + c0 * p, p, k8);
            sync();                               // every block has read G: its copies take P
            if (work) {
                dmma_each(acc, [&](int r, int q, double x, double y) {
                    const int i = r0 + r, col = c0 + q;
                    const double2 g = *reinterpret_cast<const double2*>(G + r * p + col);
                    x = (i == col && i < s ? a : 0.0) + b * g.x + c * x;
                    y = (i == col + 1 && i < s ? a : 0.0) + b * g.y + c * y;
                    *reinterpret_cast<double2*>(own + r * p + col) = make_double2(x, y);
                    if (k == 0) *reinterpret_cast<double2*>(Q + r * p + col) = make_double2(x, y);
                });
            }
            exchange();
            double aq[2][2][4] = {};
            if (work && k > 0) dmma_block(aq, Q, p, F + c0 * p, p, k8);
            double ar[2][2][4] = {};
            if (work && !last) dmma_block(ar, G, p, F + c0 * p, p, k8);
            __syncthreads();
            if (work && k > 0) put(Q, aq);
            if (work && !last) put(G, ar);        // R takes G's place
            __syncthreads();
            if (last) break;
            double ag[2][2][4] = {};
            if (work) dmma_block(ag, G, p, F + c0 * p, p, k8);
            sync();                               // every block has read P: its copies take the new G
            if (work) {
                put(G, ag);
                put(own, ag);
            }
            exchange();
        }
        sync();                                   // (no block ends while another copies into it)
    }
    // max |Q|: this block's rows, then all of them
    float qmax = 0.f;
    for (int e = tid; e < nr * s; e += 256)
        if (r0 + e / s < s) qmax = ptx::max_nan(qmax, (float)fabs(Q[(e / s) * pitch + e % s]));
    qmax = block_max(qmax);
    if (!small) {
        if (tid < active) ptx::st_cluster_f32(ptx::cluster_addr(&qmaxes[rank], tid), qmax);
        sync();
        qmax = 0.f;
        for (int k = 0; k < active; ++k) qmax = ptx::max_nan(qmax, qmaxes[k]);
        // (no block ends while another stores into it: all have, before the barrier)
    }
    const int eq = qmax > 0.f && qmax < 3e38f ? ilogbf(qmax) + 1 : 0, eu = max(umax > 0.f ? ilogbf(umax) + 1 : -100, -100);
    const double qs = scalbn(1.0, 8 - eq);
    if (rank == 0 && tid == 0) {
        M.hdr[0] = scalbnf(1.f, 8 - eu);                                      // x = u hdr[0], |x| < 256
        // a NaN or an infinity in u makes the whole of O a NaN
        const bool fine = tr * 0.0 == 0.0 && qmax < 3e38f;
        M.hdr[1] = fine ? (float)(inv * scalbn(1.0, eu - 8 + eq - 8)) : __int_as_float(0x7fc00000);
    }
    // the parts of this block's rows of the 128 (or 256) that the apply pass takes; the last block's go to the end
    constexpr int w = BIG ? 256 : 128, kblocks = w / 64;
    const int rows = small ? w : rank + 1 < active ? nr : w - r0;
    for (int e = tid; e < rows * (w / 8); e += 256) {
        const int r = e / (w / 8), k8i = e - r * (w / 8), row = r0 + r;
        const int jr = row / s, cr = row - jr * s;
        int jk = k8i * 8 / s, ck = k8i * 8 - jk * s;
        __align__(16) __half h[3][8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const double v = jr < M.J && jr == jk ? Q[(small ? cr : r) * pitch + ck] * qs : 0.0;   // (row < s)
            const double x0 = rint(v);
            h[0][k] = __double2half(x0);
            h[1][k] = __double2half(v - x0);
            h[2][k] = __double2half((v - x0) - (double)__half2float(h[1][k]));
            if (++ck == s) { ck = 0; ++jk; }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
            *reinterpret_cast<uint4*>(M.q + muon_q_at(kblocks, row, k8i, i)) = *reinterpret_cast<const uint4*>(h[i]);
    }
}

// --------------------------------------------------------------------------------------------- apply
constexpr int kApplyLoad = 512;                       // threads that load, split and store m: warps 0 .. 15
constexpr int kApplyDone = 256;                       // threads that finish p: warps 16 .. 23
constexpr int kApplyThreads = kApplyLoad + kApplyDone + 32;   // and a warp that issues the products
constexpr int kApplyAhead = 2;                        // tiles whose lines are brought to L2 ahead
constexpr int kApplyQ = 6 * kMuonPlane;               // Q of s <= 128, or two (half, column block) pieces
constexpr int kApplyV = 6 * kMuonPlane;               // two tiles of 128 rows, or one of 256
constexpr int kApplyBlock = 32 * 16 * 4;              // a finishing warp's 32 x 16 block of p, in two places
constexpr int kApplySmem = kApplyQ + kApplyV + (kApplyDone / 32) * 2 * kApplyBlock + 1024;
static_assert(kApplySmem + 1024 <= 232448, "shared memory per CTA");

// O = Q X_0 tile by tile, then p, its bf16 copy and m.  One block per SM over a contiguous run of tiles (all
// matrices' tiles in one list, so that the blocks finish together), with three roles that run side by side:
//   load     g and m of a step (the next step's are on their way), m <- the new m, u in parts to shared memory
//   products Q, kept in shared memory while the matrix lasts, times the tile: 64 columns of O in two
//            accumulators, of two such sets in turn
//   finish   p to shared memory (two blocks ahead), O out of the accumulators onto it, the new p and its copy
// BIG (s > 128): tiles of 256 rows in one place, Q's (row half, column block) pieces streamed from L2.
// 22 bytes per element: 32 adapters of rank 8 to 128 at 4096 -> 14336 (40 M elements) take 279 us for the bytes' 134,
// 65536 x 128 matrices alone (67 M, six products) 336 for 225; odd short sides cost most (their rows start off 16 bytes).  BIG: 160
// for 56.  Bound by the roles sharing an SM: of the 336, 209 are left without p's traffic, 182 without the stores of m
// and the split as well, 157 without the products, and 181 with everything but the traffic.  Loads of a step ahead in
// registers did not help (342).
template <bool BIG>
__global__ void __launch_bounds__(kApplyThreads, 1)
muon_apply_kernel(const MuonMat* __restrict__ mats, int first, int last, int tiles, int* err_flag, uint64_t timeout_ns) {
    constexpr int HALVES = BIG ? 2 : 1, PLACES = BIG ? 1 : 2;
    constexpr int PLANE = HALVES * kMuonPlane;
    constexpr int STEP = BIG ? 16 : 32;                // columns of one step of the loading threads
    constexpr int kIssueWarp = (kApplyLoad + kApplyDone) / 32;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = smem;
    uint8_t* sv = smem + kApplyQ;
    __shared__ __align__(8) uint64_t vfull[2], vfree[2], ofull[2], ofree[2], qfull[2], qfree[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ MuonMat lrec[2], frec[2];               // the loading and the finishing threads' matrices
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int u0 = (int)((int64_t)tiles * blockIdx.x / gridDim.x), u1 = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
    if (tid == 0) {
        for (int k = 0; k < 2; ++k) {
            ptx::mbar_init(&vfull[k], kApplyLoad / 32);
            ptx::mbar_init(&vfree[k], 1);
            ptx::mbar_init(&ofull[k], 1);
            ptx::mbar_init(&ofree[k], kApplyDone / 32);
            ptx::mbar_init(&qfull[k], 1);
            ptx::mbar_init(&qfree[k], 1);
        }
        abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == kIssueWarp) {
        ptx::tmem_alloc<512>(&tmem_slot);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t sq0 = ptx::smem_u32(sq), sv0 = ptx::smem_u32(sv);
    auto wait = [&](uint64_t* bar, uint32_t parity) { ptx::mbar_wait_many(bar, parity, &abort_flag, timeout_ns, err_flag); };
    int mi = muon_find(first, last - 1, u0, [&](int k) { return mats[k].apply0; });

    if (warp < kApplyLoad / 32) {
        // ------------------------------------------------------------ load
        using Tile = MuonTile<kApplyLoad, STEP, HALVES * 128>;
        constexpr int STEPS = kMuonTileL / STEP;
        Tile T;
        auto enter = [&]() {      // makes matrix mi the one whose tiles are loaded
            ptx::named_bar_sync(1, kApplyLoad);
            if (tid < (int)(sizeof(MuonMat) / 8))
                reinterpret_cast<uint64_t*>(&lrec[mi & 1])[tid] = reinterpret_cast<const uint64_t*>(mats + mi)[tid];
            ptx::named_bar_sync(1, kApplyLoad);
        };
        enter();
        T.enter(lrec[mi & 1], tid, true, 0, 64);
        // This thread's 128-byte line of a tile's g, m and p in tile 0 (BIG: and a second one): they are brought to
        // L2 two tiles ahead, so that the loads, whose number in flight registers limit, wait for L2 alone.
        int line = -1, line2 = 0;
        auto enter_line = [&](const MuonMat& M) {
            if (M.tall) {
                line = (tid & 255) * 32 < kMuonTileL * M.J * M.s ? (tid & 255) * 32 : -1;
                line2 = 256 * 32;
            } else {
                const int r = (tid & 255) >> 1, j = M.J > 1 ? r / M.s : 0, c = r - j * M.s;
                line = j < M.J && c < M.s ? c * M.L + j * kMuonTileL + (tid & 1) * 32 : -1;
                line2 = 128 * M.L;
            }
        };
        auto prefetch = [&](const MuonMat& M, int tile) {
            if (tile >= M.tiles || line < 0) return;
            const int total = M.L * M.s, e = line + tile * kMuonTileL * (M.tall ? M.J * M.s : M.J);
#pragma unroll
            for (int k = 0; k < HALVES; ++k) {
                if (e + k * line2 >= total || (k && M.tall && line + line2 >= kMuonTileL * M.s)) break;
                ptx::prefetch_l2(M.g + e + k * line2);
                ptx::prefetch_l2(M.m + e + k * line2);
                ptx::prefetch_l2(M.p + e + k * line2);
            }
        };
        enter_line(lrec[mi & 1]);
        float xs = lrec[mi & 1].hdr[0];
        int unclean = PLACES;     // places that may hold rows of a matrix with more of them
        uint32_t k = 0;           // tiles so far
        for (int u = u0; u < u1; ++u, ++k) {
            const int slot = k % PLACES;
            const uint32_t base = sv0 + slot * 3 * kMuonPlane;
            const MuonMat& C = lrec[mi & 1];
            const int tile = u - C.apply0;
            const bool last_of = tile + 1 == C.tiles;      // the next tile is another matrix's
            const uint64_t mu2 = ptx::f32x2(C.mu, C.mu);
            const bool nesterov = C.nesterov != 0;
            if (tid < 256 && u + kApplyAhead < u1) prefetch(C, tile + kApplyAhead);
#pragma unroll 1
            for (int st = 0; st < STEPS; ++st) {
                float g[Tile::NQ][4], m[Tile::NQ][4];
                T.load(C, tile, st * STEP, g, m);
#pragma unroll
                for (int i = 0; i < Tile::NQ; ++i)
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        const uint64_t gg = ptx::f32x2(g[i][q], g[i][q + 1]);
                        const uint64_t a = ptx::f32x2_fma(mu2, ptx::f32x2(m[i][q], m[i][q + 1]), gg);
                        const float2 b = ptx::f32x2_get(a), c = ptx::f32x2_get(nesterov ? ptx::f32x2_fma(mu2, a, gg) : a);
                        m[i][q] = b.x;
                        m[i][q + 1] = b.y;
                        g[i][q] = c.x;
                        g[i][q + 1] = c.y;
                    }
                T.store(C, C.m, tile, st * STEP, m);
                if (st == 0) {
                    if (k >= PLACES) wait(&vfree[slot], ((k / PLACES) & 1u) ^ 1u);
                    // rows past the matrix's are zero: their products reach no output, but must not be NaN
                    if (unclean > 0) {
                        for (int e = tid; e < 3 * PLANE / 16; e += kApplyLoad)
                            reinterpret_cast<uint4*>(sv + slot * 3 * kMuonPlane)[e] = make_uint4(0, 0, 0, 0);
                        ptx::named_bar_sync(1, kApplyLoad);
                        --unclean;
                    }
                }
                T.template put<1>(C, base, PLANE, st * STEP, xs, g);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&vfull[slot]);
            if (u + 1 < u1 && last_of) {
                unclean = PLACES;
                ++mi;
                enter();
                T.enter(lrec[mi & 1], tid, true, 0, 64);
                enter_line(lrec[mi & 1]);
                xs = lrec[mi & 1].hdr[0];
            }
        }
    } else if (warp < (kApplyLoad + kApplyDone) / 32) {
        // ------------------------------------------------------------ finish
        // A warp has 32 rows m (lanes) x 32 columns l' per half of the tile, in blocks of 32 x 16.  p comes to
        // shared memory as quads of consecutive elements (four per lane), takes scale O row by row, and
        // leaves as quads again.  A quad's cell of a block: tall [column][row], otherwise [row][column], swizzled.
        const int quarter = warp & 3, chalf = ((warp >> 2) & 1) * 32, ft = tid - kApplyLoad;
        constexpr int BLOCKS = 2 * HALVES;
        float* const places = reinterpret_cast<float*>(smem + kApplyQ + kApplyV + (ft >> 5) * 2 * kApplyBlock);
        auto enter = [&](int i) {
            ptx::named_bar_sync(2, kApplyDone);
            if (ft < (int)(sizeof(MuonMat) / 8))
                reinterpret_cast<uint64_t*>(&frec[i & 1])[ft] = reinterpret_cast<const uint64_t*>(mats + i)[ft];
            ptx::named_bar_sync(2, kApplyDone);
        };
        // this lane's quad i of block b of a tile: its first element and how many exist
        struct First {
            int e[4];      // of a tile's first block in tile 0; -1: rows past the matrix's
        };
        auto quad_row = [&](bool tall, int i) { return quarter * 32 + (tall ? (lane & 7) * 4 : 8 * i + (lane >> 2)); };
        auto quad_col = [&](bool tall, int i) { return chalf + (tall ? 4 * i + (lane >> 3) : (lane & 3) * 4); };
        auto first_of = [&](const MuonMat& M) {
            First f;
            const bool tall = M.tall != 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = quad_row(tall, i), y = quad_col(tall, i);
                if (tall) {
                    f.e[i] = r < M.J * M.s ? y * M.J * M.s + r : -1;
                } else {
                    const int j = M.J > 1 ? r / M.s : 0, c = r - j * M.s;
                    f.e[i] = j < M.J && c < M.s ? c * M.L + j * kMuonTileL + y : -1;
                }
            }
            return f;
        };
        auto quad = [&](const MuonMat& M, const First& f, int tile, int b, int i, int& n) {
            const bool tall = M.tall != 0;
            const int y0 = 16 * (b & 1), m0 = (b >> 1) * 128, w = M.J * M.s;
            const int e = f.e[i] + (tall ? (tile * kMuonTileL + y0) * w + m0 : tile * kMuonTileL * M.J + y0 + m0 * M.L);
            n = f.e[i] >= 0 ? 4 : 0;
            if (BIG && b >= 2 && quad_row(tall, i) + 128 >= M.s) n = 0;
            if (tall) {
                n = min(n, w - m0 - quad_row(true, i));
                if (tile + 1 >= M.tiles) n = min(n, M.L * M.s - e);
            } else if (tile + 1 >= M.tiles) {
                const int r = quad_row(false, i), j = M.J > 1 ? r / M.s : 0;
                n = min(n, M.L - (tile * M.J + j) * kMuonTileL - y0 - quad_col(false, i));
            }
            return e;
        };
        auto aligned = [](const MuonMat& M) { return ((M.tall ? M.J * M.s : M.L) & 3) == 0; };
        // tall and not aligned: a lane keeps its row, whose elements lie w apart: the first, and how many exist
        auto column = [&](const MuonMat& M, int tile, int b, int& n) {
            const int w = M.J * M.s, r = (b >> 1) * 128 + quarter * 32 + lane;
            const int e = (tile * kMuonTileL + chalf + 16 * (b & 1)) * w + r;
            n = r < w ? 16 : 0;
            if (n && tile + 1 >= M.tiles) n = max(0, min(16, (M.L * M.s - e + w - 1) / w));
            return e;
        };
        auto cell = [&](bool tall, int i) {
            const int r = 8 * i + (lane >> 2);
            return tall ? (4 * i + (lane >> 3)) * 32 + (lane & 7) * 4 : r * 16 + (((lane & 3) ^ (r >> 1)) & 3) * 4;
        };
        // the cursor of the blocks that are fetched
        int fu = u0, fb = 0, fmi = mi;
        uint32_t fseq = 0;
        enter(mi);
        First ff = first_of(frec[mi & 1]), pf = ff;
        int end = frec[mi & 1].apply0 + frec[mi & 1].tiles;      // of the matrix being finished
        // (The next matrix is entered when its first block is fetched: by then a block of the tile ahead of it has
        // been finished, so a matrix two before it, whose record it replaces, is behind every warp.)
        int fend = end;
        auto fetch = [&]() {
            if (fu < u1) {
                if (fu == fend) {
                    enter(++fmi);
                    ff = first_of(frec[fmi & 1]);
                    fend = frec[fmi & 1].apply0 + frec[fmi & 1].tiles;
                }
                const MuonMat& M = frec[fmi & 1];
                const uint32_t at = ptx::smem_u32(places) + (fseq & 1) * kApplyBlock;
                const bool vec = aligned(M), tall = M.tall != 0;
                if (tall && !vec) {
                    int n;
                    const int e = column(M, fu - M.apply0, fb, n), w = M.J * M.s;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        ptx::cp_async4(at + (i * 32 + lane) * 4, i < n ? M.p + e + i * w : M.p, i < n ? 4 : 0);
                } else
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    int n;
                    const int e = quad(M, ff, fu - M.apply0, fb, i, n);
                    if (vec) {
                        ptx::cp_async16(at + cell(tall, i) * 4, n > 0 ? M.p + e : M.p, n > 0 ? 16 : 0);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            ptx::cp_async4(at + cell(tall, i) * 4 + 4 * q, q < n ? M.p + e + q : M.p, q < n ? 4 : 0);
                    }
                }
                ++fseq;
                if (++fb == BLOCKS) {
                    fb = 0;
                    ++fu;
                }
            }
            ptx::cp_async_commit();
        };
        fetch();
        fetch();
        uint32_t k = 0, seq = 0;
        for (int u = u0; u < u1; ++u, ++k) {
            if (u == end) {
                ++mi;
                pf = first_of(frec[mi & 1]);
                end = frec[mi & 1].apply0 + frec[mi & 1].tiles;
            }
            const MuonMat& M = frec[mi & 1];
            const int tile = u - M.apply0;
            const bool tall = M.tall != 0, vec = aligned(M);
            float* const pp = M.p;
            __nv_bfloat16* const po = M.out;
            const float decay = M.decay, scale = -M.step * M.hdr[1];
            const uint64_t decay2 = ptx::f32x2(decay, decay), scale2 = ptx::f32x2(scale, scale);
#pragma unroll 1
            for (int b = 0; b < BLOCKS; ++b, ++seq) {
                float* const pl = places + (seq & 1) * (kApplyBlock / 4);
                ptx::cp_async_wait<1>();
                if (b == 0) {
                    wait(&ofull[k & 1], (k >> 1) & 1u);
                    ptx::tc_fence_after();
                }
                __syncwarp();
                const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16) + (k & 1) * 256 + (b >> 1) * 128 + chalf +
                                       16 * (b & 1);
                uint32_t hi[16], lo[16];
                ptx::tmem_ld16(t_row, hi);
                ptx::tmem_ld16(t_row + 64, lo);
                ptx::tmem_ld_wait();
                if (b == BLOCKS - 1) {        // the accumulators have been read
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&ofree[k & 1]);
                }
                auto update = [&](int i, float2 p) {
                    const uint64_t o = ptx::f32x2_add(ptx::f32x2(__uint_as_float(hi[i]), __uint_as_float(hi[i + 1])),
                                                      ptx::f32x2(__uint_as_float(lo[i]), __uint_as_float(lo[i + 1])));
                    return ptx::f32x2_get(ptx::f32x2_fma(scale2, o, ptx::f32x2_mul(ptx::f32x2(p.x, p.y), decay2)));
                };
                if (tall && !vec) {
                    int n;
                    const int e = column(M, tile, b, n), w = M.J * M.s;
                    float* const q = pp + e;
                    __nv_bfloat16* const qo = po + e;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 v = update(i, make_float2(pl[i * 32 + lane], pl[(i + 1) * 32 + lane]));
                        if (i < n) {
                            q[i * w] = v.x;
                            if (po) qo[i * w] = __float2bfloat16_rn(v.x);
                        }
                        if (i + 1 < n) {
                            q[(i + 1) * w] = v.y;
                            if (po) qo[(i + 1) * w] = __float2bfloat16_rn(v.y);
                        }
                    }
                    fetch();       // (into this lane's own cells)
                    continue;
                }
                if (tall) {
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 v = update(i, make_float2(pl[i * 32 + lane], pl[(i + 1) * 32 + lane]));
                        pl[i * 32 + lane] = v.x;
                        pl[(i + 1) * 32 + lane] = v.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float4* const q = reinterpret_cast<float4*>(pl + lane * 16 + ((i ^ (lane >> 1)) & 3) * 4);
                        const float4 p = *q;
                        const float2 a = update(4 * i, make_float2(p.x, p.y)), c = update(4 * i + 2, make_float2(p.z, p.w));
                        *q = make_float4(a.x, a.y, c.x, c.y);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    int n;
                    const int e = quad(M, pf, tile, b, i, n);
                    const float4 v = *reinterpret_cast<const float4*>(pl + cell(tall, i));
                    if (vec) {
                        if (n <= 0) continue;
                        *reinterpret_cast<float4*>(pp + e) = v;
                        if (po) {
                            const __nv_bfloat162 va = __floats2bfloat162_rn(v.x, v.y), vb = __floats2bfloat162_rn(v.z, v.w);
                            *reinterpret_cast<uint2*>(po + e) = make_uint2(*reinterpret_cast<const uint32_t*>(&va),
                                                                          *reinterpret_cast<const uint32_t*>(&vb));
                        }
                    } else {
                        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (q < n) {
                                pp[e + q] = x[q];
                                if (po) po[e + q] = __float2bfloat16_rn(x[q]);
                            }
                    }
                }
                __syncwarp();      // (a lane's cells are read by itself last, but its row's by every lane)
                fetch();
            }
        }
        ptx::cp_async_wait<0>();
    } else {
        // ------------------------------------------------------------ products
        // (the whole warp runs this, so that addresses stay in uniform registers; one lane issues)
        const bool one = ptx::elect_one();
        uint32_t k = 0, nq = 0;      // tiles, and Q pieces (BIG) or whole Qs, so far
        int end = -1;                // first tile past the matrix
        bool tall = false;
        int ksteps = 0;
        uint32_t idesc = 0;
        const uint8_t* q = nullptr;
        --mi;
        for (int u = u0; u < u1; ++u, ++k) {
            if (u >= end || k == 0) {
                const MuonMat& M = mats[++mi];
                end = M.apply0 + M.tiles;
                tall = M.tall != 0;
                ksteps = (min(M.J * M.s, HALVES * 128) + 15) / 16;
                idesc = ptx::idesc_f16_f32(128, 64, false, !tall);
                q = M.q;
                if (!BIG) {
                    if (k > 0) wait(&ofull[(k - 1) & 1], ((k - 1) >> 1) & 1u);   // the products that read the last Q
                    if (one) {
                        ptx::mbar_arrive_expect_tx(&qfull[0], kApplyQ);
                        ptx::bulk_load(sq, q, kApplyQ, &qfull[0]);
                    }
                    wait(&qfull[0], nq & 1u);
                    ++nq;
                }
            }
            const int slot = k % PLACES;
            const uint32_t vbase = sv0 + slot * 3 * kMuonPlane;
            const uint32_t d0 = tmem + (k & 1) * 256;
            // K step ks of the tile: its rows 16 ks ..
            const MuonDesc v0 = tall ? ptx::smem_desc_sw128(vbase, 16, 1024) : ptx::smem_desc_sw128(vbase, 8192, 1024);
            auto v_at = [&](int ks) {
                MuonDesc d = v0;
                d.lo += tall ? (uint32_t)((ks >> 2) * 8192 + (ks & 3) * 32) / 16 : (uint32_t)ks * (2048 / 16);
                return d;
            };
            wait(&vfull[slot], (k / PLACES) & 1u);
            if (k >= 2) wait(&ofree[k & 1], ((k >> 1) & 1u) ^ 1u);
            ptx::tc_fence_after();
            if constexpr (!BIG) {
                const MuonDesc q0 = ptx::smem_desc_sw128(sq0, 16, 1024);
                if (one) {
                muon_mma<true>(d0, d0 + 64, q0, v0, kMuonPlane / 16, PLANE / 16, idesc);
#pragma unroll
                for (int ks = 1; ks < 8; ++ks) {
                    if (ks >= ksteps) break;
                    MuonDesc d = q0;
                    d.lo += (uint32_t)((ks >> 2) * 3 * kMuonPlane + (ks & 3) * 32) / 16;
                    muon_mma<false>(d0, d0 + 64, d, v_at(ks), kMuonPlane / 16, PLANE / 16, idesc);
                }
                }
            } else {
                const int kb = (ksteps + 3) / 4, pieces = 2 * kb;
                auto fetch = [&](int c) {   // piece c: row half c / kb, column block c % kb
                    const uint32_t n = nq + c;
                    if (n >= 2) wait(&qfree[n & 1], ((n >> 1) & 1u) ^ 1u);
                    if (!one) return;
                    ptx::mbar_arrive_expect_tx(&qfull[n & 1], 3 * kMuonPlane);
                    ptx::bulk_load(sq + (n & 1) * 3 * kMuonPlane, q + ((int64_t)(c / kb) * 4 + c % kb) * 3 * kMuonPlane,
                                   3 * kMuonPlane, &qfull[n & 1]);
                };
                fetch(0);
                for (int c = 0; c < pieces; ++c) {
                    if (c + 1 < pieces) fetch(c + 1);
                    const uint32_t n = nq + c;
                    wait(&qfull[n & 1], (n >> 1) & 1u);
                    const int h = c / kb, b = c % kb;
                    const uint32_t dh = d0 + h * 128;
                    const MuonDesc q0 = ptx::smem_desc_sw128(sq0 + (n & 1) * 3 * kMuonPlane, 16, 1024);
                    if (one) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        if (b * 4 + ks >= ksteps) break;
                        MuonDesc d = q0;
                        d.lo += ks * 2;
                        if (ks == 0 && b == 0) muon_mma<true>(dh, dh + 64, d, v_at(0), kMuonPlane / 16, PLANE / 16, idesc);
                        else muon_mma<false>(dh, dh + 64, d, v_at(b * 4 + ks), kMuonPlane / 16, PLANE / 16, idesc);
                    }
                    ptx::tc_commit(&qfree[n & 1]);
                    }
                }
                nq += pieces;
            }
            if (one) {
                ptx::tc_commit(&vfree[slot]);
                ptx::tc_commit(&ofull[k & 1]);
            }
            __syncwarp();
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kIssueWarp) ptx::tmem_dealloc<512>(tmem);
}

}  // namespace plora
