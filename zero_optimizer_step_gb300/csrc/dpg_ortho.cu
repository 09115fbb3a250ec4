// dpg_ortho.cu -- orthogonalisation of the matrices of a plan by Newton-Schulz
// steps (see dpg_orthogonalize in include/dpg.h).
//
// Per matrix, X (m x n, m the shorter side) starts as U / max(||U||_F, eps)
// and each step computes three products
//     A = X X^T            (m x m, symmetric: only tiles j >= i, mirrored)
//     B = b A + c A A^T    (m x m, symmetric)
//     X <- a X + B X       (m x n)
// that is m^2 n + m^3 + 2 m^2 n flops, against 6 bytes per element that must
// move: bound by arithmetic from a few hundred rows up.
//
// Numbers.  The products take fp16 operands and sum in fp32.  bf16 operands
// (8 bits) leave a result 1 % off the exact one, and 70 % off for a matrix of
// rank one, because what rounding adds to X in the directions X lacks is
// multiplied by a (3.4) in every step.  Here
//   * X is a pair hi + lo / 2048 of fp16 numbers (22 bits).  The products use
//     hi; the term a X, the one that carries the amplified directions, uses
//     both, so no rounding of X is amplified.
//   * the diagonals of A and B, which are large where the matrices are close
//     to multiples of the identity, are kept in fp32 apart from the fp16
//     off-diagonal parts F: with A = D + F,
//     A A^T = F F^T + D F + F D + D^2, and B X = F_B X + D_B X.  A's diagonal
//     is summed from the unrounded X (the row sums of squares that the step
//     before leaves).
//   * B lo, which the products leave out, is taken as t D_B lo with
//     t_r = A_rr^2 / (A A^T)_rr per row: 1 for a diagonal A, where D_B lo is
//     all of it, and about 0 in the rows of a low-rank one, where D_B lo and
//     F_B lo cancel in the directions X lacks.
//   * a value is moved by -3/8 .. 3/8 of a unit in the last place, by a
//     pattern over (row + column) mod 4, before it is rounded.  Entries that
//     are all alike (a matrix of equal entries, a constant row) would round
//     alike, and sums over them would carry the whole rounding error (4.5e-3
//     at the end); so moved they round both ways (1.2e-3), at 20 to 40 % more
//     rounding noise elsewhere.
//   * every stored fp16 matrix carries a power-of-two scale that the host
//     derives from the largest value the step can produce, so nothing
//     overflows and small entries stay normal numbers.
// Together 3e-4 to 1.3e-3 of relative Frobenius error over Gaussian, spiked,
// constant and low-rank matrices, below the rounding of the bf16 result itself
// (1.7e-3).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "dpg_host.h"
#include "dpg_ortho.h"

namespace dpg {

constexpr float kLoScale = 2048.0f;
constexpr float kInvLoScale = 1.0f / 2048.0f;

struct OrthoArgs {
    const MatDesc* mats;
    unsigned char* ws;       // blocks
    float* diag_a;           // per row: A_rr
    float* diag_b;           // B_rr
    float* diag_t;           // t_r B_rr
    float* rowsq;            // per 64 columns of X and row: sum of squares (scaled as hi)
    double* part;            // norm partials, one per norm item
    float2* scal;            // per matrix: {power-of-two scale of X_0, 1 / (norm * scale)}
    int32_t* count;          // per matrix: norm items done (zero between launches)
    int32_t* status;         // 0, or the error of the first wait that ran out
    const void* update;
    int32_t f32;             // update holds fp32 (else bf16)
    int32_t step, n_steps;
    double eps;
    OrthoStep st;
    uint16_t* out;           // flat bf16
};

__device__ __forceinline__ float load_update(const OrthoArgs& a, int64_t i) {
    if (a.f32) return __ldg(static_cast<const float*>(a.update) + i);
    return __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(a.update) + i)) << 16);
}

// eight consecutive elements from i; vec: i is a multiple of 8
__device__ __forceinline__ void load_update8(const OrthoArgs& a, int64_t i, bool vec, float* x) {
    if (vec && !a.f32) {
        widen8(ld_grad_u4(static_cast<const uint16_t*>(a.update) + i), x);
    } else if (vec) {
        const F8 v = ld_grad_f8(static_cast<const float*>(a.update) + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = v.v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = load_update(a, i + j);
    }
}

// byte offset of (row, col) in a blocked matrix of `cb` column blocks per row
// of blocks that starts at block `base`
__device__ __forceinline__ int64_t blk_at(int64_t base, int cb, int row, int col) {
    return (base + int64_t(row >> 7) * cb + (col >> 6)) * kBlkBytes + (row & 127) * 128 +
           ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// scale * (1 + the rounding pattern) for columns c = 0, 1, 2, 3 (mod 4) of a
// row; a unit in the last place is 2^-11 to 2^-10 of a value, taken as 1.4 * 2^-11
struct RoundScale {
    float v[4];
    __device__ __forceinline__ RoundScale(float scale, int row) {
        constexpr float q = 1.4f / 16.0f / 2048.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = (row + j) & 3;             // -6, 2, -2, 6 sixteenths
            const float w = k == 0 ? -6.0f : k == 1 ? 2.0f : k == 2 ? -2.0f : 6.0f;
            v[j] = fmaf(scale * q, w, scale);
        }
    }
};

// ---------------------------------------------------------------------------
// Frobenius norms.  One CTA per item (<= 16384 elements of one matrix); sums
// of eight squares in fp32 (in double when that leaves fp32's range), the rest
// in double.  The CTA that finishes a matrix adds its items in item order and
// writes the scale 2^k that puts max(norm, eps) 2^k into [2^14, 2^15) -- every
// |u| 2^k is then below 2^15, and u 2^k is exact for bf16 u -- and
// 1 / (max(norm, eps) 2^k).
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 256;

__device__ __forceinline__ double block_sum(double x, double* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < kNormThreads / 32; ++w) t += sh[w];
    return t;
}

__global__ void __launch_bounds__(kNormThreads) k_ortho_norm(const __grid_constant__ OrthoArgs a,
                                                            const NormItem* items) {
    __shared__ double sh[2][kNormThreads / 32];
    __shared__ int last;
    pdl_enter();
    const NormItem it = items[blockIdx.x];
    const MatDesc& d = a.mats[it.mat];
    const int64_t base = d.off + it.start;
    const bool vec = (base & 7) == 0;
    double acc = 0.0;
    for (int e = int(threadIdx.x) * 8; e < it.count; e += kNormThreads * 8) {
        float x[8];
        if (e + 8 <= it.count) {
            load_update8(a, base + e, vec, x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = e + j < it.count ? load_update(a, base + e + j) : 0.0f;
        }
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
        if (s > 1e-30f && s < 1e30f) {
            acc += double(s);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) acc += double(x[j]) * double(x[j]);
        }
    }
    const double tot = block_sum(acc, sh[0]);
    if (threadIdx.x == 0) {
        a.part[blockIdx.x] = tot;
        __threadfence();
        last = atomicAdd(a.count + it.mat, 1) == d.norm1 - d.norm0 - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    acc = 0.0;
    for (int k = d.norm0 + int(threadIdx.x); k < d.norm1; k += kNormThreads) acc += __ldcg(a.part + k);
    const double sum = block_sum(acc, sh[1]);
    if (threadIdx.x == 0) {
        a.count[it.mat] = 0;
        const double norm = sqrt(sum);
        float2 r;
        if (!(norm <= 1.7e308)) {                       // a NaN or an infinity in the matrix
            r.x = r.y = __int_as_float(0x7FC00000);
        } else {
            const double den = norm > a.eps ? norm : a.eps;
            const int k = 14 - ilogb(den);
            r.x = float(scalbn(1.0, k));
            r.y = float(1.0 / scalbn(den, k));
        }
        a.scal[it.mat] = r;
    }
}

// ---------------------------------------------------------------------------
// U -> X_0 as fp16 blocks (hi and lo), zero in the padding.  One CTA per
// block.  A tall matrix is transposed on the way: lanes then run along X's
// rows, which are contiguous in U.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) k_ortho_load(const __grid_constant__ OrthoArgs a,
                                                   const ConvItem* items) {
    pdl_enter();
    const ConvItem it = items[blockIdx.x];
    const MatDesc& d = a.mats[it.mat];
    const float sc = a.scal[it.mat].x;
    const int64_t blk = int64_t(it.i) * d.cbx + it.j;
    unsigned char* hi = a.ws + (d.x[0] + blk) * kBlkBytes;
    unsigned char* lo = a.ws + (d.lo + blk) * kBlkBytes;
    const bool vec = !d.tall && (d.off & 7) == 0 && (d.n & 7) == 0;
    __shared__ float half_sq[kBlkRows];
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q = int(threadIdx.x) + 256 * i;
        const int row = d.tall ? q & 127 : q >> 3;
        const int ch = d.tall ? 4 * (int(threadIdx.x) >> 7) + i : q & 7;
        const int r = it.i * kBlkRows + row, c = it.j * kBlkCols + ch * 8;
        float x[8];
        if (r < d.m && c + 8 <= d.n && vec) {
            load_update8(a, d.off + int64_t(r) * d.n + c, true, x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = r < d.m && c + j < d.n
                           ? load_update(a, d.off + (d.tall ? int64_t(c + j) * d.m + r
                                                            : int64_t(r) * d.n + c + j))
                           : 0.0f;
        }
        RoundScale rs(1.0f, row);
        if (!a.f32) rs.v[0] = rs.v[1] = rs.v[2] = rs.v[3] = 1.0f;   // bf16 is exact as it is
        uint32_t h[4], l[4];
        if (!d.tall) sq = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = r < d.m && c + 2 * j < d.n ? x[2 * j] * sc : 0.0f;
            const float v = r < d.m && c + 2 * j + 1 < d.n ? x[2 * j + 1] * sc : 0.0f;
            sq = fmaf(u, u, fmaf(v, v, sq));
            h[j] = pack_half2(u * rs.v[2 * j & 3], v * rs.v[(2 * j + 1) & 3]);
            const float2 f = unpack_half2(h[j]);
            l[j] = pack_half2((u - f.x) * kLoScale, (v - f.y) * kLoScale);
        }
        const int at = row * 128 + ((ch ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
        if (!d.tall) {   // a row's eight chunks lie in eight lanes
            sq += __shfl_xor_sync(0xFFFFFFFFu, sq, 1);
            sq += __shfl_xor_sync(0xFFFFFFFFu, sq, 2);
            sq += __shfl_xor_sync(0xFFFFFFFFu, sq, 4);
            if (ch == 0) a.rowsq[d.rowsq + int64_t(it.j) * d.rows_pad + r] = sq;
        }
    }
    if (d.tall) {        // and here in two threads
        if (threadIdx.x >= 128) half_sq[threadIdx.x & 127] = sq;
        __syncthreads();
        if (threadIdx.x < 128)
            a.rowsq[d.rowsq + int64_t(it.j) * d.rows_pad + it.i * kBlkRows + int(threadIdx.x)] =
                sq + half_sq[threadIdx.x];
    }
}

// ---------------------------------------------------------------------------
// What a product does with 32 consecutive sums acc of row r, columns c0 ..
// c0 + 31 (c0 a multiple of 32).  mirror: the tile lies above the diagonal,
// its transpose is written too (a warp's lanes are 32 consecutive rows).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void store_sym(const OrthoArgs& a, const MatDesc& d, int64_t base, int r,
                                          int c0, const float* v, bool mirror) {
    uint32_t h[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) h[j] = pack_half2(v[2 * j], v[2 * j + 1]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(a.ws + blk_at(base, d.cba, r, c0 + 8 * q)) =
            make_uint4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
    if (mirror) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            *reinterpret_cast<uint16_t*>(a.ws + blk_at(base, d.cba, c0 + 2 * j, r)) = uint16_t(h[j]);
            *reinterpret_cast<uint16_t*>(a.ws + blk_at(base, d.cba, c0 + 2 * j + 1, r)) =
                uint16_t(h[j] >> 16);
        }
    }
}

// A_rr from the row's sums of squares
__device__ __forceinline__ float row_square(const OrthoArgs& a, const MatDesc& d, int r) {
    const float* p = a.rowsq + d.rowsq + r;
    float s = 0.0f;
#pragma unroll 8
    for (int k = 0; k < d.kn; ++k) s += p[int64_t(k) * d.rows_pad];
    return s;
}

// diag: the row's sum of squares of X, where the columns hold the diagonal of
// A.  Returns the new X's sum of squares over the 32 columns (kProdX).
template <int PROD>
__device__ __forceinline__ float finish32(const OrthoArgs& a, const MatDesc& d, int mat, int r, int c0,
                                          float* acc, bool mirror, float diag) {
    const OrthoStep& s = a.st;
    const float inv_sx = a.step == 0 ? a.scal[mat].y : s.inv_sx;
    if constexpr (PROD == kProdA) {
        const float k = inv_sx * inv_sx;
        const RoundScale rs(s.sa, r);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float v = acc[j] * k;
            if (c0 + j == r) a.diag_a[d.diag + r] = diag * k;
            acc[j] = c0 + j == r ? 0.0f : v * rs.v[j & 3];
        }
        store_sym(a, d, d.a, r, c0, acc, mirror);
    } else if constexpr (PROD == kProdB) {
        const float dr = a.diag_a[d.diag + r];
        const float k = s.c * s.inv_sa * s.inv_sa;
        const RoundScale rs(s.sb, r);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 f4 = *reinterpret_cast<const uint4*>(a.ws + blk_at(d.a, d.cba, r, c0 + 8 * q));
            const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 p = unpack_half2(f[j >> 1]);
                const float fv = ((j & 1) ? p.y : p.x) * s.inv_sa;
                const int c = c0 + 8 * q + j;
                const float dc = a.diag_a[d.diag + c];
                const float v = fmaf(k, acc[8 * q + j], fmaf(s.c, dr + dc, s.b) * fv);
                // fv is 0 on the diagonal: v is c (F F^T)_rr there
                if (c == r) {
                    const float db = fmaf(fmaf(s.c, dr, s.b), dr, v), d2 = dr * dr;
                    const float aa = fmaf(acc[8 * q + j] * s.inv_sa, s.inv_sa, d2);   // (A A^T)_rr
                    a.diag_b[d.diag + r] = db;
                    a.diag_t[d.diag + r] = aa > 0.0f ? db * (d2 / aa) : 0.0f;
                }
                acc[8 * q + j] = c == r ? 0.0f : v * rs.v[j & 3];
            }
        }
        store_sym(a, d, d.b, r, c0, acc, mirror);
    } else {
        const float k = inv_sx * s.inv_sb;
        const float bx = a.diag_b[d.diag + r] * inv_sx, ax = s.a * inv_sx;
        const float al = fmaf(a.diag_t[d.diag + r], inv_sx, ax) * kInvLoScale, ah = ax + bx;
        float sq = 0.0f;
        const RoundScale rs(s.sx_next, r);
        const bool last = a.step + 1 == a.n_steps;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = c0 + 8 * q;
            const int64_t lo_at = blk_at(d.lo, d.cbx, r, c);
            const uint4 h4 = *reinterpret_cast<const uint4*>(a.ws + blk_at(d.x[a.step & 1], d.cbx, r, c));
            const uint4 l4 = *reinterpret_cast<const uint4*>(a.ws + lo_at);
            const uint32_t h[4] = {h4.x, h4.y, h4.z, h4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
            float x[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = unpack_half2(h[j]), w = unpack_half2(l[j]);
                x[2 * j] = fmaf(ah, u.x, fmaf(al, w.x, k * acc[8 * q + 2 * j]));
                x[2 * j + 1] = fmaf(ah, u.y, fmaf(al, w.y, k * acc[8 * q + 2 * j + 1]));
            }
            if (!last) {
                uint32_t nh[4], nl[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = x[2 * j] * s.sx_next, w = x[2 * j + 1] * s.sx_next;
                    sq = fmaf(u, u, fmaf(w, w, sq));
                    nh[j] = pack_half2(x[2 * j] * rs.v[2 * j & 3], x[2 * j + 1] * rs.v[(2 * j + 1) & 3]);
                    const float2 f = unpack_half2(nh[j]);
                    nl[j] = pack_half2((u - f.x) * kLoScale, (w - f.y) * kLoScale);
                }
                *reinterpret_cast<uint4*>(a.ws + blk_at(d.x[(a.step + 1) & 1], d.cbx, r, c)) =
                    make_uint4(nh[0], nh[1], nh[2], nh[3]);
                *reinterpret_cast<uint4*>(a.ws + lo_at) = make_uint4(nl[0], nl[1], nl[2], nl[3]);
            } else if (r < d.m) {
                if (d.tall) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c + j < d.n)
                            a.out[d.off + int64_t(c + j) * d.m + r] =
                                __bfloat16_as_ushort(__float2bfloat16_rn(x[j]));
                } else {
                    uint16_t* o = a.out + d.off + int64_t(r) * d.n + c;
                    if (c + 8 <= d.n && ((d.off | d.n) & 7) == 0) {
                        *reinterpret_cast<uint4*>(o) = narrow8(x);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c + j < d.n) o[j] = __bfloat16_as_ushort(__float2bfloat16_rn(x[j]));
                    }
                }
            }
        }
        return sq;
    }
    return 0.0f;
}

// ---------------------------------------------------------------------------
// Tensor-core products.  A pair of CTAs on two SMs (a cluster of 2) computes a
// 256 x 256 tile: CTA r holds rows 128 r .. of the left operand and columns
// 128 r .. of the right one, 32 KB per 64-deep stage and SM, and the pair's
// tcgen05.mma (cta_group::2) reads both halves.  A 128 x 256 tile on one SM
// would need 48 KB per stage for the same arithmetic, more than L2 delivers.
// Persistent: every pair takes tiles cluster, cluster + clusters, ...
// Roles per CTA: warp 0 copies (TMA, kStages ahead), warp 1 of CTA 0 issues
// the products into one of two 256-column accumulators, warps 2..9 finish the
// other accumulator meanwhile (warp w reads tensor-memory lanes 32 (w mod 4)).
// ---------------------------------------------------------------------------
constexpr int kStages = 6;
constexpr int kHalfBytes = 128 * 64 * 2;              // one operand of one stage in one CTA
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kEpiWarps = 8;
constexpr int kOrthoThreads = 32 * (2 + kEpiWarps);
constexpr int kOrthoSmem = kStages * kStageBytes + 1024;   // + alignment to 1 KB
constexpr uint64_t kWaitNs = 2000000000ull;           // bound of every wait

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// the address of `addr` (this CTA's shared memory) in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n"
                 " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                 " selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// What the roles of a CTA share.
struct OrthoShared {
    uint64_t full[kStages], empty[kStages], tfull[2], tempty[2];
    uint32_t tmem;
    volatile int abort;     // some wait of this CTA ran out
};

// true once the phase of `parity` completed; false when the bound ran out or
// another role gave up (recorded in *status, the tiles after it are skipped)
__device__ __forceinline__ bool wait_bounded(OrthoShared& sh, uint64_t* bar, uint32_t parity, int32_t* status) {
    const uint32_t at = smem_u32(bar);
    if (try_wait(at, parity)) return true;
    const uint64_t until = global_ns() + kWaitNs;
    while (!try_wait(at, parity)) {
        if (sh.abort) return false;
        if (global_ns() > until) {
            sh.abort = 1;
            atomicCAS(status, 0, DPG_ERR_DEVICE_TIMEOUT);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(0), "r"(row), "r"(bar) : "memory");
}

// Shared-memory descriptors of the 128-byte swizzle: rows of 64 K-values (8
// rows every 1024 bytes), or 64-column groups (8 K-rows every 1024 bytes, the
// next 64 columns 8192 bytes on).
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, bool by_column) {
    return uint64_t(addr >> 4) | (uint64_t(by_column ? 8192 >> 4 : 1) << 16) |
           (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// fp16 operands, fp32 sums, 256 x 256; right operand by rows or by columns
__device__ __forceinline__ uint32_t mma_shape(bool by_column) {
    return (1u << 4) | (by_column ? 1u << 16 : 0u) | (uint32_t(kOrthoTile >> 3) << 17) |
           (uint32_t(kOrthoTile >> 4) << 24);
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
                 :: "r"(d), "l"(a), "l"(b), "r"(shape), "r"(add ? 1u : 0u) : "memory");
}
// arrives at `bar` of both CTAs once every product issued so far is done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(smem_u32(bar)), "h"(uint16_t(3)) : "memory");
}
__device__ __forceinline__ void load_acc32(uint32_t tmem, float* v) {
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
                 " tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                   "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
                   "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
                   "=r"(r[31])
                 : "r"(tmem) : "memory");
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}

// Where the operands of a tile start, in blocks.
struct TileOperands {
    int64_t left, right;    // first block of the left operand's rows; of the right operand
    int right_step;         // kProdX: blocks in a row of X
    int kblocks;
};
__device__ __forceinline__ TileOperands operands_of(const MatDesc& d, int prod, int step, const OrthoTile& t,
                                                    int rank) {
    TileOperands o;
    const int64_t x = d.x[step & 1];
    const int64_t from = prod == kProdA ? x : prod == kProdB ? d.a : d.b;
    const int cb = prod == kProdA ? d.cbx : d.cba;
    o.kblocks = prod == kProdA ? d.kn : d.km;
    o.left = from + int64_t(t.i * 2 + rank) * cb;
    o.right = prod == kProdX ? x + t.j * 4 + rank * 2 : from + int64_t(t.j * 2 + rank) * cb;
    o.right_step = d.cbx;
    return o;
}

__global__ void __cluster_dims__(2) __launch_bounds__(kOrthoThreads, 1)
k_ortho_product(const __grid_constant__ OrthoArgs a, const __grid_constant__ CUtensorMap rows128,
                const __grid_constant__ CUtensorMap rows64, const OrthoTile* tiles, int n_tiles,
                int prod) {
    extern __shared__ unsigned char dyn[];
    __shared__ OrthoShared sh;
    const uint32_t stage0 = (smem_u32(dyn) + 1023u) & ~1023u;
    const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
    const uint32_t rank = cluster_rank();
    const int pairs = int(gridDim.x >> 1), pair = int(blockIdx.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(smem_u32(&sh.full[s])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(smem_u32(&sh.empty[s])) : "memory");
        }
        for (int b = 0; b < 2; ++b) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(smem_u32(&sh.tfull[b])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;"
                         :: "r"(smem_u32(&sh.tempty[b])), "r"(2 * kEpiWarps) : "memory");
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    pdl_enter();
    const uint32_t tmem = sh.tmem;

    if (warp == 0 && lane == 0) {
        // ---- copies ----
        int s = 0;
        uint32_t par = 1;             // the first pass over the ring finds it empty
        bool ok = true;
        for (int t = pair; t < n_tiles && ok; t += pairs) {
            const OrthoTile tile = tiles[t];
            const MatDesc& d = a.mats[tile.mat];
            const TileOperands o = operands_of(d, prod, a.step, tile, int(rank));
            for (int kb = 0; kb < o.kblocks; ++kb) {
                if (!(ok = wait_bounded(sh, &sh.empty[s], par, a.status))) break;
                const uint32_t bar = map_to(smem_u32(&sh.full[s]), 0);
                if (rank == 0)
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                                 :: "r"(smem_u32(&sh.full[s])), "r"(2 * kStageBytes) : "memory");
                const uint32_t dst = stage0 + uint32_t(s) * kStageBytes;
                copy_box(dst, &rows128, int((o.left + kb) * kBlkRows), bar);
                if (prod == kProdX) {
                    const int64_t blk = o.right + int64_t(kb >> 1) * o.right_step;
                    const int row = int(blk * kBlkRows) + (kb & 1) * 64;
                    copy_box(dst + kHalfBytes, &rows64, row, bar);
                    copy_box(dst + kHalfBytes + 8192, &rows64, row + kBlkRows, bar);
                } else {
                    copy_box(dst + kHalfBytes, &rows128, int((o.right + kb) * kBlkRows), bar);
                }
                if (++s == kStages) {
                    s = 0;
                    par ^= 1;
                }
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---- products ----
        const bool by_column = prod == kProdX;
        const uint32_t shape = mma_shape(by_column);
        int s = 0, it = 0;
        uint32_t par = 0;
        bool ok = true;
        for (int t = pair; t < n_tiles && ok; t += pairs, ++it) {
            const MatDesc& d = a.mats[tiles[t].mat];
            const int kblocks = prod == kProdA ? d.kn : d.km;
            const int buf = it & 1;
            if (!(ok = wait_bounded(sh, &sh.tempty[buf], uint32_t((it >> 1) & 1) ^ 1u, a.status))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!(ok = wait_bounded(sh, &sh.full[s], par, a.status))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = stage0 + uint32_t(s) * kStageBytes;
                const uint64_t left = desc_of(at, false), right = desc_of(at + kHalfBytes, by_column);
#pragma unroll
                for (int k = 0; k < 4; ++k)   // 16 deep each
                    mma_pair(tmem + uint32_t(buf) * kOrthoTile, left + 2 * k,
                             right + (by_column ? 128 : 2) * k, shape, (kb | k) != 0);
                commit_pair(&sh.empty[s]);
                if (++s == kStages) {
                    s = 0;
                    par ^= 1;
                }
            }
            if (ok) commit_pair(&sh.tfull[buf]);
        }
    } else if (warp >= 2) {
        // ---- epilogue ----
        const int quad = warp & 3, half = (warp - 2) >> 2;
        int it = 0;
        for (int t = pair; t < n_tiles; t += pairs, ++it) {
            const OrthoTile tile = tiles[t];
            const MatDesc& d = a.mats[tile.mat];
            const int buf = it & 1;
            const int r = tile.i * kOrthoTile + int(rank) * 128 + quad * 32 + lane;
            const bool mirror = prod != kProdX && tile.j > tile.i;
            float diag = 0.0f;
            if (prod == kProdA && tile.i == tile.j && half == int(rank)) diag = row_square(a, d, r);
            const bool ok = wait_bounded(sh, &sh.tfull[buf], uint32_t((it >> 1) & 1), a.status);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            float sq = 0.0f;
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                const int col = half * 128 + g * 32;
                float acc[32];
                load_acc32(tmem + uint32_t(buf) * kOrthoTile + uint32_t(col) + (uint32_t(quad * 32) << 16), acc);
                if (g == 3) {         // the accumulator is free for the tile after next
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                                     :: "r"(map_to(smem_u32(&sh.tempty[buf]), 0)) : "memory");
                }
                const int c0 = tile.j * kOrthoTile + col;
                if (prod == kProdA) {
                    finish32<kProdA>(a, d, tile.mat, r, c0, acc, mirror, diag);
                } else if (prod == kProdB) {
                    finish32<kProdB>(a, d, tile.mat, r, c0, acc, mirror, diag);
                } else {
                    sq += finish32<kProdX>(a, d, tile.mat, r, c0, acc, mirror, diag);
                    if (g & 1) {
                        a.rowsq[d.rowsq + int64_t(c0 >> 6) * d.rows_pad + r] = sq;
                        sq = 0.0f;
                    }
                }
            }
        }
    }
    __syncwarp();
    if (sh.abort) {   // the copies this CTA has in flight land within this time
        const uint64_t until = global_ns() + 2000000ull;
        while (global_ns() < until) {}
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
template <typename T>
static cudaError_t put(unsigned char* base, size_t* at, const std::vector<T>& v, T** out) {
    *out = reinterpret_cast<T*>(base + *at);
    const size_t bytes = v.size() * sizeof(T);
    *at += round256(bytes);
    return bytes ? cudaMemcpy(*out, v.data(), bytes, cudaMemcpyHostToDevice) : cudaSuccess;
}

// The workspace as rows of 64 fp16 values, copied `box_rows` rows at a time
// with no re-arrangement: the blocks are stored as shared memory wants them.
static int encode_map(CUtensorMap* map, void* base, int64_t rows, uint32_t box_rows) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                CUtensorMapFloatOOBfill);
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    DPG_CUDA_TRY(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                                  &found));
    if (found != cudaDriverEntryPointSuccess || !fn)
        return fail(DPG_ERR_CUDA, "matrices upload: the driver has no tensor maps");
    const cuuint64_t dims[2] = {kBlkCols, cuuint64_t(rows)}, strides[1] = {kBlkCols * 2};
    const cuuint32_t box[2] = {kBlkCols, box_rows}, step[2] = {1, 1};
    const CUresult e = reinterpret_cast<Encode>(fn)(
        map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, dims, strides, box, step,
        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return e == CUDA_SUCCESS ? DPG_OK : fail(DPG_ERR_CUDA, "matrices upload: tensor map error %d", int(e));
}

int upload_matrices(Matrices& m) {
    std::lock_guard<std::mutex> g(m.mu);
    int dev = 0;
    DPG_CUDA_TRY(cudaGetDevice(&dev));
    if (m.device >= 0) {
        if (m.device != dev)
            return fail(DPG_ERR_INVALID_ARG, "matrices live on device %d but device %d is current",
                        m.device, dev);
        return DPG_OK;
    }
    const size_t bytes = round256(m.mats.size() * sizeof(MatDesc)) +
                         round256(m.tiles[0].size() * sizeof(OrthoTile)) +
                         round256(m.tiles[1].size() * sizeof(OrthoTile)) +
                         round256(m.tiles[2].size() * sizeof(OrthoTile)) +
                         round256(m.norm_items.size() * sizeof(NormItem)) +
                         round256(m.conv_items.size() * sizeof(ConvItem)) +
                         round256(m.apply_items.size() * sizeof(ApplyItem)) +
                         round256(m.scales.size() * sizeof(double));
    void *ws = nullptr, *tables = nullptr;
    cudaError_t e = cudaMalloc(&tables, bytes ? bytes : 256);
    if (e == cudaSuccess) e = cudaMalloc(&ws, size_t(m.workspace_bytes));
    unsigned char* t = static_cast<unsigned char*>(tables);
    size_t at = 0;
    if (e == cudaSuccess) e = put(t, &at, m.mats, &m.d_mats);
    for (int k = 0; k < 3 && e == cudaSuccess; ++k) e = put(t, &at, m.tiles[k], &m.d_tiles[k]);
    if (e == cudaSuccess) e = put(t, &at, m.norm_items, &m.d_norm_items);
    if (e == cudaSuccess) e = put(t, &at, m.conv_items, &m.d_conv_items);
    if (e == cudaSuccess) e = put(t, &at, m.apply_items, &m.d_apply_items);
    if (e == cudaSuccess) e = put(t, &at, m.scales, &m.d_scales);
    // arrival counters and the status word start at zero
    if (e == cudaSuccess)
        e = cudaMemset(static_cast<unsigned char*>(ws) + m.o_count, 0, size_t(m.workspace_bytes - m.o_count));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        cudaFree(tables);
        cudaFree(ws);
        cudaGetLastError();
        return fail(e == cudaErrorMemoryAllocation ? DPG_ERR_OOM : DPG_ERR_CUDA,
                    "matrices upload: %s", cudaGetErrorString(e));
    }
    int clusters = 0;
    if (m.n_blocks > 0) {
        static_assert(sizeof(CUtensorMap) == sizeof(m.maps[0]), "room for a tensor map");
        CUtensorMap map;
        for (int k = 0; k < 2; ++k) {
            const int st = encode_map(&map, ws, m.n_blocks * kBlkRows, k ? 64 : 128);
            if (st != DPG_OK) {
                cudaFree(tables);
                cudaFree(ws);
                return st;
            }
            std::memcpy(m.maps[k], &map, sizeof map);
        }
        e = cudaFuncSetAttribute(k_ortho_product, cudaFuncAttributeMaxDynamicSharedMemorySize, kOrthoSmem);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kOrthoThreads);
        cfg.dynamicSmemBytes = kOrthoSmem;
        cudaLaunchAttribute pair[1];
        pair[0].id = cudaLaunchAttributeClusterDimension;
        pair[0].val.clusterDim.x = 2;
        pair[0].val.clusterDim.y = pair[0].val.clusterDim.z = 1;
        cfg.attrs = pair;
        cfg.numAttrs = 1;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, k_ortho_product, &cfg);
        if (e != cudaSuccess || clusters < 1) {
            cudaFree(tables);
            cudaFree(ws);
            cudaGetLastError();
            return fail(DPG_ERR_CUDA, "matrices upload: %s", cudaGetErrorString(e));
        }
    }
    m.clusters = clusters;
    m.d_tables = t;
    m.ws = static_cast<unsigned char*>(ws);
    m.device = dev;
    return DPG_OK;
}

int check_matrices(Matrices& m, void* stream) {
    if (m.device < 0) return DPG_OK;   // nothing has run
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int32_t word = 0;
    DPG_CUDA_TRY(cudaMemcpyAsync(&word, m.ws + m.o_status, sizeof word, cudaMemcpyDeviceToHost, s));
    DPG_CUDA_TRY(cudaMemsetAsync(m.ws + m.o_status, 0, sizeof word, s));
    DPG_CUDA_TRY(cudaStreamSynchronize(s));
    if (word != 0)
        return fail(word, "orthogonalisation: a wait on the device ran out; its results are incomplete");
    return DPG_OK;
}

void release_matrices(Matrices& m) {
    std::lock_guard<std::mutex> g(m.mu);
    if (m.device < 0) return;
    int cur = -1;
    const bool have_cur = cudaGetDevice(&cur) == cudaSuccess;
    if (cudaSetDevice(m.device) == cudaSuccess) {
        cudaFree(m.d_tables);
        cudaFree(m.ws);
    }
    if (have_cur) cudaSetDevice(cur);
    cudaGetLastError();
    m.device = -1;
}

static int launch_product(const Matrices& m, const OrthoArgs& a, int prod, cudaStream_t s, const char* who) {
    CUtensorMap map[2];
    std::memcpy(map, m.maps, sizeof map);
    const int n = int(m.tiles[prod].size());
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(2 * (n < m.clusters ? n : m.clusters)));
    cfg.blockDim = dim3(kOrthoThreads);
    cfg.dynamicSmemBytes = kOrthoSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = t_programmatic ? 1 : 0;
    const OrthoTile* tiles = m.d_tiles[prod];
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_ortho_product, a, map[0], map[1], tiles, n, prod);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return fail(DPG_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    }
    return after_launch(who);
}

int ortho_launch(Matrices& m, const void* update, int32_t update_dtype, const dpg_muon_hparams* hp,
                 void* out, void* stream, const char* who) {
    OrthoStep steps[DPG_MAX_NS_STEPS];
    int st = ortho_steps(hp, steps, who);
    if (st != DPG_OK || m.mats.empty()) return st;
    OrthoArgs a{};
    a.mats = m.d_mats;
    a.ws = m.ws;
    a.diag_a = reinterpret_cast<float*>(m.ws + m.o_diag);
    a.diag_b = a.diag_a + m.n_diag;
    a.diag_t = a.diag_b + m.n_diag;
    a.rowsq = reinterpret_cast<float*>(m.ws + m.o_rowsq);
    a.part = reinterpret_cast<double*>(m.ws + m.o_part);
    a.scal = reinterpret_cast<float2*>(m.ws + m.o_scal);
    a.count = reinterpret_cast<int32_t*>(m.ws + m.o_count);
    a.status = reinterpret_cast<int32_t*>(m.ws + m.o_status);
    a.update = update;
    a.f32 = update_dtype == DPG_F32;
    a.n_steps = hp->n_steps;
    a.eps = hp->eps;
    a.out = static_cast<uint16_t*>(out);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = launch_k(k_ortho_norm, unsigned(m.norm_items.size()), kNormThreads, s, who, a,
                  static_cast<const NormItem*>(m.d_norm_items));
    if (st == DPG_OK)
        st = launch_k(k_ortho_load, unsigned(m.conv_items.size()), 256, s, who, a,
                      static_cast<const ConvItem*>(m.d_conv_items));
    for (int k = 0; k < hp->n_steps && st == DPG_OK; ++k) {
        a.step = k;
        a.st = steps[k];
        for (int prod = 0; prod < 3 && st == DPG_OK; ++prod) st = launch_product(m, a, prod, s, who);
    }
    return st;
}

}  // namespace dpg
