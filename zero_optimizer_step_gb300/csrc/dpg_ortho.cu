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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

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

// Returns the new X's sum of squares over the 32 columns (kProdX).
template <int PROD>
__device__ __forceinline__ float finish32(const OrthoArgs& a, const MatDesc& d, int mat, int r, int c0,
                                         float* acc, bool mirror) {
    const OrthoStep& s = a.st;
    const float inv_sx = a.step == 0 ? a.scal[mat].y : s.inv_sx;
    if constexpr (PROD == kProdA) {
        const float k = inv_sx * inv_sx;
        const RoundScale rs(s.sa, r);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float v = acc[j] * k;
            if (c0 + j == r) a.diag_a[d.diag + r] = row_square(a, d, r) * k;
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
// One product of one step, plain form: a CTA per 256 x 256 tile, a thread per
// row, 32 columns at a time.
// ---------------------------------------------------------------------------
template <int PROD>
__global__ void __launch_bounds__(256) k_ortho_product(const __grid_constant__ OrthoArgs a,
                                                      const OrthoTile* tiles) {
    __shared__ float sb[kBlkCols][33];
    pdl_enter();
    const OrthoTile t = tiles[blockIdx.x];
    const MatDesc& d = a.mats[t.mat];
    const int r = t.i * kOrthoTile + int(threadIdx.x);
    const int64_t x = d.x[a.step & 1];
    const int64_t pa = PROD == kProdA ? x : PROD == kProdB ? d.a : d.b;
    const int ca = PROD == kProdA ? d.cbx : d.cba;
    const int kblocks = PROD == kProdA ? d.kn : d.km;
    float sq = 0.0f;
    for (int g = 0; g < kOrthoTile / 32; ++g) {
        const int c0 = t.j * kOrthoTile + g * 32;
        float acc[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[j] = 0.0f;
        for (int kb = 0; kb < kblocks; ++kb) {
            __syncthreads();
            for (int e = threadIdx.x; e < kBlkCols * 32; e += 256) {
                const int k = PROD == kProdX ? e >> 5 : e & 63, c = PROD == kProdX ? e & 31 : e >> 6;
                const int64_t at = PROD == kProdX ? blk_at(x, d.cbx, kb * 64 + k, c0 + c)
                                                  : blk_at(pa, ca, c0 + c, kb * 64 + k);
                sb[k][c] = __half2float(*reinterpret_cast<const __half*>(a.ws + at));
            }
            __syncthreads();
            for (int k8 = 0; k8 < 8; ++k8) {
                const uint4 v = *reinterpret_cast<const uint4*>(a.ws + blk_at(pa, ca, r, kb * 64 + k8 * 8));
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 p = unpack_half2(u[k >> 1]);
                    const float f = (k & 1) ? p.y : p.x;
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[j] = fmaf(f, sb[k8 * 8 + k][j], acc[j]);
                }
            }
        }
        const float s = finish32<PROD>(a, d, t.mat, r, c0, acc, PROD != kProdX && t.j > t.i);
        if (PROD == kProdX) {
            sq = (g & 1) ? sq + s : s;
            if (g & 1) a.rowsq[d.rowsq + int64_t(c0 >> 6) * d.rows_pad + r] = sq;
        }
    }
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
    m.d_tables = t;
    m.ws = static_cast<unsigned char*>(ws);
    m.device = dev;
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
        const OrthoTile* const* t = m.d_tiles;
        st = launch_k(k_ortho_product<kProdA>, unsigned(m.tiles[0].size()), 256, s, who, a, t[0]);
        if (st == DPG_OK)
            st = launch_k(k_ortho_product<kProdB>, unsigned(m.tiles[1].size()), 256, s, who, a, t[1]);
        if (st == DPG_OK)
            st = launch_k(k_ortho_product<kProdX>, unsigned(m.tiles[2].size()), 256, s, who, a, t[2]);
    }
    return st;
}

}  // namespace dpg
