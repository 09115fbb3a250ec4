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
//     both, so the rounding of X itself is not amplified.
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
// Together 3e-4 to 1.3e-3 of relative Frobenius error after five default steps
// over Gaussian, spiked, constant and low-rank matrices, below the rounding of
// the bf16 result itself (1.7e-3); 1.9e-3 for rank m / 2 and 2.7e-3 where every
// row stands twice, whose diagonals in fp32 and off-diagonal parts in fp16 do
// not cancel exactly.
//
// What they leave grows with the a of every step to come, and is more where few
// rows average it.  In the early steps of schedules that multiply it by more
// (both_halves), and in all steps for up to 128 rows, A and B are pairs of fp16 numbers too and the products take hi hi + lo hi + hi lo, as three sums
// in one accumulator; t is 1.  That leaves 5e-6 (256 x 512) to 2e-5 (512 x 1024)
// at full rank, 1e-4 at low rank, as binary32 does, for two to three times the
// time.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <exception>

#include "dpg_async.cuh"
#include "dpg_host.h"
#include "dpg_ortho.h"

namespace dpg {

constexpr float kInvLoScale = 1.0f / kLoScale;

struct OrthoArgs {
    const MatDesc* mats;
    unsigned char* ws;       // blocks
    unsigned char* ws_low;   // blocks of the second workspace
    int32_t both_steps;      // the first so many steps take both halves
    float* diag_a;           // per row: A_rr
    float* diag_b;           // B_rr
    float* diag_t;           // t_r B_rr
    float* rowsq;            // per 64 columns of X and row: sum of squares (scaled as hi)
    double* part;            // norm partials, one per norm item
    float2* scal;            // per matrix: {power-of-two scale of X_0, 1 / (norm * scale)}
    int32_t* count;          // per matrix: norm items done (zero between launches)
    int32_t* status;         // 0, or the error of the first wait that ran out
    uint64_t wait_ns;        // bound of every wait
    int64_t skip;            // test only: the first CTA does not fetch this stage of its operands (-1: none)
    int32_t* done;           // per matrix and product: CTA tiles finished in this call
    int32_t* join;           // per group of parts, CTA and finishing warp: parts left in this call
    const OrthoTile* queue;  // tiles of a step, pair p's at [queue_first[p], queue_first[p + 1])
    const int32_t* queue_first;
    const void* update;
    int32_t f32;             // update holds fp32 (else bf16)
    int32_t n_steps;
    double eps;
    float eps_frac;          // eps = eps_frac 2^eps_exp, eps_frac in [1, 2)
    int32_t eps_exp;
    uint16_t* out;           // flat bf16
    OrthoStep st[DPG_MAX_NS_STEPS];
};

template <bool F32>
__device__ __forceinline__ float load_update(const OrthoArgs& a, int64_t i) {
    if (F32) return __ldg(static_cast<const float*>(a.update) + i);
    return __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(a.update) + i)) << 16);
}

// Eight consecutive elements as they are in memory (loads in flight hold four
// registers for bf16 so, not eight).
template <bool F32>
struct Raw8;
template <>
struct Raw8<true> {
    F8 v;
    __device__ __forceinline__ void load(const OrthoArgs& a, int64_t i) {
        v = ld_grad_f8(static_cast<const float*>(a.update) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) v.v[j] = 0.0f;
    }
    // the first `n` elements from i on, singly; zeros after them
    __device__ __forceinline__ void load_some(const OrthoArgs& a, int64_t i, int n) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v.v[j] = j < n ? __ldg(static_cast<const float*>(a.update) + i + j) : 0.0f;
    }
    __device__ __forceinline__ void widen(float* x) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = v.v[j];
    }
};
template <>
struct Raw8<false> {
    uint4 v;
    __device__ __forceinline__ void load(const OrthoArgs& a, int64_t i) {
        v = ld_grad_u4(static_cast<const uint16_t*>(a.update) + i);
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load_some(const OrthoArgs& a, int64_t i, int n) {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = j < n ? __ldg(static_cast<const uint16_t*>(a.update) + i + j) : 0;
        v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    __device__ __forceinline__ void widen(float* x) const { widen8(v, x); }
};

__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

__device__ __forceinline__ uint64_t unpack_pair(uint32_t h) {
    const float2 f = unpack_half2(h);
    return pair_of(f.x, f.y);
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t p) {
    const float2 f = halves_of(p);
    return pack_half2(f.x, f.y);
}

// scale * (1 + the rounding pattern) for columns c = 0, 1, 2, 3 (mod 4) of a
// row; a unit in the last place is 2^-11 to 2^-10 of a value, taken as 1.4 * 2^-11
struct RoundScale {
    float v[4];
    __device__ __forceinline__ RoundScale(float scale, int row) {
        constexpr float q = 1.4f / 16.0f / 2048.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // -6, 2, -2, 6 sixteenths for (row + j) mod 4 = 0 .. 3; as a chain of selections it
            // became a table in constant memory, 750 cycles for every use
            const int k = row + j;
            const float w = float((k & 1) * 8 + (k & 2) * 2 - 6);
            v[j] = fmaf(scale * q, w, scale);
        }
    }
    // for columns 2 j, 2 j + 1
    __device__ __forceinline__ uint64_t pair(int j) const { return pair_of(v[2 * j & 3], v[(2 * j + 1) & 3]); }
};

// ---------------------------------------------------------------------------
// Frobenius norms.  One CTA per item (16384 elements of one matrix or up to
// eight times as many, see lay_out): sums
// of squares in fp32, item sums and everything after in double.  Vectors whose
// squares leave fp32's range (|u| beyond about 1e15, below 1e-15) are squared
// in double: this GPU's binary64 rate is a few operations per SM and cycle, so
// a binary64 sum per vector, with its conversions and its reduction, took four
// times as long as the loads.  The CTA that finishes a matrix adds its items
// in item order and writes the scale 2^k that puts max(norm, eps) 2^k into
// [2^14, 2^15) -- every |u| 2^k is then below 2^15, and u 2^k is exact for
// bf16 u -- and 1 / (max(norm, eps) 2^k).  Reads each element once: 134 MB
// (a 1B model's layer) in 26 us, 5.2 TB/s; 19 MB in 10.5 us, where the launch,
// one memory latency and the last CTA's sum are half.
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 256;

// sum of f over the CTA in fp32 plus sum of w (mostly zero everywhere) in double
__device__ __forceinline__ double block_sum(float f, double w, double* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xFFFFFFFFu, f, o);
    if (__any_sync(0xFFFFFFFFu, w != 0.0)) {     // a NaN differs from zero too
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
    }
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = double(f) + w;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int k = 0; k < kNormThreads / 32; ++k) t += sh[k];
    return t;                                    // in thread 0
}

// adds eight squares to f, or to w where fp32 cannot hold them
__device__ __forceinline__ void square8(const float* x, float& f, double& w) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
    if (s > 1e-30f && s < 1e30f) {
        f += s;
        return;
    }
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
    if (s == 0.0f && top == 0.0f) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) w += double(x[j]) * double(x[j]);
}

template <bool F32>
__global__ void __launch_bounds__(kNormThreads) k_ortho_norm(const __grid_constant__ OrthoArgs a,
                                                            const NormItem* items) {
    __shared__ double sh[kNormThreads / 32];
    __shared__ int last;
    pdl_enter();
    const NormItem it = items[blockIdx.x];
    const MatDesc& d = a.mats[it.mat];
    const int64_t base = d.off + it.start;
    constexpr int kFly = F32 ? 4 : 8;   // vectors in flight per thread
    static_assert(kNormChunk % (kFly * kNormThreads * 8) == 0, "whole batches");
    float f = 0.0f;
    double w = 0.0;
    if (it.count % kNormChunk == 0 && (base & 7) == 0) {
        const int per = it.count / (kNormThreads * 8);
#pragma unroll 1
        for (int k = 0; k < per; k += kFly) {
            Raw8<F32> raw[kFly];
#pragma unroll
            for (int u = 0; u < kFly; ++u)
                raw[u].load(a, base + (int64_t(k + u) * kNormThreads + threadIdx.x) * 8);
#pragma unroll
            for (int u = 0; u < kFly; ++u) {
                float x[8];
                raw[u].widen(x);
                square8(x, f, w);
            }
        }
    } else {
        for (int e = int(threadIdx.x) * 8; e < it.count; e += kNormThreads * 8) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = e + j < it.count ? load_update<F32>(a, base + e + j) : 0.0f;
            square8(x, f, w);
        }
    }
    const double tot = block_sum(f, w, sh);
    if (threadIdx.x == 0) {
        a.part[blockIdx.x] = tot;
        __threadfence();
        last = atomicAdd(a.count + it.mat, 1) == d.norm1 - d.norm0 - 1;
    }
    __syncthreads();
    if (!last || threadIdx.x >= 32) return;
    __threadfence();
    double sum = 0.0;
    for (int k = d.norm0 + int(threadIdx.x); k < d.norm1; k += 32) sum += __ldcg(a.part + k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (threadIdx.x == 0) {
        a.count[it.mat] = 0;
        float2 r;
        if (!(sum <= 1.7e308)) {                        // a NaN or an infinity in the matrix
            r.x = r.y = __int_as_float(0x7FC00000);
        } else {
            // sum = f 4^e, f in [1, 4): the norm is sqrt(f) 2^e (binary64 square roots and
            // quotients cost microseconds here); below eps, eps = g 2^e instead
            const double low = a.eps * a.eps;
            const int e2 = int((__double_as_longlong(sum) >> 52) & 0x7FF) - 1023, e = e2 >> 1;
            const bool small = sum < low;
            const double unit = __longlong_as_double((long long)(1023 - 2 * e) << 52);   // 4^-e
            const int k = 14 - (small ? a.eps_exp : e);
            const float den = small ? a.eps_frac : sqrtf(float(sum * unit));             // in [1, 2)
            r.x = ldexpf(1.0f, k);
            r.y = (1.0f / 16384.0f) / den;
        }
        a.scal[it.mat] = r;
    }
}

// ---------------------------------------------------------------------------
// U -> X_0 as fp16 blocks (hi and lo), zero in the padding, and the row sums
// of squares.  One CTA per two neighbouring blocks (128 x 128).  Moves 4 bytes
// per element of a bf16 update (lo, all zero, is left out), 8 of an fp32 one.
// A tall matrix is transposed through shared memory: 16-byte loads along U's
// rows; 2-byte loads along X's rows took four times as long as the copy.
// 134 MB read and 134 MB written in 57 us (4.7 TB/s), 34 + 34 MB in 14 us.
// ---------------------------------------------------------------------------
constexpr int kLoadPitch = 136;   // fp16 values of a transposed row: 16-byte rows, banks 4 words apart
constexpr int kLoadSmem = kBlkRows * kLoadPitch * 2;

__device__ __forceinline__ void split16(float u, float rounded, float scale, uint16_t& hi, uint16_t& lo) {
    const __half h = __float2half_rn(rounded);
    hi = __half_as_ushort(h);
    lo = __half_as_ushort(__float2half_rn((u - __half2float(h)) * scale));
}

// How many of the call's steps take both halves of a matrix's operands.
__device__ __forceinline__ int both_steps_of(const OrthoArgs& a, const MatDesc& d) {
    return d.both ? a.n_steps : a.both_steps;
}
// What X's low half is multiplied by as step `step` reads it: 2048 where only
// its own sums do, 1 where products read it beside the high half.
__device__ __forceinline__ float lo_scale_of(const OrthoArgs& a, const MatDesc& d, int step) {
    return step < both_steps_of(a, d) ? 1.0f : kLoScale;
}

template <bool F32, bool TALL>
__device__ __forceinline__ void load_blocks(const OrthoArgs& a, const MatDesc& d, const ConvItem& it,
                                            uint16_t* sm) {
    const float lo_scale = lo_scale_of(a, d, 0), inv_lo_scale = 1.0f / lo_scale;
    const float sc = a.scal[it.mat].x;
    const int64_t blk = int64_t(it.i) * d.cbx + it.j * 2;
    unsigned char* hi = a.ws + (d.x[0] + blk) * kBlkBytes;
    unsigned char* lo = a.ws + (d.lo + blk) * kBlkBytes;
    const int r0 = it.i * kBlkRows, c0 = it.j * 2 * kBlkCols, m = d.m, n = d.n;
    const int64_t off = d.off;
    uint16_t* sm_lo = sm + kBlkRows * kLoadPitch;
    if (TALL) {
        // row c of U holds X's column c: X[r][c] = U[c m + r]
        const bool vec = ((off | m) & 7) == 0;
        if (vec) {
            Raw8<F32> raw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {   // 16 columns by two vectors of 8 rows per warp
                const int q = i * 8 + int(threadIdx.x >> 5);
                const int c = c0 + (q & 7) * 16 + (int(threadIdx.x) & 15);
                const int r = r0 + ((q >> 3) * 2 + ((int(threadIdx.x) >> 4) & 1)) * 8;
                if (c < n && r < m)
                    raw[i].load(a, off + int64_t(c) * m + r);
                else
                    raw[i].zero();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int q = i * 8 + int(threadIdx.x >> 5);
                const int c = (q & 7) * 16 + (int(threadIdx.x) & 15);
                const int r = ((q >> 3) * 2 + ((int(threadIdx.x) >> 4) & 1)) * 8;
                const bool in = c0 + c < n && r0 + r < m;
                float x[8];
                raw[i].widen(x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = in ? x[j] * sc : 0.0f;
                    uint16_t h, l;
                    split16(u, F32 ? u * RoundScale(1.0f, r + j + c).v[0] : u, lo_scale, h, l);
                    sm[(r + j) * kLoadPitch + c] = h;
                    if (F32) sm_lo[(r + j) * kLoadPitch + c] = l;
                }
            }
        } else {
            for (int e = int(threadIdx.x); e < 128 * 128; e += 256) {
                const int c = e >> 7, r = e & 127;
                const float u = c0 + c < n && r0 + r < m
                                    ? load_update<F32>(a, off + int64_t(c0 + c) * m + r0 + r) * sc : 0.0f;
                uint16_t h, l;
                split16(u, F32 ? u * RoundScale(1.0f, r + c).v[0] : u, lo_scale, h, l);
                sm[r * kLoadPitch + c] = h;
                if (F32) sm_lo[r * kLoadPitch + c] = l;
            }
        }
        __syncthreads();
    }
    const bool vec = !TALL && ((off | n) & 7) == 0;
    Raw8<F32> raw[8];
    if (!TALL) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // sixteen lanes hold a row's sixteen chunks of 8
            const int r = r0 + 16 * i + (int(threadIdx.x) >> 4), c = c0 + (int(threadIdx.x) & 15) * 8;
            if (vec && r < m && c < n)
                raw[i].load(a, off + int64_t(r) * n + c);
            else
                raw[i].load_some(a, off + int64_t(r) * n + c, r < m ? n - c : 0);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 16 * i + (int(threadIdx.x) >> 4), ch = int(threadIdx.x) & 15;
        uint4 h4, l4 = make_uint4(0, 0, 0, 0);
        float sq = 0.0f;
        if (TALL) {
            h4 = *reinterpret_cast<const uint4*>(sm + row * kLoadPitch + ch * 8);
            if (F32) l4 = *reinterpret_cast<const uint4*>(sm_lo + row * kLoadPitch + ch * 8);
            const uint32_t h[4] = {h4.x, h4.y, h4.z, h4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack_half2(h[j]), g = unpack_half2(l[j]);
                const float u = fmaf(g.x, inv_lo_scale, f.x), v = fmaf(g.y, inv_lo_scale, f.y);
                sq = fmaf(u, u, fmaf(v, v, sq));
            }
        } else {
            const int r = r0 + row, c = c0 + ch * 8;
            const RoundScale rs(1.0f, row);
            float x[8];
            raw[i].widen(x);
            uint32_t h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (sc is a NaN for a matrix that is not finite: padding stays zero)
                const float u = r < m && c + 2 * j < n ? x[2 * j] * sc : 0.0f;
                const float v = r < m && c + 2 * j + 1 < n ? x[2 * j + 1] * sc : 0.0f;
                sq = fmaf(u, u, fmaf(v, v, sq));
                // a scaled bf16 value is an fp16 value: nothing to round, lo is 0
                h[j] = F32 ? pack_half2(u * rs.v[2 * j & 3], v * rs.v[(2 * j + 1) & 3]) : pack_half2(u, v);
                const float2 f = unpack_half2(h[j]);
                l[j] = pack_half2((u - f.x) * lo_scale, (v - f.y) * lo_scale);
            }
            h4 = make_uint4(h[0], h[1], h[2], h[3]);
            l4 = make_uint4(l[0], l[1], l[2], l[3]);
        }
        const int64_t at = (ch >> 3) * kBlkBytes + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(hi + at) = h4;
        if (F32) *reinterpret_cast<uint4*>(lo + at) = l4;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
        if ((ch & 7) == 0) a.rowsq[d.rowsq + int64_t(it.j * 2 + (ch >> 3)) * d.rows_pad + r0 + row] = sq;
    }
}

template <bool F32>
__global__ void __launch_bounds__(256) k_ortho_load(const __grid_constant__ OrthoArgs a, const ConvItem* items) {
    extern __shared__ __align__(16) uint16_t load_sm[];   // kLoadSmem, twice for fp32
    pdl_enter();
    const ConvItem it = items[blockIdx.x];
    const MatDesc& d = a.mats[it.mat];
    if (it.i == 0 && it.j == 0) {
        if (threadIdx.x < 3) a.done[3 * it.mat + int(threadIdx.x)] = 0;
        for (int k = int(threadIdx.x); k < 16 * d.groups; k += 256) a.join[int64_t(d.group0) * 16 + k] = 0;
    }
    if (d.tall)
        load_blocks<F32, true>(a, d, it, load_sm);
    else
        load_blocks<F32, false>(a, d, it, load_sm);
}

// ---------------------------------------------------------------------------
// The steps.  One persistent kernel runs every product of every step.  A pair
// of CTAs on two SMs (a cluster of 2) computes 256 x 256 tiles: CTA r holds
// rows 128 r .. of the left operand and columns 128 r .. of the right one, 32
// KB per 64-deep stage and SM, and the pair's tcgen05.mma (cta_group::2) reads
// both halves.  A 128 x 256 tile on one SM would need 48 KB per stage for the
// same arithmetic.
//
// Two pairs that share a left operand by multicast (clusters of four, 24 KB per
// stage and SM) were 3 % slower on every list tried, 144 SMs in use instead of
// 152: what limits large matrices is the power cap, not L2.
//
// Measured, whole calls: 218M elements of an 8B model's layer 11.2 to 11.6 ms, 1.29
// PFLOP/s of m^2 n + m^3 + 2 m^2 n flops per step (the 1.37 kW cap holds the
// clock near 1.45 GHz, where a plain fp16 library product of 8192^3 runs at
// 1.55 to 1.65); a 1B model's layer 1.79 to 1.99 ms, 1.2 PFLOP/s, of which norm
// and load are 0.08; eight GPT-2-small attention matrices 0.233 ms, 0.54 PFLOP/s.
// There, as for every list whose products last one or two rounds of tiles, the
// way from product to product bounds it: finish 2 to 3 us, stores and their
// count 1 us, operands 1 us, fifteen times.
//
// Every pair works through a queue of tiles that the host laid out once
// (balanced by cost), the same in every step: A tiles, B tiles, X tiles of all
// matrices.  A tile starts when its matrix's tiles of the product before are
// done (a counter per matrix and product in device memory), so matrices
// overlap at the ends of their products and a step needs no launch.  Queues
// follow one global order and all pairs are resident (cooperative launch), so
// the oldest unfinished tile can always run.
//
// Roles per CTA:
//   warp 0       copies operands (TMA, kStages ahead)
//   warp 1       of CTA 0: issues the products into one of two accumulators
//   warps 2..9   finish the other accumulator, 64 columns at a time in one of
//                two shared-memory slots (warp w: tensor-memory lanes 32 (w mod
//                4), 32 of the 64 columns; four warps to each slot side by side
//                were a third slower, the slots then come free together)
//   warps 10, 11 fill the slots with what the finish needs (hi and lo of X, or
//                the tile of A) and write them out, as whole contiguous blocks
//                (two warps: the next tile's first blocks come in while this
//                tile's last ones are on their way to memory).  Row-wise
//                16-byte accesses from the finishing warps themselves took 22
//                to 29 us per tile, four times the product.
// ---------------------------------------------------------------------------
constexpr int kStages = 5;
constexpr int kHalfBytes = 128 * 64 * 2;              // one operand of one stage in one CTA
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kSlots = 2;
constexpr int kSlotBytes = 2 * int(kBlkBytes);        // hi | lo, or the tile | its transpose
constexpr int kEpiWarps = 8;
constexpr int kFillWarp = 2 + kEpiWarps, kStoreWarp = kFillWarp + 1;
constexpr int kOrthoThreads = 32 * (kStoreWarp + 1);

__device__ __forceinline__ int32_t load_acquire(const int32_t* p) {
    int32_t v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// What the roles of a CTA share.
struct OrthoShared {
    uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], in_full[kSlots], out_ready[kSlots],
        slot_free[kSlots], tile_ready;
    alignas(16) float cols[kEpiWarps][32];   // a finishing warp's 32 values of A's diagonal (16-byte loads)
    uint32_t tmem;
    volatile int abort;     // some wait of this CTA ran out, or of another one
};
static_assert(offsetof(OrthoShared, cols) % 16 == 0 && (kStages * kStageBytes + kSlots * kSlotBytes) % 16 == 0,
              "16-byte shared loads");
constexpr int kOrthoSmem = kStages * kStageBytes + kSlots * kSlotBytes + int(sizeof(OrthoShared));
static_assert(kOrthoSmem <= 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ void give_up(OrthoShared& sh, int32_t* status) {
    sh.abort = 1;
    atomicCAS(status, 0, DPG_ERR_DEVICE_TIMEOUT);
}

// true once the phase of `parity` completed; false when the bound ran out or
// another role gave up (recorded in *status, the tiles after it are skipped)
__device__ __forceinline__ bool wait_bounded(OrthoShared& sh, uint64_t* bar, uint32_t parity, const OrthoArgs& a) {
    const uint32_t at = smem_u32(bar);
    if (try_wait(at, parity)) return true;
    const uint64_t until = global_ns() + a.wait_ns;
    while (!try_wait(at, parity)) {
        if (sh.abort) return false;
        if (global_ns() > until) {
            give_up(sh, a.status);
            return false;
        }
    }
    return true;
}

// The same for a counter in device memory that other CTAs raise to `target`.
// What they wrote before is visible afterwards, to copies too.
__device__ __forceinline__ bool wait_count(OrthoShared& sh, const int32_t* count, int32_t target,
                                           const OrthoArgs& a) {
    if (target > 0 && load_acquire(count) < target) {
        const uint64_t until = global_ns() + a.wait_ns;
        uint32_t polls = 0;
        while (load_acquire(count) < target) {
            if (sh.abort) return false;
            // (every sixteenth time: a second load in every round doubled the delay)
            if ((++polls & 15) == 0 && (load_acquire(a.status) != 0 || global_ns() > until)) {
                give_up(sh, a.status);
                return false;
            }
        }
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    return true;
}

// rows of 128 bytes from `row` on into this CTA's shared memory; `bar` may be
// the other CTA's
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(0), "r"(row), "r"(bar) : "memory");
}
__device__ __forceinline__ void copy_in(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copy_out(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                 :: "l"(dst), "r"(src), "r"(bytes) : "memory");
}

// Shared-memory descriptors of the 128-byte swizzle: rows of 64 K-values (8
// rows every 1024 bytes), or 64-column groups (8 K-rows every 1024 bytes, the
// next 64 columns 8192 bytes on).  The upper bits of a shared address name the
// CTA of the cluster and stay out of the descriptor.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, bool by_column) {
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(by_column ? 8192 >> 4 : 1) << 16) |
           (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// fp16 operands, fp32 sums, 256 x width; right operand by rows or by columns
__device__ __forceinline__ uint32_t mma_shape(bool by_column, int width) {
    return (1u << 4) | (by_column ? 1u << 16 : 0u) | (uint32_t(width >> 3) << 17) |
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
__device__ __forceinline__ void store_acc32(uint32_t tmem, const float* v) {
    uint32_t r[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(v[j]);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n"
                 " tcgen05.wait::st.sync.aligned;"
                 :: "r"(tmem), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                    "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
                    "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
                    "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                    "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
                    "r"(r[31])
                 : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t x) {
    asm volatile("st.shared.u16 [%0], %1;" :: "r"(at), "h"(uint16_t(x)) : "memory");
}

// ---------------------------------------------------------------------------
// What a product does with 32 consecutive sums acc: row `row` (0..127) of the
// CTA's rows, columns 32 h .. of the 64 in slot `slot`; r and c0 are the row
// and first column in the matrix.  All of a slot's values are loaded before
// the first is stored, and the arithmetic is in pairs: a warp's time here is
// issue slots and shared-memory latency, and there are only two warps per
// scheduler to hide it.
// ---------------------------------------------------------------------------
// writes 32 fp16 values into the block at `slot`, and transposed behind it:
// two groups of 64 rows (the columns) by 64 columns (the rows)
__device__ __forceinline__ void put_sym(uint32_t slot, int row, int h, const uint32_t* x, bool mirror) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        sts128(slot + row * 128 + (((4 * h + q) ^ (row & 7)) << 4), x[4 * q], x[4 * q + 1], x[4 * q + 2],
               x[4 * q + 3]);
    if (mirror) {
        const uint32_t base = slot + uint32_t(kBlkBytes) + uint32_t(row >> 6) * 8192 + uint32_t(row & 7) * 2 +
                              uint32_t(h) * 32 * 128;
        const uint32_t ch = uint32_t(row & 63) >> 3;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            sts16(base + j * 128 + ((ch ^ (j & 7)) << 4), (j & 1) ? x[j >> 1] >> 16 : x[j >> 1] & 0xFFFFu);
    }
}

// the packed values x[16] with the one of column `lane` set to zero
__device__ __forceinline__ void clear_diagonal(uint32_t* x, int lane) {
    const uint32_t keep = (lane & 1) ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] &= j == (lane >> 1) ? keep : 0xFFFFFFFFu;
}

// A_rr from the row's sums of squares: sixteen loads at a time, or their
// latencies add up to more than the product takes
__device__ __forceinline__ float row_square(const OrthoArgs& a, const MatDesc& d, int r) {
    const float* p = a.rowsq + d.rowsq + r;
    const int n = d.cbx;
    const int64_t pitch = d.rows_pad;
    float s = 0.0f;
    for (int k = 0; k < n; k += 16) {
        float v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) v[u] = k + u < n ? __ldcg(p + int64_t(k + u) * pitch) : 0.0f;
#pragma unroll
        for (int u = 0; u < 16; ++u) s += v[u];
    }
    return s;
}

// diag: the row's sum of squares of X where the columns hold A's diagonal
__device__ __forceinline__ void finish_a(const OrthoArgs& a, const OrthoStep& s, int64_t diag_at, float inv_sx,
                                         uint32_t slot, int row, int h, int r, int c0, const float* acc,
                                         bool mirror, float diag) {
    const float k = inv_sx * inv_sx;
    const RoundScale rs(s.sa * k, r);
    const uint64_t r0 = rs.pair(0), r1 = rs.pair(1);
    uint32_t x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = pack_pair(mul2(pair_of(acc[2 * j], acc[2 * j + 1]), (j & 1) ? r1 : r0));
    const int lane = row & 31;
    if (r - lane == c0) {       // the warp's rows are these columns
        a.diag_a[diag_at + r] = diag * k;
        clear_diagonal(x, lane);
    }
    put_sym(slot, row, h, x, mirror);
}

// dr: A_rr; cols: A_cc of the 32 columns, in shared memory
__device__ __forceinline__ void finish_b(const OrthoArgs& a, const OrthoStep& s, int64_t diag_at, uint32_t slot,
                                         int row, int h, int r, int c0, const float* acc, bool mirror, float dr,
                                         uint32_t cols) {
    uint4 f4[4], e4[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) f4[q] = lds128(slot + row * 128 + (((4 * h + q) ^ (row & 7)) << 4));
#pragma unroll
    for (int q = 0; q < 8; ++q) e4[q] = lds128(cols + 16 * q);
    // c (F F^T) + (b + c (D_r + D_c)) F, F in fp16 under the scale of A
    const float k = s.c * s.inv_sa * s.inv_sa, fb = fmaf(s.c, dr, s.b) * s.inv_sa, fc = s.c * s.inv_sa;
    const int lane = row & 31;
    const bool diag = r - lane == c0;   // the warp's rows are these columns
    if (diag) {                         // F_rr is 0: only the sum counts
        float ff = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) ff = j == lane ? acc[j] : ff;
        const float d2 = dr * dr, aa = fmaf(ff * s.inv_sa, s.inv_sa, d2);   // (A A^T)_rr
        const float db = fmaf(fmaf(s.c, dr, s.b), dr, k * ff);
        a.diag_b[diag_at + r] = db;
        a.diag_t[diag_at + r] = aa > 0.0f ? db * (d2 / aa) : 0.0f;
    }
    const RoundScale rs(s.sb, r);
    const uint64_t r0 = rs.pair(0), r1 = rs.pair(1);
    const uint64_t k2 = pair_of(k, k), fb2 = pair_of(fb, fb), fc2 = pair_of(fc, fc);
    uint32_t x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint4 f = f4[j >> 2], e = e4[j >> 1];
        const uint32_t fw = (j & 3) == 0 ? f.x : (j & 3) == 1 ? f.y : (j & 3) == 2 ? f.z : f.w;
        const uint64_t dc = (j & 1) ? pair_of(__uint_as_float(e.z), __uint_as_float(e.w))
                                    : pair_of(__uint_as_float(e.x), __uint_as_float(e.y));
        const uint64_t v = fma2(k2, pair_of(acc[2 * j], acc[2 * j + 1]), mul2(fma2(fc2, dc, fb2), unpack_pair(fw)));
        x[j] = pack_pair(mul2(v, (j & 1) ? r1 : r0));
    }
    if (diag) clear_diagonal(x, lane);
    put_sym(slot, row, h, x, mirror);
}

// What a step that takes both halves does with a tile of A or B.  The values
// as they are to be stored, in fp32 in place of the sums:
__device__ __forceinline__ void values_a(const OrthoArgs& a, const OrthoStep& s, int64_t diag_at, float inv_sx, int row,
                                         int r, int c0, float* acc, float diag) {
    const float k = inv_sx * inv_sx;
    const int lane = row & 31;
    const bool on = r - lane == c0;
    if (on) a.diag_a[diag_at + r] = diag * k;
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = on && j == lane ? 0.0f : acc[j] * (s.sa * k);
}
// (as finish_b, with F the sum of both halves, in the slot one behind the other)
__device__ __forceinline__ void values_b(const OrthoArgs& a, const OrthoStep& s, int64_t diag_at, uint32_t slot,
                                         int row, int h, int r, int c0, float* acc, float dr, const float* cols) {
    const float k = s.c * s.inv_sa * s.inv_sa, fb = fmaf(s.c, dr, s.b) * s.inv_sa, fc = s.c * s.inv_sa;
    const int lane = row & 31;
    const bool on = r - lane == c0;
    if (on) {
        float ff = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) ff = j == lane ? acc[j] : ff;
        const float db = fmaf(fmaf(s.c, dr, s.b), dr, k * ff);
        a.diag_b[diag_at + r] = db;
        a.diag_t[diag_at + r] = db;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t at = slot + row * 128 + (((4 * h + q) ^ (row & 7)) << 4);
        const uint4 f4 = lds128(at), l4 = lds128(at + uint32_t(kBlkBytes));
        const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 u = unpack_half2(f[j]), v = unpack_half2(l[j]);
            const int e = 8 * q + 2 * j;
            acc[e] = fmaf(k, acc[e], fmaf(fc, cols[e], fb) * (u.x + v.x)) * s.sb;
            acc[e + 1] = fmaf(k, acc[e + 1], fmaf(fc, cols[e + 1], fb) * (u.y + v.y)) * s.sb;
        }
    }
    if (on)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[j] = j == lane ? 0.0f : acc[j];
}
// one half of 32 values into the slot
__device__ __forceinline__ void put_half(uint32_t slot, int row, int h, int r, const float* v, bool mirror, bool low) {
    const RoundScale rs(1.0f, r);
    uint32_t x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        x[j] = pack_half2(v[2 * j] * rs.v[2 * j & 3], v[2 * j + 1] * rs.v[(2 * j + 1) & 3]);
        if (low) {
            const float2 f = unpack_half2(x[j]);
            x[j] = pack_half2(v[2 * j] - f.x, v[2 * j + 1] - f.y);
        }
    }
    put_sym(slot, row, h, x, mirror);
}

// ah, al: factors of hi and lo; k: of the sums; lo_scale: of the new lo.
// Returns the sum of squares of the new X.  The last step leaves bf16 values in
// the slot instead.
__device__ __forceinline__ float finish_x(const OrthoStep& s, uint32_t slot, int row, int h, int r,
                                          const float* acc, float ah, float al, float k, float lo_scale, bool has_lo,
                                          bool last) {
    uint4 h4[4], l4[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) h4[q] = lds128(slot + row * 128 + (((4 * h + q) ^ (row & 7)) << 4));
#pragma unroll
    for (int q = 0; q < 4; ++q)
        l4[q] = has_lo ? lds128(slot + uint32_t(kBlkBytes) + row * 128 + (((4 * h + q) ^ (row & 7)) << 4))
                       : make_uint4(0, 0, 0, 0);
    const RoundScale rs(s.sx_next, r);
    const uint64_t r0 = rs.pair(0), r1 = rs.pair(1);
    const uint64_t k2 = pair_of(k, k), ah2 = pair_of(ah, ah), al2 = pair_of(al, al);
    const float up = s.sx_next * lo_scale;
    const uint64_t up2 = pair_of(up, up), down2 = pair_of(-lo_scale, -lo_scale);
    uint64_t sq = 0;   // two zeros
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t hi[4] = {h4[q].x, h4[q].y, h4[q].z, h4[q].w}, lo[4] = {l4[q].x, l4[q].y, l4[q].z, l4[q].w};
        uint32_t nh[4], nl[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t sum = pair_of(acc[8 * q + 2 * j], acc[8 * q + 2 * j + 1]);
            const uint64_t x = fma2(ah2, unpack_pair(hi[j]), fma2(al2, unpack_pair(lo[j]), mul2(k2, sum)));
            if (last) {
                const float2 f = halves_of(x);
                const __nv_bfloat162 o = __floats2bfloat162_rn(f.x, f.y);
                nh[j] = *reinterpret_cast<const uint32_t*>(&o);
            } else {
                sq = fma2(x, x, sq);
                nh[j] = pack_pair(mul2(x, (j & 1) ? r1 : r0));
                // lo_scale (x sx - hi), exactly as from the separate products
                nl[j] = pack_pair(fma2(unpack_pair(nh[j]), down2, mul2(x, up2)));
            }
        }
        const uint32_t at = slot + row * 128 + (((4 * h + q) ^ (row & 7)) << 4);
        sts128(at, nh[0], nh[1], nh[2], nh[3]);
        if (!last) sts128(at + uint32_t(kBlkBytes), nl[0], nl[1], nl[2], nl[3]);
    }
    const float2 f = halves_of(sq);
    return f.x + f.y;
}

// A warp's 32 rows x 32 columns of bf16 results from the slot to the flat
// output.  By rows: four lanes per row.  A tall matrix: lanes along X's rows.
__device__ __forceinline__ void write_out(const OrthoArgs& a, const MatDesc& d, uint32_t slot, int row0, int h,
                                          int r0, int c0) {
    __syncwarp();
    const int lane = int(threadIdx.x & 31);
    if (!d.tall) {
        const bool vec = ((d.off | d.n) & 7) == 0;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int rr = 8 * p + (lane >> 2), q = lane & 3, row = row0 + rr;
            const int r = r0 + rr, c = c0 + 8 * q;
            if (r >= d.m || c >= d.n) continue;
            const uint4 v = lds128(slot + row * 128 + (((4 * h + q) ^ (row & 7)) << 4));
            uint16_t* o = a.out + d.off + int64_t(r) * d.n + c;
            if (vec) {
                *reinterpret_cast<uint4*>(o) = v;
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < d.n) o[j] = uint16_t(w[j >> 1] >> (16 * (j & 1)));
            }
        }
    } else {
        const int row = row0 + lane, r = r0 + lane;
        if (r < d.m) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 v = lds128(slot + row * 128 + (((4 * h + q) ^ (row & 7)) << 4));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = c0 + 8 * q + j;
                    if (c < d.n) a.out[d.off + int64_t(c) * d.m + r] = uint16_t(w[j >> 1] >> (16 * (j & 1)));
                }
            }
        }
    }
}

// X's low part as step `step` reads it (and step - 1 writes it): in place, or
// from buffer to buffer through the steps that take both halves.
template <bool BOTH>
__device__ __forceinline__ unsigned char* low_half(const OrthoArgs& a, const MatDesc& d, int step) {
    return BOTH && (min(step, both_steps_of(a, d)) & 1) ? (d.both ? a.ws : a.ws_low) + d.lo2 * kBlkBytes
                                                        : a.ws + d.lo * kBlkBytes;
}

// The count that must have been reached before a tile of (prod, step) starts.
__device__ __forceinline__ bool wait_operands(OrthoShared& sh, const OrthoArgs& a, const MatDesc& d, int mat,
                                              int prod, int step) {
    const int before = prod == kProdA ? kProdX : prod - 1;
    const int target = (prod == kProdA ? step : step + 1) * 2 * d.tiles[before];
    return wait_count(sh, a.done + 3 * mat + before, target, a);
}

// How many sums a product is: hi hi, lo hi, hi lo.  X_0 of a bf16 update has no lo.
__device__ __forceinline__ int sums_of(int prod, bool both, bool has_lo) {
    return !both ? 1 : prod == kProdB || has_lo ? 3 : prod == kProdX ? 2 : 1;
}
// How often a 64-column block of a tile goes through a slot.  With both halves,
// a block of A leaves as hi and as lo, one of B comes in (both halves of A's)
// before it does: their mirror images need the room of the second half.
__device__ __forceinline__ int visits_of(int prod, bool both) {
    return !both || prod == kProdX ? 1 : prod == kProdA ? 2 : 3;
}

// First 64-deep block and number of blocks of a part of a tile's sum.
__device__ __forceinline__ int2 part_of_sum(const MatDesc& d, const OrthoTile& t, int part) {
    const int all = t.prod == kProdA ? d.kn : d.km;
    const int k0 = all * part >> t.split;
    return make_int2(k0, (all * (part + 1) >> t.split) - k0);
}

// A tile of A in parts.  Every part holds sums for the whole tile, over its
// share of the columns of X; it finishes one part's share of the 64-column
// blocks and leaves the others' sums for the pairs that finish those.  Per
// group: [part][CTA][warp][block][four columns][lane], 16 bytes each, in the
// buffer of the next X: a warp writes and reads 512 contiguous bytes at once,
// and needs only what the same warp of the other pairs left.  Adds the others'
// sums, in their order, to this part's in tensor memory.  (Not inlined: beside
// the other code of the finish it made every product 0.3 us longer.)
constexpr int kSumsOfWarp = 8 * 32;   // float4 per block
__device__ __noinline__ bool join_parts(OrthoShared& sh, const OrthoArgs& a, const MatDesc& d, OrthoTile t,
                                        uint32_t sums, int step, int warp) {   // warp: 0 .. 15 of the pair's
    const int own = t.blocks >> t.split, lane = int(threadIdx.x & 31);
    const int64_t per_part = int64_t(2 * kEpiWarps) * t.blocks * kSumsOfWarp;
    float4* left = reinterpret_cast<float4*>(a.ws + d.x[(step + 1) & 1] * kBlkBytes) +
                   (int64_t(t.group - d.group0) << t.split) * per_part +
                   int64_t(warp) * t.blocks * kSumsOfWarp + lane;
#pragma unroll 1
    for (int b = 0; b < t.blocks; ++b) {
        if (b >= t.part * own && b < (t.part + 1) * own) continue;
        float v[32];
        load_acc32(sums + uint32_t(b) * 64, v);
        float4* out = left + t.part * per_part + b * kSumsOfWarp;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            __stcg(out + q * 32, make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
    }
    __syncwarp();
    bool ok = true;
    if (lane == 0) {
        int32_t* join = a.join + int64_t(t.group) * (2 * kEpiWarps) + warp;
        asm volatile("red.release.gpu.global.add.s32 [%0], 1;" :: "l"(join) : "memory");
        ok = wait_count(sh, join, (step + 1) << t.split, a);
    }
    if (!__all_sync(0xFFFFFFFFu, ok)) return false;
    __syncwarp();
#pragma unroll 1
    for (int b = t.part * own; b < (t.part + 1) * own; ++b) {
        float acc[32];
        load_acc32(sums + uint32_t(b) * 64, acc);
#pragma unroll 1
        for (int p = 0; p < 1 << t.split; ++p) {
            if (p == t.part) continue;
            const float4* in = left + p * per_part + b * kSumsOfWarp;
            float4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = __ldcg(in + q * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                acc[4 * q] += v[q].x;
                acc[4 * q + 1] += v[q].y;
                acc[4 * q + 2] += v[q].z;
                acc[4 * q + 3] += v[q].w;
            }
        }
        store_acc32(sums + uint32_t(b) * 64, acc);
    }
    return true;
}

// BOTH: some steps of some matrices take both halves of their operands.  X's low part is then an operand that other tiles
// read, so it alternates between two buffers as X does; the free one holds A's
// low part while that is needed.
template <bool BOTH>
struct LowMaps {};
template <>
struct LowMaps<true> {
    CUtensorMap rows128, rows64;     // of the second workspace
};
template <bool BOTH>
__global__ void __cluster_dims__(2) __launch_bounds__(kOrthoThreads, 1)
k_ortho_steps(const __grid_constant__ OrthoArgs a, const __grid_constant__ CUtensorMap rows128,
              const __grid_constant__ CUtensorMap rows64, const __grid_constant__ LowMaps<BOTH> low_maps) {
    // the kernel's only shared memory: starts on a multiple of 1 KB, as the swizzle wants it
    extern __shared__ __align__(1024) unsigned char dyn[];
    OrthoShared& sh = *reinterpret_cast<OrthoShared*>(dyn + kStages * kStageBytes + kSlots * kSlotBytes);
    const uint32_t stage0 = smem_u32(dyn);
    const uint32_t slot0 = stage0 + uint32_t(kStages) * kStageBytes;
    const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
    const uint32_t rank = cluster_rank();
    const int pair = int(blockIdx.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.tfull[b], 1);
            mbar_init(&sh.tempty[b], 2 * kEpiWarps);
            mbar_init(&sh.in_full[b], 1);
            mbar_init(&sh.out_ready[b], kEpiWarps);
            mbar_init(&sh.slot_free[b], 1);
        }
        mbar_init(&sh.tile_ready, 1);
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
    const int q0 = __ldg(a.queue_first + pair), q1 = __ldg(a.queue_first + pair + 1);

    if (warp == 0 && lane == 0) {
        // ---- operands ----
        // (what the loop over K needs is in registers: the copies' memory
        // clobbers would have a value of the descriptor loaded again for each)
        const uint32_t full0 = map_to(smem_u32(&sh.full[0]), 0);
        int s = 0;
        int64_t skip = blockIdx.x == 0 ? a.skip : -1;   // stages until the one left out
        uint32_t par = 1;             // the first pass over the ring finds it empty
        bool ok = true;
        for (int step = 0; step < a.n_steps && ok; ++step) {
            const bool has_lo = step > 0 || a.f32;
            for (int t = q0; t < q1 && ok; ++t) {
                const OrthoTile tile = a.queue[t];
                const MatDesc& d = a.mats[tile.mat];
                const int prod = tile.prod;
                const bool both = BOTH && step < both_steps_of(a, d);
                const int64_t x = d.x[step & 1];
                const int64_t from = prod == kProdA ? x : prod == kProdB ? d.a : d.b;
                const int cb = prod == kProdA ? d.cbx : d.cba, kblocks = part_of_sum(d, tile, tile.part).y;
                const int half = tile.blocks * 32, c0 = tile.j * tile.blocks * 64 + int(rank) * half;
                const int k0 = part_of_sum(d, tile, tile.part).x * kBlkRows;
                int left = int((from + int64_t(tile.i * 2 + int(rank)) * cb) * kBlkRows) + k0;
                int right = prod == kProdX ? int((x + (c0 >> 6)) * kBlkRows)
                                           : int((from + int64_t(c0 >> 7) * cb) * kBlkRows) + (c0 & 127) + k0;
                const uint32_t bytes = 2 * (kHalfBytes + uint32_t(half) * 128);
                const int pitch = d.cbx * kBlkRows;
                if (!(ok = wait_operands(sh, a, d, tile.mat, prod, step))) break;
                const CUtensorMap *left_map = &rows128, *right128 = &rows128, *right64 = &rows64;
                const int left_hi = left, right_hi = right, sums = sums_of(prod, both, has_lo);
                for (int k = 0, kb = 0, sum = 0; k < kblocks * sums; ++k, ++kb) {
                    if constexpr (BOTH) {
                        if (kb == kblocks) {   // the next sum
                            kb = 0;
                            // from the blocks of the high half to those of the low one: X's (or, where
                            // A is the operand, A's) in the first or the second workspace, or B's
                            const bool second = ((prod == kProdB ? step + 1 : step) & 1) != 0;
                            const int64_t low = second ? d.lo2 : d.lo;
                            const CUtensorMap* low128 = d.both ? &rows128 : &low_maps.rows128;
                            if (++sum == 1) {
                                left = left_hi + int(((prod == kProdX ? d.blo : low) - from) * kBlkRows);
                                left_map = prod == kProdX || second ? low128 : &rows128;
                            } else {
                                left = left_hi;
                                left_map = &rows128;
                                right = right_hi + int((low - (prod == kProdX ? x : from)) * kBlkRows);
                                right128 = second ? low128 : &rows128;
                                right64 = second && !d.both ? &low_maps.rows64 : &rows64;
                            }
                        }
                    }
                    if (!(ok = wait_bounded(sh, &sh.empty[s], par, a))) break;
                    const uint32_t bar = full0 + uint32_t(s) * 8;
                    if (rank == 0) mbar_expect(&sh.full[s], bytes);
                    const uint32_t dst = stage0 + uint32_t(s) * kStageBytes;
                    if (skip-- != 0) copy_box(dst, left_map, left + kb * kBlkRows, bar);
                    if (prod == kProdX) {
                        const int row = right + (kb >> 1) * pitch + (kb & 1) * 64;
                        copy_box(dst + kHalfBytes, right64, row, bar);
                        if (half == 128) copy_box(dst + kHalfBytes + 8192, right64, row + kBlkRows, bar);
                    } else {
                        copy_box(dst + kHalfBytes, half == 128 ? right128 : right64, right + kb * kBlkRows, bar);
                    }
                    if (++s == kStages) {
                        s = 0;
                        par ^= 1;
                    }
                }
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---- products ----
        int s = 0, it = 0;
        uint32_t par = 0;
        bool ok = true;
        for (int step = 0; step < a.n_steps && ok; ++step) {
            const bool has_lo = step > 0 || a.f32;
            for (int t = q0; t < q1 && ok; ++t, ++it) {
                const OrthoTile tile = a.queue[t];
                const MatDesc& d = a.mats[tile.mat];
                const bool both = BOTH && step < both_steps_of(a, d);
                const bool by_column = tile.prod == kProdX;
                const uint32_t shape = mma_shape(by_column, tile.blocks * 64);
                const int kblocks = part_of_sum(d, tile, tile.part).y * sums_of(tile.prod, both, has_lo);
                const int buf = it & 1;
                if (!(ok = wait_bounded(sh, &sh.tempty[buf], uint32_t((it >> 1) & 1) ^ 1u, a))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!(ok = wait_bounded(sh, &sh.full[s], par, a))) break;
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
        }
    } else if (warp == kFillWarp && lane == 0) {
        // ---- slots in ----
        uint32_t n = 0;               // 64-column blocks so far; block n uses slot n mod 2
        int before = 2;               // blocks of the tile before
        bool ok = true;
        for (int step = 0; step < a.n_steps && ok; ++step) {
            const bool has_lo = step > 0 || a.f32;
            for (int t = q0; t < q1 && ok; ++t) {
                const OrthoTile tile = a.queue[t];
                const MatDesc& d = a.mats[tile.mat];
                const bool both = BOTH && step < both_steps_of(a, d);
                const int prod = tile.prod, blocks = tile.blocks >> tile.split;   // (parts: of A, which reads no blocks)
                const int64_t blk = int64_t(tile.i * 2 + int(rank)) * (prod == kProdX ? d.cbx : d.cba) + tile.j * blocks;
                const unsigned char* in = a.ws + ((prod == kProdB ? d.a : d.x[step & 1]) + blk) * kBlkBytes;
                // (of X, or A's in the buffer that X's goes to next)
                const unsigned char* lo = low_half<BOTH>(a, d, prod == kProdB ? step + 1 : step) + blk * kBlkBytes;
                const bool two = prod == kProdX ? has_lo : both;
                const int visits = visits_of(prod, both);
                if (!(ok = wait_operands(sh, a, d, tile.mat, prod, step))) break;
                for (int g = 0; g < blocks && ok; ++g)
                    for (int v = 0; v < visits; ++v, ++n) {
                        const uint32_t sl = n & 1, at = slot0 + sl * kSlotBytes;
                        if (!(ok = wait_bounded(sh, &sh.slot_free[sl], ((n >> 1) & 1) ^ 1u, a))) break;
                        // Tells the finishing warps, which so need not watch the counter in memory
                        // themselves (ten watchers per CTA instead of two delayed it by a
                        // microsecond).  They have all seen it for the tile before, or they could
                        // miss a phase: a block of that tile is finished, the one in this slot or,
                        // if it had one only, the one in the other slot.
                        if (g == 0 && v == 0) {
                            if (before == 1 &&
                                !(ok = wait_bounded(sh, &sh.slot_free[sl ^ 1], ((n - 1) >> 1) & 1, a)))
                                break;
                            mbar_arrive(&sh.tile_ready);
                        }
                        if (prod == kProdA || v > 0) {
                            mbar_arrive(&sh.in_full[sl]);
                            continue;
                        }
                        mbar_expect(&sh.in_full[sl], uint32_t(kBlkBytes) * (two ? 2 : 1));
                        copy_in(at, in + g * kBlkBytes, uint32_t(kBlkBytes), &sh.in_full[sl]);
                        if (two) copy_in(at + uint32_t(kBlkBytes), lo + g * kBlkBytes, uint32_t(kBlkBytes), &sh.in_full[sl]);
                    }
                before = blocks * visits;
            }
        }
    } else if (warp == kStoreWarp && lane == 0) {
        // ---- slots out ----
        uint32_t n = 0;               // as above
        bool ok = true;
        for (int step = 0; step < a.n_steps && ok; ++step) {
            const bool last = step + 1 == a.n_steps;
            for (int t = q0; t < q1 && ok; ++t) {
                const OrthoTile tile = a.queue[t];
                const MatDesc& d = a.mats[tile.mat];
                const bool both = BOTH && step < both_steps_of(a, d);
                const int prod = tile.prod, blocks = tile.blocks >> tile.split, visits = visits_of(prod, both);
                const int c0 = tile.j * tile.blocks + tile.part * blocks;
                const bool mirror = prod != kProdX && (c0 >> 2) > tile.i;
                const int cb = prod == kProdX ? d.cbx : d.cba;
                // the CTA's first block in memory, and its mirror image's columns
                const int64_t blk = int64_t(tile.i * 2 + int(rank)) * cb + c0;
                unsigned char* out = a.ws + ((prod == kProdA ? d.a : prod == kProdB ? d.b : d.x[(step + 1) & 1]) +
                                             blk) * kBlkBytes;
                // where the low half goes: X's, or A's beside it, or B's
                unsigned char* low = BOTH && both && prod == kProdB
                                         ? (d.both ? a.ws : a.ws_low) + d.blo * kBlkBytes
                                         : low_half<BOTH>(a, d, step + 1);
                unsigned char* lo = low + blk * kBlkBytes;
                const int64_t image_at = int64_t(tile.i * 4 + int(rank) * 2) * kBlkBytes;
                unsigned char* image = a.ws + (prod == kProdA ? d.a : d.b) * kBlkBytes + image_at;
                int32_t* done = a.done + 3 * tile.mat + prod;
                for (int g = 0; g < blocks && ok; ++g)
                    for (int v = 0; v < visits; ++v, ++n) {
                        const uint32_t sl = n & 1, at = slot0 + sl * kSlotBytes;
                        if (!(ok = wait_bounded(sh, &sh.out_ready[sl], (n >> 1) & 1, a))) break;
                        if (prod != kProdX) {
                            // with both halves the last two of a block's visits leave hi and lo
                            const bool is_low = both && v + 1 == visits;
                            if (both && v + 2 < visits) {
                                mbar_arrive(&sh.slot_free[sl]);
                                continue;
                            }
                            copy_out((is_low ? lo : out) + g * kBlkBytes, at, uint32_t(kBlkBytes));
                            if (mirror) {     // 64 rows from this block's first column, 2 x 64 columns
                                unsigned char* m = (is_low ? low + image_at : image) +
                                                   int64_t((c0 + g) >> 1) * cb * kBlkBytes + ((c0 + g) & 1) * 8192;
                                copy_out(m, at + uint32_t(kBlkBytes), 8192);
                                copy_out(m + kBlkBytes, at + uint32_t(kBlkBytes) + 8192, 8192);
                            }
                        } else if (!last) {
                            copy_out(out + g * kBlkBytes, at, uint32_t(kBlkBytes));
                            copy_out(lo + g * kBlkBytes, at + uint32_t(kBlkBytes), uint32_t(kBlkBytes));
                        }
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        mbar_arrive(&sh.slot_free[sl]);
                    }
                if (!ok) break;
                // all of the tile is in memory before its count (the release covers what the
                // finishing warps wrote, too: they arrived at out_ready after it)
                asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                asm volatile("fence.proxy.async;" ::: "memory");
                asm volatile("red.release.gpu.global.add.s32 [%0], 1;" :: "l"(done) : "memory");
            }
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else if (warp >= 2 && warp < kFillWarp) {
        // ---- finish ----
        const int quad = warp & 3, half = (warp - 2) >> 2;   // the warp's rows, its 32 columns of 64
        const int row0 = quad * 32, row = row0 + lane;
        float* cols = sh.cols[warp - 2];
        int it = 0;
        uint32_t n = 0;               // as above
        bool ok = true;
        for (int step = 0; step < a.n_steps && ok; ++step) {
            const OrthoStep s = a.st[step];
            const bool last = step + 1 == a.n_steps;
            const bool has_lo = step > 0 || a.f32;
            for (int t = q0; t < q1 && ok; ++t, ++it) {
                const OrthoTile tile = a.queue[t];
                const MatDesc& d = a.mats[tile.mat];
                const int prod = tile.prod, buf = it & 1, blocks = tile.blocks >> tile.split;
                const int first = tile.part * blocks;        // of the tile's blocks, the first to finish here
                const int c0 = (tile.j * tile.blocks + first) * 64;
                const int r0 = tile.i * kOrthoTile + int(rank) * 128 + row0, r = r0 + lane;
                const int64_t diag_at = d.diag;
                const bool both = BOTH && step < both_steps_of(a, d);
                const float inv_lo = both ? 1.0f : kInvLoScale, lo_next = BOTH ? lo_scale_of(a, d, step + 1) : kLoScale;
                const bool mirror = prod != kProdX && (c0 >> 8) > tile.i;
                ok = wait_bounded(sh, &sh.tile_ready, uint32_t(it & 1), a);
                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                // what the rows need, fetched while the product runs
                const float inv_sx = step == 0 ? __ldcg(&a.scal[tile.mat].y) : s.inv_sx;
                float p0 = 0.0f, p1 = 0.0f, dc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sq = 0.0f;
                if (prod == kProdA) {
                    // if the tile holds the diagonal of these rows, in this warp's 32 columns
                    if (r0 >= c0 && r0 < c0 + blocks * 64 && half == (quad & 1)) p0 = row_square(a, d, r);
                } else if (prod == kProdB) {
                    p0 = __ldcg(a.diag_a + d.diag + r);
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        if (g < blocks) dc[g] = __ldcg(a.diag_a + d.diag + c0 + g * 64 + half * 32 + lane);
                } else {
                    p0 = fmaf(__ldcg(a.diag_b + d.diag + r), inv_sx, s.a * inv_sx);
                    p1 = fmaf(__ldcg(a.diag_t + d.diag + r), inv_sx, s.a * inv_sx) * inv_lo;
                }
                ok = wait_bounded(sh, &sh.tfull[buf], uint32_t((it >> 1) & 1), a);
                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t sums = tmem + uint32_t(buf) * kOrthoTile + uint32_t(half) * 32 + (uint32_t(row0) << 16);
                if (tile.split && !(ok = join_parts(sh, a, d, tile, sums, step, int(rank) * kEpiWarps + warp - 2)))
                    break;
#pragma unroll 1
                for (int g = 0; g < blocks; ++g, ++n) {
                    const int c = c0 + g * 64 + half * 32;
                    const uint32_t sl = n & 1, slot = slot0 + sl * kSlotBytes;
                    float acc[32];
                    load_acc32(sums + uint32_t(first + g) * 64, acc);
                    if (g + 1 == blocks) {   // the accumulator is free for the tile after next
                        // (its values are in registers: relaxed, a release would first wait for
                        // this warp's stores, a microsecond)
                        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                        __syncwarp();
                        if (lane == 0)
                            asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];"
                                         :: "r"(map_to(smem_u32(&sh.tempty[buf]), 0)) : "memory");
                    }
                    ok = wait_bounded(sh, &sh.in_full[sl], (n >> 1) & 1, a);
                    if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                    if (BOTH && both && prod != kProdX) {
                        const int visits = visits_of(prod, both);
                        if (prod == kProdA) {
                            values_a(a, s, diag_at, inv_sx, row, r, c, acc, p0);
                        } else {
                            __syncwarp();
                            cols[lane] = g == 0 ? dc[0] : g == 1 ? dc[1] : g == 2 ? dc[2] : dc[3];
                            __syncwarp();
                            values_b(a, s, diag_at, slot, row, half, r, c, acc, p0, cols);
                        }
#pragma unroll 1
                        for (int v = 0; v < visits; ++v) {
                            const uint32_t sv = n & 1;
                            if (v > 0) {
                                ok = wait_bounded(sh, &sh.in_full[sv], (n >> 1) & 1, a);
                                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                            }
                            if (v + 2 >= visits)
                                put_half(slot0 + sv * kSlotBytes, row, half, r, acc, mirror, v + 1 == visits);
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sh.out_ready[sv]);
                            if (v + 1 < visits) ++n;      // (the loop counts the last)
                        }
                        if (!ok) break;
                        continue;
                    }
                    if (prod == kProdA) {
                        finish_a(a, s, diag_at, inv_sx, slot, row, half, r, c, acc, mirror, p0);
                    } else if (prod == kProdB) {
                        __syncwarp();
                        cols[lane] = g == 0 ? dc[0] : g == 1 ? dc[1] : g == 2 ? dc[2] : dc[3];
                        __syncwarp();
                        finish_b(a, s, diag_at, slot, row, half, r, c, acc, mirror, p0, smem_u32(cols));
                    } else {
                        sq += finish_x(s, slot, row, half, r, acc, p0, p1, inv_sx * s.inv_sb, lo_next, has_lo, last);
                        if (last) {
                            write_out(a, d, slot, row0, half, r0, c);
                        } else if (g & 1) {   // of this warp's 32 columns in two blocks
                            a.rowsq[d.rowsq + int64_t((c0 >> 6) + (g & 2) + half) * d.rows_pad + r] = sq * s.sx_next * s.sx_next;
                            sq = 0.0f;
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.out_ready[sl]);
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

// The tables of the weight update, which needs nothing else; m.mu is held.
static int upload_update_tables(Matrices& m) {
    int dev = 0;
    DPG_CUDA_TRY(cudaGetDevice(&dev));
    if (m.device >= 0) {
        if (m.device != dev)
            return fail(DPG_ERR_INVALID_ARG, "matrices live on device %d but device %d is current",
                        m.device, dev);
        return DPG_OK;
    }
    const size_t bytes = round256(m.apply_items.size() * sizeof(ApplyItem)) +
                         round256(m.scales.size() * sizeof(double));
    void* tables = nullptr;
    cudaError_t e = cudaMalloc(&tables, bytes ? bytes : 256);
    size_t at = 0;
    if (e == cudaSuccess) e = put(static_cast<unsigned char*>(tables), &at, m.apply_items, &m.d_apply_items);
    if (e == cudaSuccess) e = put(static_cast<unsigned char*>(tables), &at, m.scales, &m.d_scales);
    if (e == cudaSuccess) e = upload_done();
    if (e != cudaSuccess) {
        cudaFree(tables);
        cudaGetLastError();
        return fail(e == cudaErrorMemoryAllocation ? DPG_ERR_OOM : DPG_ERR_CUDA, "matrices upload: %s",
                    cudaGetErrorString(e));
    }
    m.d_update_tables = static_cast<unsigned char*>(tables);
    m.device = dev;
    return DPG_OK;
}

int upload_for_update(Matrices& m) {
    std::lock_guard<std::mutex> g(m.mu);
    return upload_update_tables(m);
}

// The second workspace, which only steps that take both halves need; m.mu is
// held, the tables are there.
static int upload_low(Matrices& m) {
    if (m.ws_low || m.n_low_blocks == 0) return DPG_OK;
    void* low = nullptr;
    const cudaError_t e = cudaMalloc(&low, size_t(m.n_low_blocks * kBlkBytes));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(e == cudaErrorMemoryAllocation ? DPG_ERR_OOM : DPG_ERR_CUDA, "matrices upload: %s",
                    cudaGetErrorString(e));
    }
    for (int k = 0; k < 2; ++k) {
        CUtensorMap map;
        const int st = encode_map(&map, low, m.n_low_blocks * kBlkRows, k ? 64 : 128);
        if (st != DPG_OK) {
            cudaFree(low);
            return st;
        }
        std::memcpy(m.maps[2 + k], &map, sizeof map);
    }
    m.ws_low = static_cast<unsigned char*>(low);
    return DPG_OK;
}

int upload_matrices(Matrices& m, bool both) {
    std::lock_guard<std::mutex> g(m.mu);
    int st = upload_update_tables(m);
    if (st != DPG_OK) return st;
    if (m.ws) return both ? upload_low(m) : DPG_OK;
    // how many CTA pairs are resident at once decides the queues
    int clusters = 1;
    if (!m.mats.empty()) {
        DPG_CUDA_TRY(cudaFuncSetAttribute(k_ortho_load<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          2 * kLoadSmem));
        DPG_CUDA_TRY(cudaFuncSetAttribute(k_ortho_steps<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOrthoSmem));
        DPG_CUDA_TRY(cudaFuncSetAttribute(k_ortho_steps<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOrthoSmem));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kOrthoThreads);
        cfg.dynamicSmemBytes = kOrthoSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        DPG_CUDA_TRY(cudaOccupancyMaxActiveClusters(&clusters, k_ortho_steps<false>, &cfg));
        if (clusters < 1) return fail(DPG_ERR_CUDA, "matrices upload: no CTA pair fits this device");
    }
    if (!m.small.empty()) {
        st = gram_prepare();
        if (st != DPG_OK) return st;
    }
    try {
        lay_queue(m, clusters);
    } catch (const std::exception&) {
        return fail(DPG_ERR_OOM, "matrices upload: out of host memory");
    }
    const size_t bytes = round256(m.mats.size() * sizeof(MatDesc)) +
                         round256(m.queue.size() * sizeof(OrthoTile)) +
                         round256(m.queue_first.size() * sizeof(int32_t)) +
                         round256(m.small.size() * sizeof(SmallDesc)) +
                         round256(m.gram_items.size() * sizeof(SmallItem)) +
                         round256(m.prod_items.size() * sizeof(SmallItem)) +
                         round256(m.small_order.size() * sizeof(int32_t)) +
                         round256(m.norm_items.size() * sizeof(NormItem)) +
                         round256(m.conv_items.size() * sizeof(ConvItem));
    void *ws = nullptr, *tables = nullptr;
    cudaError_t e = cudaMalloc(&tables, bytes ? bytes : 256);
    if (e == cudaSuccess) e = cudaMalloc(&ws, size_t(m.workspace_bytes));
    unsigned char* t = static_cast<unsigned char*>(tables);
    size_t at = 0;
    if (e == cudaSuccess) e = put(t, &at, m.mats, &m.d_mats);
    if (e == cudaSuccess) e = put(t, &at, m.queue, &m.d_queue);
    if (e == cudaSuccess) e = put(t, &at, m.queue_first, &m.d_queue_first);
    if (e == cudaSuccess) e = put(t, &at, m.small, &m.d_small);
    if (e == cudaSuccess) e = put(t, &at, m.gram_items, &m.d_gram_items);
    if (e == cudaSuccess) e = put(t, &at, m.prod_items, &m.d_prod_items);
    if (e == cudaSuccess) e = put(t, &at, m.small_order, &m.d_small_order);
    if (e == cudaSuccess) e = put(t, &at, m.norm_items, &m.d_norm_items);
    if (e == cudaSuccess) e = put(t, &at, m.conv_items, &m.d_conv_items);
    // arrival counters and the status word start at zero
    if (e == cudaSuccess)
        e = cudaMemset(static_cast<unsigned char*>(ws) + m.o_count, 0, size_t(m.o_status + 256 - m.o_count));
    if (e == cudaSuccess) e = upload_done();
    if (e != cudaSuccess) {
        cudaGetLastError();
        st = fail(e == cudaErrorMemoryAllocation ? DPG_ERR_OOM : DPG_ERR_CUDA, "matrices upload: %s",
                  cudaGetErrorString(e));
    }
    static_assert(sizeof(CUtensorMap) == sizeof(m.maps[0]), "room for a tensor map");
    for (int k = 0; k < 2 && st == DPG_OK && m.n_blocks > 0; ++k) {
        CUtensorMap map;
        st = encode_map(&map, ws, m.n_blocks * kBlkRows, k ? 64 : 128);
        std::memcpy(m.maps[k], &map, sizeof map);
    }
    if (st != DPG_OK) {
        cudaFree(tables);
        cudaFree(ws);
        return st;
    }
    m.d_tables = t;
    m.ws = static_cast<unsigned char*>(ws);
    return both ? upload_low(m) : DPG_OK;
}

int check_matrices(Matrices& m, void* stream) {
    if (!m.ws) return DPG_OK;          // nothing has run
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
        cudaFree(m.d_update_tables);
        cudaFree(m.d_tables);
        cudaFree(m.ws);
        cudaFree(m.ws_low);
    }
    if (have_cur) cudaSetDevice(cur);
    cudaGetLastError();
    m.ws = nullptr;
    m.device = -1;
}

int ortho_launch(Matrices& m, const void* update, int32_t update_dtype, const dpg_muon_hparams* hp,
                 const OrthoSchedule& sch, void* out, void* stream, const char* who) {
    OrthoArgs a{};
    std::memcpy(a.st, sch.st, sizeof a.st);
    const WaitFault fault{t_staged_skip, t_staged_timeout_ns > 0 ? uint64_t(t_staged_timeout_ns) : kOrthoWaitNs};
    t_staged_skip = -1;
    t_staged_timeout_ns = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Everything that reads `update` comes before anything that writes `out`,
    // which may share its memory.
    int st = gram_read(m, update, update_dtype, hp, out, s, who);
    if (st != DPG_OK) return st;
    if (m.mats.empty()) return gram_finish(m, update, hp, sch, fault, out, s, who);
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
    a.done = reinterpret_cast<int32_t*>(m.ws + m.o_done);
    a.join = reinterpret_cast<int32_t*>(m.ws + m.o_join);
    a.skip = fault.skip;
    a.wait_ns = fault.wait_ns;
    a.queue = m.d_queue;
    a.queue_first = m.d_queue_first;
    a.ws_low = m.ws_low;
    a.both_steps = sch.both_steps;
    a.n_steps = hp->n_steps;
    a.eps = hp->eps;
    int exp = 0;
    a.eps_frac = float(2.0 * std::frexp(hp->eps, &exp));
    a.eps_exp = exp - 1;
    a.out = static_cast<uint16_t*>(out);
    st = launch_k(a.f32 ? k_ortho_norm<true> : k_ortho_norm<false>, unsigned(m.norm_items.size()), kNormThreads,
                  s, who, a, static_cast<const NormItem*>(m.d_norm_items));
    if (st == DPG_OK)
        st = launch_k(a.f32 ? k_ortho_load<true> : k_ortho_load<false>, unsigned(m.conv_items.size()), 256,
                      a.f32 ? 2 * kLoadSmem : kLoadSmem, s, who, a, static_cast<const ConvItem*>(m.d_conv_items));
    if (st == DPG_OK) st = gram_finish(m, update, hp, sch, fault, out, s, who);
    if (st != DPG_OK) return st;
    CUtensorMap map[2];
    std::memcpy(map, m.maps, sizeof map);
    LowMaps<true> low_maps = {};
    if (m.ws_low) {
        std::memcpy(&low_maps.rows128, m.maps[2], sizeof map[0]);
        std::memcpy(&low_maps.rows64, m.maps[3], sizeof map[0]);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(2 * m.pairs));
    cfg.blockDim = dim3(kOrthoThreads);
    cfg.dynamicSmemBytes = kOrthoSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;   // the pairs wait for one another
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = sch.both_steps > 0 || m.any_both
                              ? cudaLaunchKernelEx(&cfg, k_ortho_steps<true>, a, map[0], map[1], low_maps)
                              : cudaLaunchKernelEx(&cfg, k_ortho_steps<false>, a, map[0], map[1], LowMaps<false>{});
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return fail(DPG_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    }
    return after_launch(who);
}

}  // namespace dpg
