// dpg_norm.cu -- layer norm, its gradients, and the sums of the gain's and the
// bias's gradients over the rows (see dpg_layer_norm and
// dpg_layer_norm_backward in include/dpg.h).
//
// Both passes are streams of HBM traffic: forward 2 + 2 bytes per bf16 element,
// backward 4 + 2.  Forward, a row is held in the registers of a warp (up to 1024
// columns) or of a CTA (up to 32768), so that it is read once: the mean, then the squares
// about it, then the result.  Backward, the rows of a warp (up to 768 columns) or of a CTA
// (up to 16384) lie in shared memory, where they are read twice; registers hold the sums
// over the rows.  Longer rows are read again from L2.  16384 x 4096 bf16: forward 42 us (268
// MB, 6.4 TB/s, 0.94 of the copy's rate), backward 75 (403 MB, 5.4 TB/s), bound by its 25
// instructions an element beside the loads; 8192 x 768 6.4 and 14 to 15.5 (4.6 and 11.3 in a
// loop over one set of rows, which lie in L2), bound by latency and, backward, by the second
// kernel (2.6 us).  Widths that are no multiple of 8 are moved element by element: 9000 x 771
// 14.6 and 26.6, where the bytes would take 4.1 and 6.1.  fp32 16384 x 4096: 102 and 219, of
// 79 and 119.
//
// Backward, a warp or a CTA keeps to the same columns over many rows, and adds
// what each row gives to the gain's and the bias's gradients in registers; at
// the end it leaves its sums in the workspace, and a second kernel adds those in
// order.  The number of parts goes by the sizes alone, so the sums are the same
// bits on every call.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <limits>

#include "dpg_device.cuh"
#include "dpg_host.h"

namespace dpg {

constexpr int64_t kNormMaxSide = int64_t(1) << 30;
constexpr int kNormSms = 152;        // CTAs of a backward pass go by a GB300's SMs (see norm_parts)

struct NormArgs {
    const void* x;
    const void* gain;                // nullable
    const void* bias;                // nullable
    void* y;
    float* mean;                     // nullable with rstd
    float* rstd;
    int64_t rows;
    int32_t cols;
    int32_t params_f32;
    float eps;
};

struct NormBackArgs {
    const void* dy;
    const void* x;
    const void* gain;                // nullable
    const float* mean;
    const float* rstd;
    void* dx;                        // nullable
    float* part;                     // [parts][2][cols]; NULL: no sums
    int64_t rows;
    int32_t cols;
    int32_t params_f32;
    int32_t parts;
};

// ---------------------------------------------------------------------------
// A row in registers: T threads hold V groups of 8 elements each.
//   kRowFull  groups are 8 neighbours, loaded 16 bytes at a time, and fill the row:
//          no bounds to check (a third of the instructions at 4096 columns)
//   kRowVec   the same, the last groups may lie behind the row
//   kRowOdd   the T threads hold neighbouring elements, loaded singly (widths that
//          are no multiple of 8, unaligned buffers)
// ---------------------------------------------------------------------------
enum NormMode : int { kRowOdd = 0, kRowVec = 1, kRowFull = 2 };

template <int MODE, int T>
__device__ __forceinline__ int column_of(int lane, int v, int j) {
    return MODE == kRowOdd ? (v * 8 + j) * T + lane : (lane + v * T) * 8 + j;
}
template <int MODE, int T>
__device__ __forceinline__ bool group_in(int cols, int lane, int v) {
    return MODE == kRowFull || column_of<MODE, T>(lane, v, 0) < cols;
}
// where a thread's columns of a row start
template <bool F32, int MODE>
__device__ __forceinline__ const unsigned char* start_of(const void* p, int64_t row_at, int lane) {
    return static_cast<const unsigned char*>(p) + (row_at + (MODE == kRowOdd ? lane : lane * 8)) * (F32 ? 4 : 2);
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t twice(float x) { return pair_of(x, x); }
__device__ __forceinline__ float sum_of(uint64_t p) {
    const float2 f = halves_of(p);
    return f.x + f.y;
}
__device__ __forceinline__ void unpair(const uint64_t* p, float* f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 t = halves_of(p[j]);
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
    }
}
// s / n, rounded to nearest: a product with inv = 1 / n and one residual (Markstein 1990)
__device__ __forceinline__ float over(float s, float n, float inv) {
    const float q = s * inv;
    const float r = fmaf(fmaf(-q, n, s), inv, q);
    return fabsf(q) < 3.4e38f ? r : q;            // (not of an infinity)
}
// 1 / sqrt(v) within an ulp: the approximation and one of Newton's steps
__device__ __forceinline__ float inverse_root(float v) {
    const float r = rsqrtf(v);
    const float e = fmaf(-v * r, r, 1.0f);
    return r > 0.0f && r < 3.4e38f ? fmaf(0.5f * r, e, r) : r;
}

template <bool F32>
struct NormRaw {
    uint4 q[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ void widen_pairs(const NormRaw<F32>& r, uint64_t* p) {
    if (F32) {
        const uint4 a = r.q[0], b = r.q[F32 ? 1 : 0];
        p[0] = pair_of(__uint_as_float(a.x), __uint_as_float(a.y));
        p[1] = pair_of(__uint_as_float(a.z), __uint_as_float(a.w));
        p[2] = pair_of(__uint_as_float(b.x), __uint_as_float(b.y));
        p[3] = pair_of(__uint_as_float(b.z), __uint_as_float(b.w));
    } else {
        float f[8];
        widen8(r.q[0], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = pair_of(f[2 * j], f[2 * j + 1]);
    }
}

// Group v of a row whose columns of this thread start at p; zeros behind the last.
// (Plain loads: the output may be the input.)
template <bool F32, int MODE, int T>
__device__ __forceinline__ NormRaw<F32> load_group(const unsigned char* p, int cols, int lane, int v) {
    NormRaw<F32> r;
    if (MODE != kRowOdd) {
        const unsigned char* at = p + v * T * 8 * (F32 ? 4 : 2);
        const bool in = group_in<MODE, T>(cols, lane, v);
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); ++k) {
            r.q[k] = make_uint4(0, 0, 0, 0);
            if (in)
                asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(r.q[k].x), "=r"(r.q[k].y), "=r"(r.q[k].z), "=r"(r.q[k].w)
                             : "l"(at + 16 * k));
        }
    } else {
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            e[j] = column_of<kRowOdd, T>(lane, v, j) >= cols ? 0u
                   : F32 ? *(reinterpret_cast<const volatile uint32_t*>(p) + (v * 8 + j) * T)
                         : uint32_t(*(reinterpret_cast<const volatile uint16_t*>(p) + (v * 8 + j) * T));
        }
        if (F32) {
            r.q[0] = make_uint4(e[0], e[1], e[2], e[3]);
            r.q[F32 ? 1 : 0] = make_uint4(e[4], e[5], e[6], e[7]);
        } else {
            r.q[0] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
        }
    }
    return r;
}

// Zeroes what lies behind the last column: the whole group, or single elements.
template <int MODE, int T>
__device__ __forceinline__ void mask_group(int cols, int lane, int v, uint64_t* p) {
    if (MODE == kRowVec) {
        if (!group_in<kRowVec, T>(cols, lane, v)) p[0] = p[1] = p[2] = p[3] = 0;
    } else if (MODE == kRowOdd) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = halves_of(p[j]);
            p[j] = pair_of(column_of<kRowOdd, T>(lane, v, 2 * j) < cols ? t.x : 0.0f,
                           column_of<kRowOdd, T>(lane, v, 2 * j + 1) < cols ? t.y : 0.0f);
        }
    }
}

template <bool F32, int MODE, int T>
__device__ __forceinline__ void store_group(unsigned char* p, int cols, int lane, int v, const uint64_t* pairs) {
    float f[8];
    unpair(pairs, f);
    if (MODE != kRowOdd) {
        if (!group_in<MODE, T>(cols, lane, v)) return;
        unsigned char* at = p + v * T * 8 * (F32 ? 4 : 2);
        if (F32) {
            st_u4(at, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
            st_u4(at + 16, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
        } else {
            st_u4(at, narrow8(f));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (column_of<kRowOdd, T>(lane, v, j) >= cols) continue;
            if (F32) reinterpret_cast<float*>(p)[(v * 8 + j) * T] = f[j];
            else reinterpret_cast<__nv_bfloat16*>(p)[(v * 8 + j) * T] = __float2bfloat16_rn(f[j]);
        }
    }
}

// Group v of a gain or bias of bf16 or fp32 (PF32); these stay in L1 from row to row.
template <bool PF32, int MODE, int T>
__device__ __forceinline__ void load_params(const void* p, int cols, int lane, int v, uint64_t* out) {
    NormRaw<PF32> r;
    if (MODE != kRowOdd) {
        const bool in = group_in<MODE, T>(cols, lane, v);
        const uint4* at = reinterpret_cast<const uint4*>(start_of<PF32, MODE>(p, 0, lane) + v * T * 8 * (PF32 ? 4 : 2));
#pragma unroll
        for (int k = 0; k < (PF32 ? 2 : 1); ++k) r.q[k] = in ? __ldg(at + k) : make_uint4(0, 0, 0, 0);
        widen_pairs<PF32>(r, out);
    } else {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column_of<kRowOdd, T>(lane, v, j);
            f[j] = c >= cols ? 0.0f
                   : PF32    ? __ldg(static_cast<const float*>(p) + c)
                             : __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(p) + c)) << 16);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = pair_of(f[2 * j], f[2 * j + 1]);
    }
}

// Sum over the T threads of a row, the same in all of them.  `sh` holds a value
// per warp and is free again after the next call's barrier (calls alternate
// between two).
template <int T>
__device__ __forceinline__ float row_sum(float a, float* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    if (T == 32) return a;
    constexpr int kWarps = T / 32;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = a;
    __syncthreads();
    a = sh[threadIdx.x & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    return a;
}
// The same for two sums (2 values per warp in `sh`): lanes 0 .. 15 add up a, the
// others b, at half the exchanges.
template <int T>
__device__ __forceinline__ float2 row_sums(float a, float b, float* sh) {
    const bool low = (threadIdx.x & 16) == 0;
    float t = (low ? a : b) + __shfl_xor_sync(0xFFFFFFFFu, low ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    if (T > 32) {
        constexpr int kWarps = T / 32, kLanes = kWarps < 16 ? kWarps : 16;
        if ((threadIdx.x & 15) == 0) sh[(threadIdx.x >> 5) + (low ? 0 : kWarps)] = t;
        __syncthreads();
        const float* from = sh + (low ? 0 : kWarps);
        t = from[threadIdx.x & (kLanes - 1)];
        if (kWarps > 16) t += from[16 + (threadIdx.x & 15)];
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
    const float other = __shfl_xor_sync(0xFFFFFFFFu, t, 16);
    return low ? make_float2(t, other) : make_float2(other, t);
}

// Four sums over the 256 threads of a CTA (32 values in `sh`): each quarter of a warp
// adds up one of them.
__device__ __forceinline__ float4 row_sums4(float a, float b, float c, float d, float* sh) {
    const bool low = (threadIdx.x & 16) == 0, even = (threadIdx.x & 8) == 0;
    const float x = (low ? a : c) + __shfl_xor_sync(0xFFFFFFFFu, low ? c : a, 16);
    const float y = (low ? b : d) + __shfl_xor_sync(0xFFFFFFFFu, low ? d : b, 16);
    float t = (even ? x : y) + __shfl_xor_sync(0xFFFFFFFFu, even ? y : x, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    const int quarter = int(threadIdx.x & 31) >> 3;
    if ((threadIdx.x & 7) == 0) sh[quarter * 8 + (threadIdx.x >> 5)] = t;
    __syncthreads();
    t = sh[quarter * 8 + (threadIdx.x & 7)];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    return make_float4(__shfl_sync(0xFFFFFFFFu, t, 0), __shfl_sync(0xFFFFFFFFu, t, 8), __shfl_sync(0xFFFFFFFFu, t, 16),
                       __shfl_sync(0xFFFFFFFFu, t, 24));
}

template <int T>
constexpr int norm_threads() { return T == 32 ? 256 : T; }

// CTAs to an SM: as many as leave the registers of a row and of the next
template <bool F32, int T, int V>
constexpr int norm_ctas() {
    return T == 32 ? (V == 1 ? 4 : F32 && V > 2 ? 2 : 3) : T == 1024 ? 1 : (V <= 2 ? 1024 : F32 ? 512 : 768) / T;
}

// y = x * rstd, times the gain, plus the bias; which of them there are, and their
// type, is known to the instance (a branch to every group cost an instruction an
// element)
template <bool F32, int MODE, int T, int V, bool GAIN, bool BIAS, bool PF32>
__device__ __forceinline__ void finish_row(const NormArgs& a, int lane, uint64_t (*x)[4], float rstd, unsigned char* y) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        uint64_t g[4], b[4] = {0, 0, 0, 0};
        if (GAIN) load_params<PF32, MODE, T>(a.gain, a.cols, lane, v, g);
        if (BIAS) load_params<PF32, MODE, T>(a.bias, a.cols, lane, v, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[v][j] = mul2(x[v][j], twice(rstd));
            if (GAIN) x[v][j] = BIAS ? fma2(x[v][j], g[j], b[j]) : mul2(x[v][j], g[j]);
            else if (BIAS) x[v][j] = add2(x[v][j], b[j]);
        }
        store_group<F32, MODE, T>(y, a.cols, lane, v, x[v]);
    }
}

// Warps (T = 32) or CTAs stay and take row after row; the next is on its way while
// one is worked on.  (A CTA to every row or eight spent half its time on its start
// and on loads of the parameters behind the statistics.)
template <bool F32, int MODE, int T, int V>
__global__ void __launch_bounds__(norm_threads<T>(), norm_ctas<F32, T, V>()) k_layer_norm(const __grid_constant__ NormArgs a) {
    __shared__ float sh[2][64];
    pdl_enter();
    constexpr int kSize = F32 ? 4 : 2;
    const int lane = int(threadIdx.x) % T;
    const int64_t first = int64_t(blockIdx.x) * (norm_threads<T>() / T) + int(threadIdx.x) / T;
    const int64_t step = int64_t(gridDim.x) * (norm_threads<T>() / T), skip = step * a.cols * kSize;
    const unsigned char* from = start_of<F32, MODE>(a.x, first * a.cols, lane);
    unsigned char* to = const_cast<unsigned char*>(start_of<F32, MODE>(a.y, first * a.cols, lane));
    const int kind = (a.gain ? 1 : 0) + (a.bias ? 2 : 0) + (a.params_f32 ? 4 : 0);
    const float n = float(a.cols), inv = 1.0f / n;
    NormRaw<F32> raw[V];
    if (first < a.rows) {
#pragma unroll
        for (int v = 0; v < V; ++v) raw[v] = load_group<F32, MODE, T>(from, a.cols, lane, v);
    }
    for (int64_t r = first; r < a.rows; r += step) {
        uint64_t x[V][4], s = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            widen_pairs<F32>(raw[v], x[v]);
#pragma unroll
            for (int j = 0; j < 4; ++j) s = add2(s, x[v][j]);
        }
        from += skip;
        if (r + step < a.rows) {
#pragma unroll
            for (int v = 0; v < V; ++v) raw[v] = load_group<F32, MODE, T>(from, a.cols, lane, v);
        }
        const float mean = over(row_sum<T>(sum_of(s), sh[0]), n, inv);
        s = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[v][j] = add2(x[v][j], twice(-mean));
            mask_group<MODE, T>(a.cols, lane, v, x[v]);
#pragma unroll
            for (int j = 0; j < 4; ++j) s = fma2(x[v][j], x[v][j], s);
        }
        const float rstd = inverse_root(over(row_sum<T>(sum_of(s), sh[1]), n, inv) + a.eps);
        if (lane == 0 && a.mean) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
        switch (kind) {
            case 1: finish_row<F32, MODE, T, V, true, false, false>(a, lane, x, rstd, to); break;
            case 2: finish_row<F32, MODE, T, V, false, true, false>(a, lane, x, rstd, to); break;
            case 3: finish_row<F32, MODE, T, V, true, true, false>(a, lane, x, rstd, to); break;
            case 5: finish_row<F32, MODE, T, V, true, false, true>(a, lane, x, rstd, to); break;
            case 6: finish_row<F32, MODE, T, V, false, true, true>(a, lane, x, rstd, to); break;
            case 7: finish_row<F32, MODE, T, V, true, true, true>(a, lane, x, rstd, to); break;
            default: finish_row<F32, MODE, T, V, false, false, false>(a, lane, x, rstd, to); break;
        }
        to += skip;
    }
}

__device__ __forceinline__ float load_one(const void* p, int32_t f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
}

// The same for rows of any length, read three times.  A thread adds at most 128 terms in
// fp32, and such sums in 64 bits: one chain of 2^14 equal terms is off by 1e-4 of its sum
// (rows of 2^24 columns), since each addition to a long sum may be rounded the same way.
constexpr int kLongThreads = 1024;
constexpr int kChain = 128;
template <bool F32, typename A>
__device__ __forceinline__ float long_sum(const void* p, int64_t at, int cols, A add) {
    double sum = 0.0;
    for (int c = int(threadIdx.x); c < cols;) {
        const int end = min(cols, c + kChain * kLongThreads);
        float s = 0.0f;
#pragma unroll 8
        for (; c < end; c += kLongThreads) s = add(s, load_one(p, F32, at + c));
        sum += double(s);
    }
    return float(sum);
}
__device__ __forceinline__ void store_one(void* p, int32_t f32, int64_t i, float v) {
    if (f32) static_cast<float*>(p)[i] = v;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

template <bool F32>
__global__ void __launch_bounds__(kLongThreads) k_layer_norm_long(const __grid_constant__ NormArgs a) {
    __shared__ float sh[2][64];
    pdl_enter();
    const int64_t at = int64_t(blockIdx.x) * a.cols;
    const auto add = [](float s, float x) { return s + x; };
    const float sum = long_sum<F32>(a.x, at, a.cols, add);
    const float mean = row_sum<kLongThreads>(sum, sh[0]) / float(a.cols);
    const auto square = [mean](float s, float x) { return fmaf(x - mean, x - mean, s); };
    const float squares = long_sum<F32>(a.x, at, a.cols, square);
    const float rstd = 1.0f / sqrtf(row_sum<kLongThreads>(squares, sh[1]) / float(a.cols) + a.eps);
    if (threadIdx.x == 0 && a.mean) {
        a.mean[blockIdx.x] = mean;
        a.rstd[blockIdx.x] = rstd;
    }
    for (int c = int(threadIdx.x); c < a.cols; c += kLongThreads) {
        float v = (load_one(a.x, F32, at + c) - mean) * rstd;
        if (a.gain) v *= load_one(a.gain, a.params_f32, c);
        if (a.bias) v += load_one(a.bias, a.params_f32, c);
        store_one(a.y, F32, at + c, v);
    }
}

// ---------------------------------------------------------------------------
// Backward.  CTA p takes rows p, p + parts, ... (T = 32: its eight warps take
// eight rows at a time).  A thread's groups of x and dy come through shared memory,
// one to four rows ahead (asynchronous copies, which only the thread itself waits for):
// a second set of registers for the next row left one CTA to an SM.
// ---------------------------------------------------------------------------
// CTAs of 256 threads with bf16 rows take two rows at a time: one exchange of sums for both
// (16384 x 4096 83 -> 75 us, 2048 columns 50 either way)
template <bool F32, int MODE, int T>
constexpr bool row_pairs() { return !F32 && MODE != kRowOdd && T == 256; }

// rows ahead: 128 KB to a row of 16384 fp32 columns leave one; two to a warp (8192 x 768 not
// in L2 13.1 us, with three 14.1), which leave room for two CTAs of fp32 rows
template <bool F32, int T, int V>
constexpr int rows_ahead() { return !F32 && T == 256 ? 4 : F32 && T * V == 2048 ? 1 : T == 32 ? 2 : 3; }

template <bool F32, int T, int V>
constexpr int back_smem() { return rows_ahead<F32, T, V>() * norm_threads<T>() * V * 2 * (F32 ? 32 : 16); }

template <bool F32, int MODE, int T, int V>
struct BackRows {
    uint4* own;                                    // this thread's first piece in shared memory
    const unsigned char *x, *dy;                   // its columns of the row to fetch next (kRowOdd: of the row at hand)
    NormRaw<F32> direct[MODE == kRowOdd ? 2 * V : 1]; // odd widths and unaligned rows: loaded as they are needed
    static constexpr int kPieces = F32 ? 2 : 1, kThreads = norm_threads<T>(), kAhead = rows_ahead<F32, T, V>();
    static constexpr int kSlot = 2 * V * kPieces * kThreads;

    // piece k of group v of x (0) or dy (1) of slot s; neighbouring threads' pieces are neighbours
    __device__ __forceinline__ uint4* piece(int s, int which, int v, int k) const {
        return own + s * kSlot + ((which * V + v) * kPieces + k) * kThreads;
    }
    __device__ __forceinline__ void fetch(const NormBackArgs& a, bool more, int s, int lane, int64_t skip) {
        if (MODE == kRowOdd) return;
        if (more) {
            const uint32_t to = uint32_t(__cvta_generic_to_shared(piece(s, 0, 0, 0)));
#pragma unroll
            for (int which = 0; which < 2; ++which)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (group_in<MODE, T>(a.cols, lane, v))
#pragma unroll
                        for (int k = 0; k < kPieces; ++k)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                         :: "r"(to + ((which * V + v) * kPieces + k) * kThreads * 16),
                                            "l"((which ? dy : x) + v * T * 8 * (F32 ? 4 : 2) + 16 * k) : "memory");
            x += skip;
            dy += skip;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void arrive(const NormBackArgs& a, int lane, int64_t skip) {
        if (MODE != kRowOdd) {
            asm volatile("cp.async.wait_group %0;" :: "n"(kAhead - (row_pairs<F32, MODE, T>() ? 2 : 1)) : "memory");
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                direct[2 * v] = load_group<F32, kRowOdd, T>(x, a.cols, lane, v);
                direct[2 * v + 1] = load_group<F32, kRowOdd, T>(dy, a.cols, lane, v);
            }
            x += skip;
            dy += skip;
        }
    }
    __device__ __forceinline__ void get(const NormBackArgs& a, int s, int which, int lane, int v, uint64_t* f) const {
        NormRaw<F32> raw;
        if (MODE != kRowOdd) {
            const bool in = group_in<MODE, T>(a.cols, lane, v);
#pragma unroll
            for (int k = 0; k < kPieces; ++k) raw.q[k] = in ? *piece(s, which, v, k) : make_uint4(0, 0, 0, 0);
        } else {
            raw = direct[MODE == kRowOdd ? 2 * v + which : 0];
        }
        widen_pairs<F32>(raw, f);
    }
};

// A row's sums: what it adds to the gradients, and (in pairs) the sums of g and g n.
// With `keep`, x - mean and g stay in d and g.
template <bool F32, int MODE, int T, int V, int GAIN>
__device__ __forceinline__ void back_sums(const NormBackArgs& a, const BackRows<F32, MODE, T, V>& rows, int s, int lane,
                                          float mean, float rstd, uint64_t (*dg)[4], uint64_t (*db)[4], uint64_t* d,
                                          uint64_t* g, uint64_t& s1, uint64_t& s2) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        uint64_t gain[4];
        rows.get(a, s, 0, lane, v, d);
        rows.get(a, s, 1, lane, v, g);
        if (GAIN) load_params<GAIN == 2, MODE, T>(a.gain, a.cols, lane, v, gain);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = add2(d[j], twice(-mean));
        mask_group<MODE, T>(a.cols, lane, v, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t n = mul2(d[j], twice(rstd));
            dg[v][j] = fma2(g[j], n, dg[v][j]);
            db[v][j] = add2(db[v][j], g[j]);
            if (GAIN) g[j] = mul2(g[j], gain[j]);
            s1 = add2(s1, g[j]);
            s2 = fma2(g[j], n, s2);
        }
    }
}

// dx = (g - (x - mean) (rstd c2)) rstd - rstd c1; `KEPT`: d and g hold x - mean and g.  (The
// square of rstd would leave fp32 from 1.8e19 on, where deviations are below 5e-20.)
template <bool F32, int MODE, int T, int V, int GAIN, bool KEPT>
__device__ __forceinline__ void back_row(const NormBackArgs& a, const BackRows<F32, MODE, T, V>& rows, int s, int lane,
                                         float mean, float rstd, float c1, float c2, uint64_t* d, uint64_t* g,
                                         unsigned char* dx) {
    const uint64_t k1 = twice(-rstd * c1), k2 = twice(-rstd * c2), k = twice(rstd);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (!KEPT) {                               // (from shared memory again: registers hold the sums)
            uint64_t gain[4];
            rows.get(a, s, 0, lane, v, d);
            rows.get(a, s, 1, lane, v, g);
            if (GAIN) load_params<GAIN == 2, MODE, T>(a.gain, a.cols, lane, v, gain);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[j] = add2(d[j], twice(-mean));
                if (GAIN) g[j] = mul2(g[j], gain[j]);
            }
        }
        uint64_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = fma2(fma2(d[j], k2, g[j]), k, k1);
        store_group<F32, MODE, T>(dx, a.cols, lane, v, out);
    }
}

// eight neighbouring sums; workspaces start on 16-byte boundaries, most on 32-byte ones
__device__ __forceinline__ void store_sums(float* to, const float* sums) {
    if ((reinterpret_cast<uintptr_t>(to) & 31) == 0) {
        F8 f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f.v[j] = sums[j];
        st_f8(to, f);
    } else {
        *reinterpret_cast<float4*>(to) = make_float4(sums[0], sums[1], sums[2], sums[3]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(sums[4], sums[5], sums[6], sums[7]);
    }
}

template <bool F32, int MODE, int T, int V>
__global__ void __launch_bounds__(norm_threads<T>(), T == 32 ? 2 : T <= 256 ? (V == 1 ? 4 : 3) : 1)
k_layer_norm_back(const __grid_constant__ NormBackArgs a) {
    constexpr int kRows = norm_threads<T>() / T;   // rows of a CTA at a time
    constexpr int kAhead = rows_ahead<F32, T, V>(), kSize = F32 ? 4 : 2;
    constexpr bool kKeep = V == 1;                 // more would not fit beside the sums
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float sh[2][64];
    pdl_enter();
    const int lane = int(threadIdx.x) % T, group = int(threadIdx.x) / T;
    const int64_t first = int64_t(blockIdx.x) * kRows + group, step = int64_t(gridDim.x) * kRows;
    const int64_t skip = step * a.cols * kSize;
    const int gain = a.gain ? a.params_f32 ? 2 : 1 : 0;
    BackRows<F32, MODE, T, V> rows;
    rows.own = reinterpret_cast<uint4*>(dyn) + threadIdx.x;
    rows.x = start_of<F32, MODE>(a.x, first * a.cols, lane);
    rows.dy = start_of<F32, MODE>(a.dy, first * a.cols, lane);
    unsigned char* to = const_cast<unsigned char*>(start_of<F32, MODE>(a.dx, first * a.cols, lane));
    for (int s = 0; s < kAhead; ++s) rows.fetch(a, first + s * step < a.rows, s, lane, skip);
    uint64_t dg[V][4], db[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[v][j] = db[v][j] = 0;
    const float n = float(a.cols), inv = 1.0f / n;
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (first < a.rows) {
        next_mean = __ldg(a.mean + first);
        next_rstd = __ldg(a.rstd + first);
    }
    int half = 0, s = 0;
    if constexpr (row_pairs<F32, MODE, T>()) {
        float after_mean = 0.0f, after_rstd = 0.0f;
        if (first + step < a.rows) {
            after_mean = __ldg(a.mean + first + step);
            after_rstd = __ldg(a.rstd + first + step);
        }
        for (int64_t r = first; r < a.rows; r += 2 * step, half ^= 1) {
            const float mean0 = next_mean, rstd0 = next_rstd, mean1 = after_mean, rstd1 = after_rstd;
            if (r + 2 * step < a.rows) {
                next_mean = __ldg(a.mean + r + 2 * step);
                next_rstd = __ldg(a.rstd + r + 2 * step);
            }
            if (r + 3 * step < a.rows) {
                after_mean = __ldg(a.mean + r + 3 * step);
                after_rstd = __ldg(a.rstd + r + 3 * step);
            }
            rows.arrive(a, lane, skip);
            const int two = r + step < a.rows ? 2 : 1;
            float t0 = 0.0f, t1 = 0.0f, t2 = 0.0f, t3 = 0.0f;
#pragma unroll 1
            for (int u = 0; u < two; ++u) {
                const float mean = u ? mean1 : mean0, rstd = u ? rstd1 : rstd0;
                uint64_t s1 = 0, s2 = 0, d[4], g[4];
                if (gain == 1) back_sums<F32, MODE, T, V, 1>(a, rows, s + u, lane, mean, rstd, dg, db, d, g, s1, s2);
                else if (gain == 2) back_sums<F32, MODE, T, V, 2>(a, rows, s + u, lane, mean, rstd, dg, db, d, g, s1, s2);
                else back_sums<F32, MODE, T, V, 0>(a, rows, s + u, lane, mean, rstd, dg, db, d, g, s1, s2);
                t0 = t2, t1 = t3;
                t2 = sum_of(s1), t3 = sum_of(s2);
            }
            if (two == 1) t0 = t2, t1 = t3;
            if (a.dx) {
                const float4 t = row_sums4(t0, t1, t2, t3, sh[half]);
#pragma unroll 1
                for (int u = 0; u < two; ++u) {
                    const float mean = u ? mean1 : mean0, rstd = u ? rstd1 : rstd0;
                    const float c1 = over(u ? t.z : t.x, n, inv), c2 = over(u ? t.w : t.y, n, inv);
                    uint64_t d[4], g[4];
                    if (gain == 0) back_row<F32, MODE, T, V, 0, false>(a, rows, s + u, lane, mean, rstd, c1, c2, d, g, to);
                    else if (gain == 1) back_row<F32, MODE, T, V, 1, false>(a, rows, s + u, lane, mean, rstd, c1, c2, d, g, to);
                    else back_row<F32, MODE, T, V, 2, false>(a, rows, s + u, lane, mean, rstd, c1, c2, d, g, to);
                    to += skip;
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) rows.fetch(a, r + (kAhead + u) * step < a.rows, s + u, lane, skip);
            s ^= 2;                                // of four slots
        }
    } else {
        for (int64_t r = first; r < a.rows; r += step, half ^= 1) {
            const float mean = next_mean, rstd = next_rstd;
            if (r + step < a.rows) {
                next_mean = __ldg(a.mean + r + step);
                next_rstd = __ldg(a.rstd + r + step);
            }
            rows.arrive(a, lane, skip);
            uint64_t s1 = 0, s2 = 0, d[4], g[4];
            if (gain == 1) back_sums<F32, MODE, T, V, 1>(a, rows, s, lane, mean, rstd, dg, db, d, g, s1, s2);
            else if (gain == 2) back_sums<F32, MODE, T, V, 2>(a, rows, s, lane, mean, rstd, dg, db, d, g, s1, s2);
            else back_sums<F32, MODE, T, V, 0>(a, rows, s, lane, mean, rstd, dg, db, d, g, s1, s2);
            if (a.dx) {
                const float2 t = row_sums<T>(sum_of(s1), sum_of(s2), sh[half]);
                const float c1 = over(t.x, n, inv), c2 = over(t.y, n, inv);
                if (kKeep || gain == 0) back_row<F32, MODE, T, V, 0, kKeep>(a, rows, s, lane, mean, rstd, c1, c2, d, g, to);
                else if (gain == 1) back_row<F32, MODE, T, V, 1, false>(a, rows, s, lane, mean, rstd, c1, c2, d, g, to);
                else back_row<F32, MODE, T, V, 2, false>(a, rows, s, lane, mean, rstd, c1, c2, d, g, to);
                to += skip;
            }
            rows.fetch(a, r + kAhead * step < a.rows, s, lane, skip);
            s = s + 1 == kAhead ? 0 : s + 1;
        }
    }
    if (!a.part) return;
    float dgf[V][8], dbf[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        unpair(dg[v], dgf[v]);
        unpair(db[v], dbf[v]);
    }
    float* out = a.part + int64_t(blockIdx.x) * 2 * a.cols;
    if (T == 32) {                                 // the warps' sums, in order
        if (MODE != kRowOdd) asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        constexpr int kSums = T * V * 8;
        static_assert(T > 32 || back_smem<F32, T, V>() >= 2 * kRows * kSums * 4, "room for the warps' sums");
        float* sums = reinterpret_cast<float*>(dyn);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sums[(group * 2) * kSums + (v * 8 + j) * 32 + lane] = dgf[v][j];
                sums[(group * 2 + 1) * kSums + (v * 8 + j) * 32 + lane] = dbf[v][j];
            }
        __syncthreads();
        for (int k = int(threadIdx.x); k < 2 * kSums; k += norm_threads<T>()) {
            const int at = k % kSums, c = column_of<MODE, T>(at & 31, at >> 8, (at >> 5) & 7);
            if (c >= a.cols) continue;
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < kRows; ++w) t += sums[w * 2 * kSums + k];
            out[(k / kSums) * int64_t(a.cols) + c] = t;
        }
    } else if (MODE != kRowOdd) {                  // (one by one, 32 bytes apart, took 4 us of 64 rows of 4096)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (group_in<MODE, T>(a.cols, lane, v)) {
                float* at = out + column_of<MODE, T>(lane, v, 0);
                store_sums(at, dgf[v]);
                store_sums(at + a.cols, dbf[v]);
            }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = column_of<MODE, T>(lane, v, j);
                if (c < a.cols) {
                    out[c] = dgf[v][j];
                    out[a.cols + c] = dbf[v][j];
                }
            }
    }
}

// W neighbouring elements: 8 on a 16-byte boundary, or one.  (Plain loads: the output
// may be the input.)
template <int W>
__device__ __forceinline__ void load_some(const void* p, int32_t f32, int64_t i, float* v) {
    if constexpr (W == 1) {
        v[0] = load_one(p, f32, i);
    } else if (f32) {
        const NormRaw<true> r = load_group<true, kRowFull, 1>(static_cast<const unsigned char*>(p) + i * 4, 0, 0, 0);
        uint64_t f[4];
        widen_pairs<true>(r, f);
        unpair(f, v);
    } else {
        const NormRaw<false> r = load_group<false, kRowFull, 1>(static_cast<const unsigned char*>(p) + i * 2, 0, 0, 0);
        uint64_t f[4];
        widen_pairs<false>(r, f);
        unpair(f, v);
    }
}

// Rows of any length: first the sums, CTA (columns, part) over rows part,
// part + parts, ...; then dx, which may take the place of dy or x.  W: neighbouring
// columns to a thread (4000 x 20000 bf16, both kernels, 210 us with eight; 365 with one and rows on 1024
// threads, of which one CTA fits an SM).
template <int W>
__global__ void __launch_bounds__(256) k_layer_norm_columns(const __grid_constant__ NormBackArgs a, int32_t f32) {
    pdl_enter();
    const int64_t c = (int64_t(blockIdx.x) * 256 + threadIdx.x) * W;
    if (c >= a.cols) return;
    float dg[W] = {}, db[W] = {};
#pragma unroll 2
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        float y[W], x[W];
        load_some<W>(a.dy, f32, r * a.cols + c, y);
        load_some<W>(a.x, f32, r * a.cols + c, x);
        const float mean = __ldg(a.mean + r), rstd = __ldg(a.rstd + r);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            dg[j] = fmaf(y[j], (x[j] - mean) * rstd, dg[j]);
            db[j] += y[j];
        }
    }
    float* out = a.part + int64_t(blockIdx.y) * 2 * a.cols + c;
    if constexpr (W == 1) {
        out[0] = dg[0];
        out[a.cols] = db[0];
    } else {
        store_sums(out, dg);
        store_sums(out + a.cols, db);
    }
}

constexpr int kDxThreads = 512;
// a thread's sums of g and g n over a row, 128 terms in fp32 at a time as in long_sum
template <int W, bool F32, int GAIN>
__device__ __forceinline__ float2 dx_sums(const NormBackArgs& a, int64_t at, float mean, float rstd) {
    double sum1 = 0.0, sum2 = 0.0;
    for (int c = int(threadIdx.x) * W; c < a.cols;) {
        const int end = min(a.cols, c + kChain * kDxThreads);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll (W == 1 ? 4 : 1)
        for (; c < end; c += kDxThreads * W) {
            float g[W], x[W], k[W];
            load_some<W>(a.dy, F32, at + c, g);
            load_some<W>(a.x, F32, at + c, x);
            if (GAIN) load_some<W>(a.gain, GAIN == 2, c, k);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (GAIN) g[j] *= k[j];
                s1 += g[j];
                s2 = fmaf(g[j], (x[j] - mean) * rstd, s2);
            }
        }
        sum1 += double(s1);
        sum2 += double(s2);
    }
    return make_float2(float(sum1), float(sum2));
}

template <int W, bool F32>
__global__ void __launch_bounds__(kDxThreads, F32 ? 2 : 3) k_layer_norm_dx_long(const __grid_constant__ NormBackArgs a) {
    __shared__ float sh[64];
    pdl_enter();
    const int64_t r = blockIdx.x, at = r * a.cols;
    const float mean = __ldg(a.mean + r), rstd = __ldg(a.rstd + r);
    float2 t = !a.gain ? dx_sums<W, F32, 0>(a, at, mean, rstd) : a.params_f32 ? dx_sums<W, F32, 2>(a, at, mean, rstd)
                                                                              : dx_sums<W, F32, 1>(a, at, mean, rstd);
    t = row_sums<kDxThreads>(t.x, t.y, sh);
    const float c1 = t.x / float(a.cols), c2 = t.y / float(a.cols);
    for (int64_t c = int64_t(threadIdx.x) * W; c < a.cols; c += kDxThreads * W) {
        float g[W], x[W], k[W];
        load_some<W>(a.dy, F32, at + c, g);
        load_some<W>(a.x, F32, at + c, x);
        if (a.gain) load_some<W>(a.gain, a.params_f32, c, k);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (a.gain) g[j] *= k[j];
            g[j] = rstd * (g[j] - c1 - (x[j] - mean) * rstd * c2);
        }
        if constexpr (W == 1) {
            store_one(a.dx, F32, at + c, g[0]);
        } else if constexpr (F32) {
            float* to = static_cast<float*>(a.dx) + at + c;
            *reinterpret_cast<float4*>(to) = make_float4(g[0], g[1], g[2], g[3]);
            *reinterpret_cast<float4*>(to + 4) = make_float4(g[4], g[5], g[6], g[7]);
        } else {
            st_u4(static_cast<unsigned char*>(a.dx) + (at + c) * 2, narrow8(g));
        }
    }
}

// Adds the parts in order: 32 columns to a CTA, 16 threads to a column, then
// their sums along a fixed tree.  (32 threads: 512 x 4096 12.8 us instead of 8.4, more
// of 12000 columns 2 us more; 16384 x 4096 0.7 less.)
// MANY (more than 4096 parts): no chain is longer than 256 of them; to look for the end of one
// costs few parts 2 us (8192 x 768 19.5 -> 21.5 us with the rows' kernel).
struct NormSumArgs {
    const float* part;
    void* out[2];                  // dgain, dbias (either may be NULL)
    int32_t parts, cols, f32, add;
};
constexpr int kSumRows = 16;
template <bool MANY>
__global__ void __launch_bounds__(32 * kSumRows) k_layer_norm_sums(const __grid_constant__ NormSumArgs a) {
    __shared__ float sh[kSumRows][33];
    pdl_enter();
    const int64_t c = int64_t(blockIdx.x) * 32 + (threadIdx.x & 31);
    const int which = blockIdx.y, row = int(threadIdx.x >> 5);
    if (!a.out[which]) return;
    constexpr int kFly = 8;                        // loads in flight
    float s = 0.0f, before = 0.0f;
    int n = 0;
    if (c < a.cols)
        for (int p = row; p < a.parts; p += kSumRows * kFly) {
            float t[kFly];
#pragma unroll
            for (int u = 0; u < kFly; ++u)
                t[u] = p + kSumRows * u < a.parts ? __ldcg(a.part + (int64_t(p + kSumRows * u) * 2 + which) * a.cols + c) : 0.0f;
#pragma unroll
            for (int u = 0; u < kFly; ++u) s += t[u];
            if (MANY && ++n == 256 / kFly) {
                before += s;
                s = 0.0f;
                n = 0;
            }
        }
    if (MANY) s += before;
    sh[row][threadIdx.x & 31] = s;
    __syncthreads();
    const int part = int(threadIdx.x) % kSumRows;      // kSumRows neighbouring threads add up a column
    s = sh[part][threadIdx.x / kSumRows];
#pragma unroll
    for (int o = kSumRows / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int64_t mine = int64_t(blockIdx.x) * 32 + threadIdx.x / kSumRows;
    if (part != 0 || mine >= a.cols) return;
    if (a.f32) {
        float* p = static_cast<float*>(a.out[which]) + mine;
        *p = a.add ? *p + s : s;
    } else {
        static_cast<__nv_bfloat16*>(a.out[which])[mine] = __float2bfloat16_rn(s);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static int norm_shape(int64_t rows, int64_t cols, int32_t dtype, int32_t param_dtype, const char* who) {
    if (rows < 0 || cols < 0 || rows > kNormMaxSide || cols > kNormMaxSide)
        return fail(DPG_ERR_INVALID_ARG, "%s: %lld x %lld outside [0, 2^30]", who, (long long)rows, (long long)cols);
    if (dtype != DPG_BF16 && dtype != DPG_F32) return fail(DPG_ERR_INVALID_ARG, "%s: dtype %d unknown", who, dtype);
    if (param_dtype != DPG_BF16 && param_dtype != DPG_F32)
        return fail(DPG_ERR_INVALID_ARG, "%s: param_dtype %d unknown", who, param_dtype);
    return DPG_OK;
}

static int norm_pointer(const void* p, int32_t dtype, bool may_be_null, const char* name, const char* who) {
    if (!p && !may_be_null) return fail(DPG_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
    if (!aligned(p, dtype == DPG_BF16 ? 2 : 4)) return fail(DPG_ERR_MISALIGNED, "%s: %s misaligned", who, name);
    return DPG_OK;
}

// CTAs of a backward pass, which leave as many parts: as many as the SMs hold at a
// time.  With sums and few rows fewer: a part costs 16 bytes a column (written, and
// read again), a CTA's next row a latency and its own bytes; both sums are equal at
// the root of rows (110000 / cols + 20) parts (512 x 4096: 152 parts 7.8 us, 456 parts
// 12.8 with sums, 4.7 and 3.4 without).  And no more than leave the same number of
// rows to the longest.  With so many rows that a thread would add more than kPartRows
// terms in one fp32 chain, each of which may be rounded the same way (16M rows of 8: 7e-5
// of the sum), twice as many parts, three times as many, ...
constexpr int64_t kPartRows = 1024;
static int norm_parts(int64_t rows, int64_t cols, bool f32, bool sums) {
    const int64_t groups = cols <= 768 ? (rows + 7) / 8 : rows;
    const int64_t held = cols <= 768 ? 2 : cols <= 2048 ? 4 : cols <= 4096 ? (f32 ? 2 : 3) : cols <= 8192 ? (f32 ? 1 : 2)
                         : cols <= 16384 ? 1 : 2;
    const int64_t root = int64_t(std::sqrt(double(groups) * (110000.0 / double(cols < 1 ? 1 : cols) + 20.0))) + 1;
    int64_t most = sums && root < held * kNormSms ? root : held * kNormSms;
    if (sums && groups > most * kPartRows) most *= (groups + most * kPartRows - 1) / (most * kPartRows);
    const int64_t each = (groups + most - 1) / most;
    return int(groups < 1 ? 1 : (groups + each - 1) / each);
}

template <bool F32, int MODE, int T, int V>
static int launch_norm_as(const NormArgs& a, cudaStream_t s, const char* who) {
    constexpr int per = norm_threads<T>() / T;
    auto k = k_layer_norm<F32, MODE, T, V>;
    int dev = 0, grid = 0;
    DPG_CUDA_TRY(cudaGetDevice(&dev));
    const int st = grid_for(reinterpret_cast<const void*>(k), norm_threads<T>(), dev, (a.rows + per - 1) / per, &grid);
    return st != DPG_OK ? st : launch_k(k, unsigned(grid), norm_threads<T>(), s, who, a);
}
template <int T, int V>
static int launch_norm(const NormArgs& a, bool f32, bool vec, cudaStream_t s, const char* who) {
    const int mode = !vec ? kRowOdd : a.cols == T * V * 8 ? kRowFull : kRowVec;
    if (f32)
        return mode == kRowFull ? launch_norm_as<true, kRowFull, T, V>(a, s, who)
               : mode == kRowVec ? launch_norm_as<true, kRowVec, T, V>(a, s, who) : launch_norm_as<true, kRowOdd, T, V>(a, s, who);
    return mode == kRowFull ? launch_norm_as<false, kRowFull, T, V>(a, s, who)
           : mode == kRowVec ? launch_norm_as<false, kRowVec, T, V>(a, s, who) : launch_norm_as<false, kRowOdd, T, V>(a, s, who);
}

template <bool F32, int MODE, int T, int V>
static int launch_back_as(const NormBackArgs& a, cudaStream_t s, const char* who) {
    auto k = k_layer_norm_back<F32, MODE, T, V>;
    constexpr int smem = MODE != kRowOdd || T == 32 ? back_smem<F32, T, V>() : 0;
    static std::atomic<uint64_t> once{0};
    const int st = smem > 0 ? allow_smem(reinterpret_cast<const void*>(k), smem, once, who) : DPG_OK;
    return st != DPG_OK ? st : launch_k(k, unsigned(a.parts), norm_threads<T>(), size_t(smem), s, who, a);
}
template <int T, int V>
static int launch_back(const NormBackArgs& a, bool f32, bool vec, cudaStream_t s, const char* who) {
    const int mode = !vec ? kRowOdd : a.cols == T * V * 8 ? kRowFull : kRowVec;
    if (f32)
        return mode == kRowFull ? launch_back_as<true, kRowFull, T, V>(a, s, who)
               : mode == kRowVec ? launch_back_as<true, kRowVec, T, V>(a, s, who) : launch_back_as<true, kRowOdd, T, V>(a, s, who);
    return mode == kRowFull ? launch_back_as<false, kRowFull, T, V>(a, s, who)
           : mode == kRowVec ? launch_back_as<false, kRowVec, T, V>(a, s, who) : launch_back_as<false, kRowOdd, T, V>(a, s, who);
}

}  // namespace dpg

using dpg::fail;

extern "C" {

int dpg_layer_norm(const void* x, int32_t dtype, int64_t rows, int64_t cols, const void* gain, const void* bias,
                   int32_t param_dtype, double eps, void* y, float* mean, float* rstd, void* stream) {
    dpg::clear_error();
    const char* who = "dpg_layer_norm";
    const dpg::Trace trace(who);
    int st = dpg::norm_shape(rows, cols, dtype, param_dtype, who);
    if (st != DPG_OK) return st;
    // (not one that fp32 makes an infinity or a zero of)
    if (!(eps >= 0.0 && eps <= double(std::numeric_limits<float>::max())) || (eps > 0.0 && float(eps) == 0.0f))
        return fail(DPG_ERR_INVALID_ARG, "%s: eps %g", who, eps);
    if ((mean == nullptr) != (rstd == nullptr))
        return fail(DPG_ERR_INVALID_ARG, "%s: mean and rstd are kept together", who);
    if (rows == 0 || cols == 0) return DPG_OK;
    st = dpg::norm_pointer(x, dtype, false, "x", who);
    if (st == DPG_OK) st = dpg::norm_pointer(y, dtype, false, "y", who);
    if (st == DPG_OK) st = dpg::norm_pointer(gain, param_dtype, true, "gain", who);
    if (st == DPG_OK) st = dpg::norm_pointer(bias, param_dtype, true, "bias", who);
    if (st == DPG_OK) st = dpg::norm_pointer(mean, DPG_F32, true, "mean", who);
    if (st == DPG_OK) st = dpg::norm_pointer(rstd, DPG_F32, true, "rstd", who);
    if (st != DPG_OK) return st;
    if (mean && mean == rstd) return fail(DPG_ERR_INVALID_ARG, "%s: mean and rstd share a buffer", who);
    dpg::NormArgs a{};
    a.x = x;
    a.gain = gain;
    a.bias = bias;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.cols = int32_t(cols);
    a.params_f32 = param_dtype == DPG_F32;
    a.eps = float(eps);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = dtype == DPG_F32;
    const bool vec = cols % 8 == 0 && dpg::aligned(x, 16) && dpg::aligned(y, 16) && dpg::aligned(gain, 16) &&
                     dpg::aligned(bias, 16);
    if (cols <= 256) return dpg::launch_norm<32, 1>(a, f32, vec, s, who);
    if (cols <= 512) return dpg::launch_norm<32, 2>(a, f32, vec, s, who);
    if (cols <= 768) return dpg::launch_norm<32, 3>(a, f32, vec, s, who);
    if (cols <= 1024) return dpg::launch_norm<32, 4>(a, f32, vec, s, who);
    if (cols <= 2048) return dpg::launch_norm<128, 2>(a, f32, vec, s, who);
    if (cols <= 4096) return dpg::launch_norm<128, 4>(a, f32, vec, s, who);
    if (cols <= 8192) return dpg::launch_norm<256, 4>(a, f32, vec, s, who);
    if (cols <= 16384) return dpg::launch_norm<512, 4>(a, f32, vec, s, who);
    if (cols <= 32768) return dpg::launch_norm<1024, 4>(a, f32, vec, s, who);
    return dpg::launch_k(f32 ? dpg::k_layer_norm_long<true> : dpg::k_layer_norm_long<false>, unsigned(rows), dpg::kLongThreads, s,
                         who, a);
}

int64_t dpg_layer_norm_workspace(int64_t rows, int64_t cols) {
    if (rows < 0 || cols <= 0 || rows > dpg::kNormMaxSide || cols > dpg::kNormMaxSide) return 0;
    // of the type that needs more: with many rows fp32, of which an SM holds fewer, may take more parts
    const int parts = std::max(dpg::norm_parts(rows, cols, false, true), dpg::norm_parts(rows, cols, true, true));
    return int64_t(parts) * 2 * cols * int64_t(sizeof(float));
}

int dpg_layer_norm_backward(const void* dy, const void* x, int32_t dtype, int64_t rows, int64_t cols,
                            const void* gain, int32_t param_dtype, const float* mean, const float* rstd, void* dx,
                            void* dgain, void* dbias, int32_t grad_dtype, int32_t accumulate, void* workspace,
                            void* stream) {
    dpg::clear_error();
    const char* who = "dpg_layer_norm_backward";
    const dpg::Trace trace(who);
    int st = dpg::norm_shape(rows, cols, dtype, param_dtype, who);
    if (st != DPG_OK) return st;
    if (grad_dtype != DPG_BF16 && grad_dtype != DPG_F32)
        return fail(DPG_ERR_INVALID_ARG, "%s: grad_dtype %d unknown", who, grad_dtype);
    if (accumulate && grad_dtype != DPG_F32)
        return fail(DPG_ERR_INVALID_ARG, "%s: only fp32 gradients are added to", who);
    const bool sums = dgain || dbias;
    if (cols == 0 || (rows == 0 && (!sums || accumulate))) return DPG_OK;
    if (rows > 0) {
        st = dpg::norm_pointer(dy, dtype, false, "dy", who);
        if (st == DPG_OK) st = dpg::norm_pointer(x, dtype, false, "x", who);
        if (st == DPG_OK) st = dpg::norm_pointer(gain, param_dtype, true, "gain", who);
        if (st == DPG_OK) st = dpg::norm_pointer(mean, DPG_F32, false, "mean", who);
        if (st == DPG_OK) st = dpg::norm_pointer(rstd, DPG_F32, false, "rstd", who);
        if (st == DPG_OK) st = dpg::norm_pointer(dx, dtype, true, "dx", who);
    }
    if (st == DPG_OK) st = dpg::norm_pointer(dgain, grad_dtype, true, "dgain", who);
    if (st == DPG_OK) st = dpg::norm_pointer(dbias, grad_dtype, true, "dbias", who);
    if (st != DPG_OK) return st;
    if (sums && !workspace) return fail(DPG_ERR_INVALID_ARG, "%s: workspace is NULL", who);
    if (sums && !dpg::aligned(workspace, 16)) return fail(DPG_ERR_MISALIGNED, "%s: workspace misaligned", who);
    if (dgain && dgain == dbias) return fail(DPG_ERR_INVALID_ARG, "%s: dgain and dbias share a buffer", who);
    if (!sums && !dx) return DPG_OK;
    const bool f32 = dtype == DPG_F32;
    dpg::NormBackArgs a{};
    a.dy = dy;
    a.x = x;
    a.gain = gain;
    a.mean = mean;
    a.rstd = rstd;
    a.dx = dx;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    a.rows = rows;
    a.cols = int32_t(cols);
    a.params_f32 = param_dtype == DPG_F32;
    a.parts = dpg::norm_parts(rows, cols, f32, sums);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = cols % 8 == 0 && dpg::aligned(x, 16) && dpg::aligned(dy, 16) && dpg::aligned(dx, 16) &&
                     dpg::aligned(gain, 16);
    if (cols <= 256) st = dpg::launch_back<32, 1>(a, f32, vec, s, who);
    else if (cols <= 512) st = dpg::launch_back<32, 2>(a, f32, vec, s, who);
    else if (cols <= 768) st = dpg::launch_back<32, 3>(a, f32, vec, s, who);
    else if (cols <= 1024) st = dpg::launch_back<128, 1>(a, f32, vec, s, who);
    else if (cols <= 2048) st = dpg::launch_back<256, 1>(a, f32, vec, s, who);
    else if (cols <= 4096) st = dpg::launch_back<256, 2>(a, f32, vec, s, who);
    else if (cols <= 8192) st = dpg::launch_back<512, 2>(a, f32, vec, s, who);
    else if (cols <= 16384) st = dpg::launch_back<512, 4>(a, f32, vec, s, who);
    else {
        if (sums) {
            cudaLaunchConfig_t cfg = {};
            const int wide = vec ? 2048 : 256;
            cfg.gridDim = dim3(unsigned((cols + wide - 1) / wide), unsigned(a.parts));
            cfg.blockDim = dim3(256);
            cfg.stream = s;
            const cudaError_t e = cudaLaunchKernelEx(&cfg, vec ? dpg::k_layer_norm_columns<8> : dpg::k_layer_norm_columns<1>, a, int32_t(f32));
            if (e != cudaSuccess) {
                (void)cudaGetLastError();
                return fail(DPG_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
            }
            st = dpg::after_launch(who);
        }
        if (st == DPG_OK && dx && rows > 0) {
            auto k = f32 ? (vec ? dpg::k_layer_norm_dx_long<8, true> : dpg::k_layer_norm_dx_long<1, true>)
                         : (vec ? dpg::k_layer_norm_dx_long<8, false> : dpg::k_layer_norm_dx_long<1, false>);
            st = dpg::launch_k(k, unsigned(rows), dpg::kDxThreads, s, who, a);
        }
    }
    if (st != DPG_OK || !sums) return st;
    dpg::NormSumArgs t{};
    t.part = a.part;
    t.out[0] = dgain;
    t.out[1] = dbias;
    t.parts = a.parts;
    t.cols = a.cols;
    t.f32 = grad_dtype == DPG_F32;
    t.add = accumulate != 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((cols + 31) / 32), 2);
    cfg.blockDim = dim3(32 * dpg::kSumRows);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dpg::t_programmatic ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, a.parts > 256 * dpg::kSumRows ? dpg::k_layer_norm_sums<true> : dpg::k_layer_norm_sums<false>, t);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return fail(DPG_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    }
    return dpg::after_launch(who);
}

}  // extern "C"
