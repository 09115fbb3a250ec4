// dpg_fp4.cu -- quantisation to 4-bit floating point and back (see
// dpg_fp4_quantize, dpg_fp4_dequantize and dpg_allgather_params_fp4 in
// include/dpg.h).
//
// A block of 16 (or 32) elements x has the scale s = the least E4M3 (E8M0) value
// with max|x| <= 6 s, and the codes nearest to x / s on 0, .5, 1, 1.5, 2, 3, 4, 6.
// Every decision is exact:
//   * s by a product with 1/6 rounded up, then compared with its neighbours
//     through 6 s, which is exact;
//   * y = x / s for an E8M0 scale is a product with a power of two; for an E4M3
//     one it is the correctly rounded quotient, from the reciprocal and one
//     residual (Markstein 1990).  A borderline m s has at most 7 bits, so a
//     quotient whose x is not on it rounds to something else than m, and ties stay
//     ties.  The product with the reciprocal alone is off by one unit for 11 of the
//     56 borderlines, and would round those ties up.
//   * stochastic: between the values the place of y, in codes, is linear, and so are
//     the bits of an fp32 number between powers of two.  2^-126 y has y's place in its
//     bits, in units of 2^-22 codes: below y = 1, where the values are 0 and 1/2, it is
//     subnormal, and those are 1/2 apart too.  y goes up where the fraction is above
//     (2 u + 1) 2^-17, a whole number of units, so the place may be rounded up to one.
//     That is done from below: x times the reciprocal, both rounded down, and one
//     residual, whose product with the reciprocal is at most 2^-21 units short; x / s
//     is on a whole number of units, or 1/15 from it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <exception>
#include <vector>

#include "dpg_async.cuh"
#include "dpg_fp4.h"
#include "dpg_host.h"
#include "dpg_ortho.h"

namespace dpg {

constexpr int kQuantTile = 128;         // rows and columns of a CTA's tile

struct QuantSide {
    unsigned char* codes;               // NULL: this orientation is not wanted
    unsigned char* scales;
    int64_t pitch, tiles;               // of its codes, of its scales (see dpg_fp4.h)
    int64_t vectors;                    // groups of 8 elements in a row (of random bits)
};

struct QuantArgs {
    const void* x;
    int64_t rows, cols, stride;
    int64_t tiles_c;                    // tiles in a row of tiles
    int32_t vec;                        // 16-byte loads are allowed
    const int64_t* seed;                // NULL: nearest
    int64_t seed_plus;
    float* amax;                        // E4M3: the largest magnitude, and behind it its parts
    float* amax_copy;                   // the other side's (NULL: none)
    int32_t parts;                      // that k_fp4_amax left (0: this launch, one cluster, finds it)
    QuantSide row, col;
};

// ---------------------------------------------------------------------------
// Largest finite magnitude, as the bits of an fp32 number: these order like the
// numbers.  Every CTA leaves the one of its share behind the result's place, and
// the CTAs of the quantisation take the largest of them: nothing to set to zero
// before, and no atomics (9700 on one address took 12 us).  A CTA of 1024 threads to
// an SM, 128 KB of loads on their way: 25 us for 134 MB (5.3 TB/s, which read nothing
// but new lines of HBM); with 255 CTAs of 512, of which some SMs had one and some two,
// quantising 16384 x 4096 bf16 took 92 us instead of 82.
// ---------------------------------------------------------------------------
constexpr int kAmaxCtas = 152;           // a GB300's SMs
static_assert(kAmaxCtas < DPG_FP4_AMAX_FLOATS, "room for the parts");

template <bool F32>
__device__ __forceinline__ uint32_t magnitude_bits(uint32_t w) {      // of one fp32 or two bf16 values
    if (F32) {
        const uint32_t a = w & 0x7FFFFFFFu;
        return a < 0x7F800000u ? a : 0u;
    }
    uint32_t lo = (w << 16) & 0x7FFFFFFFu, hi = w & 0x7FFF0000u;
    lo = lo < 0x7F800000u ? lo : 0u;
    hi = hi < 0x7F800000u ? hi : 0u;
    return lo > hi ? lo : hi;
}
template <bool F32>
__device__ __forceinline__ uint32_t magnitude_bits4(uint4 v) {
    return max(max(magnitude_bits<F32>(v.x), magnitude_bits<F32>(v.y)),
               max(magnitude_bits<F32>(v.z), magnitude_bits<F32>(v.w)));
}
// the same with NaNs and infinities among them; bf16: of the two halves each
template <bool F32>
__device__ __forceinline__ uint32_t any_magnitude(uint32_t m, uint4 v) {
    if constexpr (F32) {
        return max(max(max(m, v.x & 0x7FFFFFFFu), max(v.y & 0x7FFFFFFFu, v.z & 0x7FFFFFFFu)), v.w & 0x7FFFFFFFu);
    } else {
        m = __vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
        return __vmaxu2(__vmaxu2(m, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
    }
}
// largest over 32 W threads, in all of them
template <int W>
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* sh) {
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
    __syncthreads();
    return __reduce_max_sync(0xFFFFFFFFu, sh[threadIdx.x & (W - 1)]);
}
constexpr int kAmaxThreads = 1024;

template <bool F32>
__global__ void __launch_bounds__(kAmaxThreads) k_fp4_amax(const void* x, int64_t rows, int64_t cols, int64_t stride,
                                                  int64_t pieces, uint32_t* parts) {
    __shared__ uint32_t sh[kAmaxThreads / 32];
    pdl_enter();
    uint32_t m = 0;
    constexpr int kPer = F32 ? 4 : 8, kFly = 8;      // elements of 16 bytes, loads in flight
    if (pieces == 0) {                               // rows back to back
        const int64_t n = rows * cols, t = int64_t(blockIdx.x) * kAmaxThreads + threadIdx.x,
                      step = int64_t(gridDim.x) * kAmaxThreads;
        // up to the first 16-byte boundary, and behind the last one, singly
        const int64_t head = min(n, int64_t((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (F32 ? 4 : 2));
        const int64_t vecs = (n - head) / kPer, tail = head + vecs * kPer;
        const unsigned char* p = static_cast<const unsigned char*>(x) + head * (F32 ? 4 : 2);
        for (int64_t i = t; i < vecs; i += kFly * step) {
            uint4 v[kFly];
#pragma unroll
            for (int u = 0; u < kFly; ++u)
                v[u] = i + u * step < vecs ? *reinterpret_cast<const uint4*>(p + (i + u * step) * 16) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kFly; ++u) m = any_magnitude<F32>(m, v[u]);
        }
        if (!F32) m = max(m << 16, m) & 0xFFFF0000u;
        if (m >= 0x7F800000u) {                      // not all are finite: the largest of those that are
            m = 0;
            for (int64_t i = t; i < vecs; i += step) m = max(m, magnitude_bits4<F32>(*reinterpret_cast<const uint4*>(p + i * 16)));
        }
        if (t < head + n - tail) {
            const int64_t j = t < head ? t : tail + t - head;
            m = max(m, F32 ? magnitude_bits<true>(static_cast<const uint32_t*>(x)[j])
                           : magnitude_bits<false>(static_cast<const uint16_t*>(x)[j]));
        }
    } else {
        // pieces of rows between 16-byte boundaries, those at a row's ends singly
        const int64_t n = rows * pieces, t = int64_t(blockIdx.x) * kAmaxThreads + threadIdx.x,
                      step = int64_t(gridDim.x) * kAmaxThreads;
        constexpr int kSize = F32 ? 4 : 2;
        uint32_t ends = 0;
        auto load = [&](int64_t i, bool singly) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (i >= n) return v;
            const int64_t r = (i | pieces) > 0x7FFFFFFF ? i / pieces : int64_t(uint32_t(i) / uint32_t(pieces));
            const unsigned char* row = static_cast<const unsigned char*>(x) + r * stride * kSize;
            const int64_t e = (i - r * pieces) * kPer - int(reinterpret_cast<uintptr_t>(row) & 15) / kSize;
            if (e >= 0 && e + kPer <= cols) v = *reinterpret_cast<const uint4*>(row + e * kSize);
            else if (singly)
                for (int64_t c = max(e, int64_t(0)); c < min(e + kPer, cols); ++c)
                    ends = max(ends, F32 ? magnitude_bits<true>(reinterpret_cast<const uint32_t*>(row)[c])
                                         : magnitude_bits<false>(reinterpret_cast<const uint16_t*>(row)[c]));
            return v;
        };
        for (int64_t i = t; i < n; i += kFly * step) {
            uint4 v[kFly];
#pragma unroll
            for (int u = 0; u < kFly; ++u) v[u] = load(i + u * step, true);
#pragma unroll
            for (int u = 0; u < kFly; ++u) m = any_magnitude<F32>(m, v[u]);
        }
        if (!F32) m = max(m << 16, m) & 0xFFFF0000u;
        if (m >= 0x7F800000u) {
            m = 0;
            for (int64_t i = t; i < n; i += step) m = max(m, magnitude_bits4<F32>(load(i, false)));
        }
        m = max(m, ends);
    }
    m = block_max<kAmaxThreads / 32>(m, sh);
    if (threadIdx.x == 0) parts[blockIdx.x] = m;
}

// ---------------------------------------------------------------------------
// One block
// ---------------------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011)
__device__ __forceinline__ uint4 philox(uint64_t n, uint32_t side, uint2 key) {
    uint32_t x0 = uint32_t(n), x1 = uint32_t(n >> 32), x2 = side, x3 = 0, k0 = key.x, k1 = key.y;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = uint64_t(x0) * 0xD2511F53u, b = uint64_t(x2) * 0xCD9E8D57u;
        x0 = uint32_t(b >> 32) ^ x1 ^ k0;
        x2 = uint32_t(a >> 32) ^ x3 ^ k1;
        x1 = uint32_t(b);
        x3 = uint32_t(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

// E4M3 value of a byte (0 .. 0x7E)
__device__ __forceinline__ float e4m3_value(int byte) {
    return byte < 8 ? float(byte) * 0.001953125f : __uint_as_float(uint32_t(byte + 960) << 20);
}

constexpr int kInverses = 128;     // of every E4M3 value, in shared memory

struct BlockScale {
    int byte;          // as stored
    float s, inv;      // E4M3: scale * 2^e; about 1 / (scale * 2^e), 0 for 0 or where `bad`
    bool bad;          // a NaN or an infinity in the block
};

// of a block whose largest magnitude has the bits `top`; E4M3: unit = 2^-e, whole =
// 2^e, inverses[byte] = 1 / its value (stochastic: rounded down)
template <bool F32, bool MX>
__device__ __forceinline__ BlockScale block_scale(uint32_t top, float unit, float whole, const float* inverses) {
    BlockScale b;
    b.bad = top >= 0x7F800000u;
    if (MX) {
        const int e = int(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
        const int k = e < 0 ? 0 : e;
        b.byte = b.bad ? 0xFF : k;
        b.inv = b.bad ? 0.0f : __uint_as_float(uint32_t(254 - k) << 23);
        b.s = 0.0f;                                     // (not used)
        return b;
    }
    const float u = __uint_as_float(top) * unit;
    const float q = u * 0.166666672f;                   // 1/6 rounded up: at most two units above u / 6
    // E4M3 values are the fp32 numbers with three bits, down to 2^-6, and multiples of 2^-9 below
    int k;
    if (F32) {
        k = q < 0.015625f ? int(ceilf(q * 512.0f)) : int((__float_as_uint(q) + 0xFFFFFu) >> 20) - 960;
        k = k > 0x7E ? 0x7E : k;
        if (k > 0 && 6.0f * e4m3_value(k - 1) >= u) --k;
        else if (k < 0x7E && 6.0f * e4m3_value(k) < u) ++k;
    } else {
        // u has 8 bits: u / 6 is on a value, or 2^-9 of itself from it
        k = int((__float_as_uint(q) + (0xFFFFFu - 16u)) >> 20) - 960;
        if (q < 0.0156f) k = int(ceilf(__uint_as_float(__float_as_uint(q) - (q > 1e-30f ? 16u : 0u)) * 512.0f));
    }
    k = k == 0 && top != 0 ? 1 : k;                     // (u may have been too small for fp32)
    b.s = e4m3_value(k) * whole;
    b.inv = b.bad ? 0.0f : inverses[k] * unit;
    b.byte = b.bad ? 0x7F : k;
    return b;
}

// eight values to nearest codes, the first in the lowest four bits
__device__ __forceinline__ uint32_t nearest8(const uint64_t* y) {
    uint32_t r;
    const float2 a = halves_of(y[0]), b = halves_of(y[1]), c = halves_of(y[2]), d = halves_of(y[3]);
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
    return r;
}

__device__ __forceinline__ uint64_t fma2_up(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rp.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2_up(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rp.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2_down(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rm.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// The code of a place in bits 24 .. 26, from the upper (HIGH) or lower half u of the
// random bits: a quarter unit a step, 2^24 - 129 - 256 u more carries where the place
// is above 64 u + 32 units.  `inverted` is the complement.
template <bool HIGH>
__device__ __forceinline__ uint32_t round_place(uint32_t place, uint32_t inverted) {
    return place * 4u + __byte_perm(inverted, 0x7Fu, HIGH ? 0x5324 : 0x5104);
}

// B elements of a block to codes, 8 to a word.  w: the elements as they are in
// memory (bf16: two to a word); n0: number of their first group of 8 (random bits).
template <bool F32, bool MX, bool SR, int B>
__device__ __forceinline__ void encode(const uint32_t* w, const BlockScale& b, uint64_t n0, uint32_t side, uint2 key,
                                       uint32_t* out) {
    const uint64_t inv = pair_of(b.inv, b.inv), s = pair_of(-b.s, -b.s);
#pragma unroll
    for (int g = 0; g < B / 8; ++g) {
        uint64_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = 4 * g + j;                       // of a pair
            float lo, hi;
            if (F32) {
                lo = __uint_as_float(SR ? w[2 * at] & 0x7FFFFFFFu : w[2 * at]);
                hi = __uint_as_float(SR ? w[2 * at + 1] & 0x7FFFFFFFu : w[2 * at + 1]);
            } else {
                widen2(SR ? w[at] & 0x7FFF7FFFu : w[at], lo, hi);
            }
            const uint64_t x = pair_of(lo, hi);
            if (MX) y[j] = mul2(x, inv);
            else if (SR) y[j] = mul2_down(x, inv), y[j] = fma2_up(fma2(y[j], s, x), inv, y[j]);
            else y[j] = mul2(x, inv), y[j] = fma2(fma2(y[j], s, x), inv, y[j]);
        }
        if (SR) {
            const uint4 r = philox(n0 + g, side, key);
            const uint32_t h[4] = {~r.x, ~r.y, ~r.z, ~r.w};
            uint32_t lo, hi;                                // bytes that hold the signs in bit 7
            if (F32) {
                const uint32_t* v = w + 8 * g;
                lo = __byte_perm(__byte_perm(v[0], v[2], 0x0073), __byte_perm(v[4], v[6], 0x0073), 0x5410);
                hi = __byte_perm(__byte_perm(v[1], v[3], 0x0073), __byte_perm(v[5], v[7], 0x0073), 0x5410);
            } else {
                const uint32_t* v = w + 4 * g;
                lo = __byte_perm(__byte_perm(v[0], v[1], 0x0051), __byte_perm(v[2], v[3], 0x0051), 0x5410);
                hi = __byte_perm(__byte_perm(v[0], v[1], 0x0073), __byte_perm(v[2], v[3], 0x0073), 0x5410);
            }
            uint32_t t[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 p = halves_of(mul2_up(y[j], pair_of(0x1p-126f, 0x1p-126f)));
                t[2 * j] = round_place<false>(__float_as_uint(p.x), h[j]);
                t[2 * j + 1] = round_place<true>(__float_as_uint(p.y), h[j]);
            }
            const uint32_t even = __byte_perm(__byte_perm(t[0], t[2], 0x0073), __byte_perm(t[4], t[6], 0x0073), 0x5410);
            const uint32_t odd = __byte_perm(__byte_perm(t[1], t[3], 0x0073), __byte_perm(t[5], t[7], 0x0073), 0x5410);
            const uint32_t word = (odd * 16u + even) | (hi & 0x80808080u) | ((lo & 0x80808080u) >> 4);
            out[g] = b.bad ? 0u : word;
        } else {
            out[g] = b.bad ? 0u : nearest8(y);
        }
    }
}

// bits of the largest magnitude of a block (of a NaN, or of the infinity, where it has one)
template <bool F32, int B>
__device__ __forceinline__ uint32_t block_top(const uint32_t* w) {
    uint32_t top = 0;
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < B; ++j) top = max(top, w[j] & 0x7FFFFFFFu);
        return top;
    } else {
#pragma unroll
        for (int j = 0; j < B / 2; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
        return max(top << 16, top) & 0xFFFF0000u;
    }
}

// ---------------------------------------------------------------------------
// Both orientations from one read.  A CTA takes 128 x 128 elements into shared
// memory by asynchronous copies, with a thread to each block of a row and of a
// column after that; codes leave through shared memory too, 64 bytes of a row at
// a time.  (Blocks loaded to registers by the thread that takes them: lanes 32 to
// 128 bytes apart, 16 warps to an SM, 68 us for 8192 x 4096 fp32 masters.)  Rows of
// the tile are 16 bytes longer than a multiple of 128, so that neighbouring rows'
// pieces lie in different banks.
//
// What bounds it: 14336 x 4096 fp32 masters to E8M0 58 us (297 MB, 5.1 TB/s); 16384 x
// 4096 bf16 to E4M3 55 us beside the 25 of the largest magnitude, 11.4 instructions an
// element and orientation, issued in 74 % of the cycles; stochastic 119 us, 23
// instructions, of them 5 for random bits.  bf16 to E8M0 41 us, its bytes 30; the fp32
// masters to E4M3 114 us, read twice for the largest magnitude, where the bytes of one reading
// would take 44.
// ---------------------------------------------------------------------------
template <bool F32, bool SR>
struct TileOf {
    static constexpr int kPitch = F32 ? 132 : 68;          // words of a row in shared memory
    static constexpr int kBytes = kQuantTile * kPitch * 4;
    static constexpr int kPieces = F32 ? 32 : 16;          // 16-byte pieces of a row
    static constexpr int kPer = F32 ? 4 : 8;               // elements of a piece
    // Two CTAs of fp32 tiles fit an SM, four of bf16 ones (16384 x 4096 both sides 114 -> 92 us),
    // with random bits three that have more registers (512 x 2: 152, 256 x 4: 140, 256 x 3: 141;
    // 4096 x 1536 17.5, 20.5 and 17.1).
    static constexpr int kThreads = F32 ? 512 : 256;
    static constexpr int kLoads = kQuantTile * kPieces / kThreads;
};
constexpr int kCodesPitch = 72;                            // bytes of a row's codes in shared memory

template <bool F32>
constexpr int quant_smem() { return TileOf<F32, false>::kBytes + 2 * kQuantTile * kCodesPitch; }

// `bytes` (0 .. 16) of a 16-byte piece, zeros behind them
__device__ __forceinline__ void copy_piece(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}

// One piece from element `at` on, `n` of its elements in the matrix.  Where rows
// do not start on 16-byte boundaries, the two aligned pieces that hold it are
// loaded (if both lie in the matrix) and shifted into place.
template <bool F32>
__device__ __forceinline__ uint4 load_piece(const QuantArgs& a, int64_t at, int n, int64_t end) {
    constexpr int kSize = F32 ? 4 : 2, kPer = TileOf<F32, false>::kPer;
    const unsigned char* p = static_cast<const unsigned char*>(a.x) + at * kSize;
    uint32_t w[4];
    if (n >= kPer && at >= kPer && at + 2 * kPer <= end) {
        const int off = int(reinterpret_cast<uintptr_t>(p) & 15) / kSize;
        const uint4* q = reinterpret_cast<const uint4*>(p - off * kSize);
        const uint4 lo = __ldg(q), hi = __ldg(q + 1);
        uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const int words = F32 ? off : off >> 1;
#pragma unroll
        for (int j = 0; j < 6; ++j) v[j] = (words & 2) ? v[j + 2] : v[j];
#pragma unroll
        for (int j = 0; j < 5; ++j) v[j] = (words & 1) ? v[j + 1] : v[j];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = F32 ? v[j] : __funnelshift_r(v[j], v[j + 1], (off & 1) * 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (F32) {
            w[j] = j < n ? __ldg(reinterpret_cast<const uint32_t*>(p) + j) : 0u;
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(p) + 2 * j;
            const uint32_t lo = 2 * j < n ? __ldg(h) : 0u, hi = 2 * j + 1 < n ? __ldg(h + 1) : 0u;
            w[j] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// rows, cols: of the tile that the matrix has
template <bool F32, bool SR>
__device__ __forceinline__ void load_tile(const QuantArgs& a, int64_t r0, int64_t c0, int rows, int cols, uint32_t* tile) {
    using T = TileOf<F32, SR>;
    constexpr int kSize = F32 ? 4 : 2, kStep = T::kThreads / T::kPieces;     // rows from one load to the next
    const int row0 = int(threadIdx.x) / T::kPieces, piece = int(threadIdx.x) % T::kPieces;
    const int n = cols - piece * T::kPer;                                      // elements from the piece's first on
    int64_t at = (r0 + row0) * a.stride + c0 + piece * T::kPer;
    if (a.vec) {
        const int bytes = n >= T::kPer ? 16 : n > 0 ? n * kSize : 0;
        const unsigned char* p = static_cast<const unsigned char*>(a.x) + at * kSize;
        const int64_t step = kStep * a.stride * kSize;
        uint32_t dst = smem_u32(tile + row0 * T::kPitch + piece * 4);
#pragma unroll
        for (int k = 0; k < T::kLoads; ++k) {
            const int some = row0 + k * kStep < rows ? bytes : 0;
            copy_piece(dst, some ? p : a.x, some);
            p += step;
            dst += kStep * T::kPitch * 4;
        }
    } else {
        const int64_t end = (a.rows - 1) * a.stride + a.cols;
#pragma unroll 4
        for (int k = 0; k < T::kLoads; ++k) {
            *reinterpret_cast<uint4*>(tile + (row0 + k * kStep) * T::kPitch + piece * 4) =
                n > 0 && row0 + k * kStep < rows ? load_piece<F32>(a, at, n, end) : make_uint4(0, 0, 0, 0);
            at += kStep * a.stride;
        }
    }
}

// an element, or two, times 2^100 (which are below 2^-88, NaN or infinite)
template <bool F32>
__device__ __forceinline__ uint32_t larger(uint32_t w) {
    constexpr float k = 1.2676506002282294e30f;
    if (F32) return __float_as_uint(__uint_as_float(w) * k);
    float lo, hi;
    widen2(w, lo, hi);
    return __byte_perm(__float_as_uint(lo * k), __float_as_uint(hi * k), 0x7632);
}

template <bool F32, bool MX, bool SR>
__global__ void __launch_bounds__(TileOf<F32, SR>::kThreads, F32 ? 2 : SR ? 3 : 4) k_fp4_quantize(const __grid_constant__ QuantArgs a) {
    using T = TileOf<F32, SR>;
    constexpr int B = MX ? 32 : 16;                        // elements of a block
    constexpr int kBlocks = kQuantTile / B;                // blocks of a tile's row
    constexpr int kTasks = kQuantTile * kBlocks / T::kThreads;
    constexpr int kWords = B * (F32 ? 4 : 2) / 4;          // 32-bit words of a block
    constexpr int kTiles = kBlocks / 4;                    // scale tiles of a tile
    extern __shared__ __align__(16) uint32_t tile[];
    __shared__ __align__(16) unsigned char sc[2][kTiles * kFp4TileBytes];
    unsigned char* const out = reinterpret_cast<unsigned char*>(tile) + T::kBytes;
    const int64_t ti = blockIdx.x / a.tiles_c, tj = blockIdx.x % a.tiles_c;
    const int64_t r0 = ti * kQuantTile, c0 = tj * kQuantTile;
    const int tid = int(threadIdx.x);
    const int rows = int(min(a.rows - r0, int64_t(kQuantTile))), cols = int(min(a.cols - c0, int64_t(kQuantTile)));
    // After k_fp4_amax, which has itself waited for what came before it, x may be read at once.
    if (!a.parts) pdl_enter();
    load_tile<F32, SR>(a, r0, c0, rows, cols, tile);
    if (a.parts) pdl_enter();
    uint2 key = make_uint2(0, 0);
    if (SR) {                                              // (the same in the warp: its schedule stays in uniform registers)
        const uint64_t k = uint64_t(__ldg(a.seed) + a.seed_plus);
        key.x = __shfl_sync(0xFFFFFFFFu, uint32_t(k), 0);
        key.y = __shfl_sync(0xFFFFFFFFu, uint32_t(k >> 32), 0);
    }
    float unit = 1.0f, whole = 1.0f;
    bool tiny = false;
    __shared__ float inverses[MX ? 1 : kInverses];
    if (!MX) {
        __shared__ uint32_t sh[T::kThreads / 32];
        uint32_t m = 0;
        // (block_max waits)
        if (tid < kInverses)
            inverses[tid] = tid == 0 || tid == 0x7F ? 0.0f : SR ? __fdiv_rd(1.0f, e4m3_value(tid)) : 1.0f / e4m3_value(tid);
        if (a.parts) {
            if (tid < a.parts) m = __ldcg(reinterpret_cast<const uint32_t*>(a.amax) + 1 + tid);
        } else {
            asm volatile("cp.async.wait_all;" ::: "memory");       // (this thread's own pieces)
#pragma unroll
            for (int k = 0; k < T::kLoads; ++k) {
                const int id = k * T::kThreads + tid;
                m = max(m, magnitude_bits4<F32>(
                               *reinterpret_cast<const uint4*>(tile + id / T::kPieces * T::kPitch + id % T::kPieces * 4)));
            }
        }
        m = block_max<T::kThreads / 32>(m, sh);
        if (!a.parts && gridDim.x > 1) {
            __shared__ uint32_t mine;
            if (tid == 0) mine = m;
            cluster_sync();
            for (uint32_t q = 0; q < gridDim.x; ++q) {
                uint32_t other;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other) : "r"(map_to(smem_u32(&mine), q)) : "memory");
                m = max(m, other);
            }
        }
        // Where 2^-e times the inverse of a scale would leave fp32, elements are made larger first.
        const int e = fp4_exponent(m);
        tiny = e < -100;
        unit = __uint_as_float(uint32_t(127 - (tiny ? e + 100 : e)) << 23);
        whole = __uint_as_float(uint32_t(127 + (tiny ? e + 100 : e)) << 23);
        if (blockIdx.x == 0 && tid == 0) {
            *a.amax = __uint_as_float(m);
            if (a.amax_copy) *a.amax_copy = __uint_as_float(m);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const QuantSide& q = side ? a.col : a.row;
        if (!q.codes) continue;
        const int lines = side ? cols : rows, length = side ? rows : cols;     // of the quantised matrix that the tile has
        const int line = tid % kQuantTile;
        unsigned char* const place = out + (side * kQuantTile + line) * kCodesPitch;
        unsigned char* const scale = sc[side] + (line & 31) * 16 + (line >> 5) * 4;
        const uint64_t group = SR ? uint64_t((side ? c0 : r0) + line) * q.vectors + uint64_t((side ? r0 : c0) >> 3) : 0;
#pragma unroll 1
        for (int k = 0; k < kTasks; ++k) {
            const int blk = k * (T::kThreads / kQuantTile) + tid / kQuantTile;
            uint32_t w[kWords];
            if (side == 0) {
                const uint4* p = reinterpret_cast<const uint4*>(tile + line * T::kPitch + blk * kWords);
#pragma unroll
                for (int j = 0; j < kWords / 4; ++j) {
                    const uint4 v = p[j];
                    w[4 * j] = v.x;
                    w[4 * j + 1] = v.y;
                    w[4 * j + 2] = v.z;
                    w[4 * j + 3] = v.w;
                }
            } else {
                const uint32_t* p = tile + blk * B * T::kPitch + (F32 ? line : line >> 1);
                const uint32_t half = line & 1 ? 0x7632u : 0x5410u;
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    w[j] = F32 ? p[j * T::kPitch] : __byte_perm(p[2 * j * T::kPitch], p[(2 * j + 1) * T::kPitch], half);
            }
            if (tiny) {
#pragma unroll
                for (int j = 0; j < kWords; ++j) w[j] = larger<F32>(w[j]);
            }
            const BlockScale b = block_scale<F32, MX>(block_top<F32, B>(w), unit, whole, inverses);
            uint32_t codes[B / 8];
            encode<F32, MX, SR, B>(w, b, group + blk * (B / 8), side, key, codes);
            uint2* p = reinterpret_cast<uint2*>(place + blk * (B / 2));
#pragma unroll
            for (int j = 0; j < B / 16; ++j) p[j] = make_uint2(codes[2 * j], codes[2 * j + 1]);
            scale[(blk >> 2) * kFp4TileBytes + (blk & 3)] =
                static_cast<unsigned char>(line < lines && blk * B < length ? b.byte : 0);
        }
    }
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const QuantSide& q = side ? a.col : a.row;
        if (!q.codes) continue;
        const int lines = side ? cols : rows, first = tid >> 3, part = tid & 7;
        const int64_t at = ((side ? r0 : c0) >> 1) + part * 8;
        unsigned char* p = q.codes + ((side ? c0 : r0) + first) * q.pitch + at;
        if (at < q.pitch)
#pragma unroll
            for (int k = 0; k < kQuantTile; k += T::kThreads / 8) {          // 8 bytes: 16 codes of a row
                if (first + k < lines)
                    *reinterpret_cast<uint2*>(p + k * q.pitch) =
                        *reinterpret_cast<const uint2*>(out + (side * kQuantTile + first + k) * kCodesPitch + part * 8);
            }
        const int64_t i = side ? tj : ti, j0 = (side ? ti : tj) * kTiles;
        if (tid < kTiles * 32 && j0 + tid / 32 < q.tiles)
            *reinterpret_cast<uint4*>(q.scales + (i * q.tiles + j0) * kFp4TileBytes + tid * 16) =
                *reinterpret_cast<const uint4*>(sc[side] + tid * 16);
    }
    if (!MX && !a.parts && gridDim.x > 1) cluster_sync();   // the others have read this CTA's maximum
}

// ---------------------------------------------------------------------------
// Values of a quantised matrix.  A thread writes one aligned piece of a row: 32
// bytes of bf16, 64 of fp32, the 16 elements that lie there (fewer at a row's
// ends); their codes, and their scales where a block ends among them, are
// shifted into place, so rows may start anywhere.  (Pieces of 8 elements and
// conversions one by one took 33 instructions an element.)  16384 x 4096 to bf16 takes
// 30 us (172 MB, 5.7 TB/s), 38 with two stores of 16 bytes in place of one of 32; a
// thread with pieces of four rows 39, and 7.7 instead of 3.8 at 4096 x 1536.
// ---------------------------------------------------------------------------
constexpr int kPiece = 16;

struct DequantArgs {
    const unsigned char* codes;
    const unsigned char* scales;
    const float* amax;
    int64_t rows, cols, pitch, tiles, stride;
    int64_t pieces;                                     // of a row
    void* out;
};

template <bool MX>
__device__ __forceinline__ float scale_value(int byte, float unit) {
    if (MX) return byte == 0xFF ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte == 0 ? 0x00400000u : uint32_t(byte) << 23);
    return byte == 0x7F ? __uint_as_float(0x7FC00000u) : e4m3_value(byte) * unit;
}

// Eight codes as four pairs of bf16.  The two bytes of a magnitude are picked from
// tables in registers by the code's low three bits, four codes at a time.
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t* h) {
    // 0 .5 1 1.5 2 3 4 6 = 0000 3F00 3F80 3FC0 4000 4040 4080 40C0
    constexpr uint32_t hi0 = 0x3F3F3F00u, hi1 = 0x40404040u, lo0 = 0xC0800000u, lo1 = 0xC0804000u;
    const uint32_t m = w & 0x77777777u, w4 = w << 4;
    uint32_t hi = __byte_perm(hi0, hi1, m), lo = __byte_perm(lo0, lo1, m);
    h[0] = __byte_perm(lo, hi, 0x5140);
    h[1] = __byte_perm(lo, hi, 0x7362);
    hi = __byte_perm(hi0, hi1, m >> 16);
    lo = __byte_perm(lo0, lo1, m >> 16);
    h[2] = __byte_perm(lo, hi, 0x5140);
    h[3] = __byte_perm(lo, hi, 0x7362);
    // signs: bit 7 of byte j of w << 4, and of w
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] |= __byte_perm(w4, w, uint32_t(j) << 4 | uint32_t(4 + j) << 12) & 0x80008000u;
}

template <bool F32, bool MX>
__global__ void __launch_bounds__(256) k_fp4_dequantize(const __grid_constant__ DequantArgs a) {
    constexpr int kSize = F32 ? 4 : 2, kShift = MX ? 5 : 4;   // log2 of a block
    pdl_enter();
    const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t r = (a.pieces | t) > 0x7FFFFFFF ? t / a.pieces : int64_t(uint32_t(t) / uint32_t(a.pieces));
    if (r >= a.rows) return;
    unsigned char* row = static_cast<unsigned char*>(a.out) + r * a.stride * kSize;
    // elements before the row in its first piece
    const int skew = int(reinterpret_cast<uintptr_t>(row) & (kPiece * kSize - 1)) / kSize;
    const int cols = int(a.cols);
    const int e0 = int(t - r * a.pieces) * kPiece - skew;     // may be negative
    if (e0 >= cols) return;
    const int first = max(e0, 0), last = min(e0 + kPiece, cols) - 1;
    // codes: 16 from e0 on, of three neighbouring words (those that the row has)
    const int word = e0 >> 3, most = int(a.pitch >> 2) - 1;
    const uint32_t* cp = reinterpret_cast<const uint32_t*>(a.codes + r * a.pitch);
    uint32_t w[3];
    if ((e0 & 15) == 0) {
        const uint2 two = __ldg(reinterpret_cast<const uint2*>(cp + word));
        w[0] = two.x;
        w[1] = two.y;
        w[2] = 0;
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j) w[j] = __ldg(cp + min(max(word + j, 0), most));
    }
    const unsigned char* sp = a.scales + (r >> 7) * a.tiles * kFp4TileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
    const int b0 = first >> kShift, b1 = last >> kShift;
    const float unit = MX ? 1.0f : __uint_as_float(0x3F800000u + uint32_t(fp4_exponent(__float_as_uint(__ldg(a.amax)))) * 0x800000u);
    const float s0 = scale_value<MX>(__ldg(sp + int64_t(b0 >> 2) * kFp4TileBytes + (b0 & 3)), unit);
    const float s1 = b1 == b0 ? s0 : scale_value<MX>(__ldg(sp + int64_t(b1 >> 2) * kFp4TileBytes + (b1 & 3)), unit);
    const int change = (b1 << kShift) - e0;                   // first element of the second block
    const bool whole = e0 >= 0 && e0 + kPiece <= cols;
    // One scale and bf16: products in bf16 are exact (2 and 4 bits) unless the scale or a result is
    // below its normal numbers.
    if (!F32 && whole && b0 == b1 && !(s0 != 0.0f && s0 < 7.5e-37f)) {
        const __nv_bfloat162 s = __float2bfloat162_rn(s0);
        uint32_t h[8];
        F8 f;
#pragma unroll
        for (int g = 0; g < 2; ++g) widen_codes(__funnelshift_r(w[g], w[g + 1], 4 * (e0 & 7)), h + 4 * g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&h[j]), s);
            f.v[j] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&p));
        }
        st_f8(reinterpret_cast<float*>(row + int64_t(e0) * 2), f);
        return;
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t h[4];
        widen_codes(__funnelshift_r(w[g], w[g + 1], 4 * (e0 & 7)), h);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            widen2(h[j], v[2 * j], v[2 * j + 1]);
            v[2 * j] *= 8 * g + 2 * j < change ? s0 : s1;
            v[2 * j + 1] *= 8 * g + 2 * j + 1 < change ? s0 : s1;
        }
        if (whole) {
            if (F32) {
                F8 f;
#pragma unroll
                for (int j = 0; j < 8; ++j) f.v[j] = v[j];
                st_f8(reinterpret_cast<float*>(row) + e0 + 8 * g, f);
            } else {
                st_u4(row + (int64_t(e0) + 8 * g) * 2, narrow8(v));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = e0 + 8 * g + j;
                if (e < 0 || e >= cols) continue;
                if (F32) reinterpret_cast<float*>(row)[e] = v[j];
                else reinterpret_cast<__nv_bfloat16*>(row)[e] = __float2bfloat16_rn(v[j]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static int fp4_shape(int64_t rows, int64_t cols, int32_t format, const char* name, const char* who) {
    if (format != DPG_NVFP4 && format != DPG_MXFP4)
        return fail(DPG_ERR_INVALID_ARG, "%s: format %d of %s unknown", who, format, name);
    if (rows < 0 || cols < 0 || rows > kFp4MaxSide || cols > kFp4MaxSide)
        return fail(DPG_ERR_INVALID_ARG, "%s: %s: %lld x %lld outside [0, 2^30]", who, name, (long long)rows,
                    (long long)cols);
    return DPG_OK;
}

int fp4_check(const dpg_fp4* q, const char* name, const char* who) {
    const int st = fp4_shape(q->rows, q->cols, q->format, name, who);
    if (st != DPG_OK) return st;
    if (q->rows == 0 || q->cols == 0) return DPG_OK;
    if (!q->codes) return fail(DPG_ERR_INVALID_ARG, "%s: %s.codes is NULL", who, name);
    if (!q->scales) return fail(DPG_ERR_INVALID_ARG, "%s: %s.scales is NULL", who, name);
    if (q->format == DPG_NVFP4 && !q->amax) return fail(DPG_ERR_INVALID_ARG, "%s: %s.amax is NULL", who, name);
    if (!aligned(q->codes, 16)) return fail(DPG_ERR_MISALIGNED, "%s: %s.codes misaligned", who, name);
    if (!aligned(q->scales, 16)) return fail(DPG_ERR_MISALIGNED, "%s: %s.scales misaligned", who, name);
    if (q->format == DPG_NVFP4 && !aligned(q->amax, 4))
        return fail(DPG_ERR_MISALIGNED, "%s: %s.amax misaligned", who, name);
    return DPG_OK;
}

// x's type, alignment and row stride
static int strided_check(const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t stride, const char* name,
                         const char* who) {
    if (dtype != DPG_BF16 && dtype != DPG_F32)
        return fail(DPG_ERR_INVALID_ARG, "%s: dtype %d of %s unknown", who, dtype, name);
    if (rows == 0 || cols == 0) return DPG_OK;
    if (!p) return fail(DPG_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
    if (!aligned(p, dtype == DPG_BF16 ? 2 : 4)) return fail(DPG_ERR_MISALIGNED, "%s: %s misaligned", who, name);
    if (rows > 1 && (stride < cols || stride > (int64_t(1) << 40)))
        return fail(DPG_ERR_INVALID_ARG, "%s: row stride %lld of %s, which has %lld columns", who, (long long)stride,
                    name, (long long)cols);
    return DPG_OK;
}

// checks one quantisation and fills `a`, whose seed is the caller's
static int quant_args(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                      const dpg_fp4* by_row, const dpg_fp4* by_col, QuantArgs& a, const char* who) {
    if (!by_row && !by_col) return fail(DPG_ERR_INVALID_ARG, "%s: by_row and by_col are NULL", who);
    for (int side = 0; side < 2; ++side) {
        const dpg_fp4* q = side ? by_col : by_row;
        if (!q) continue;
        const char* name = side ? "by_col" : "by_row";
        const int st = fp4_check(q, name, who);
        if (st != DPG_OK) return st;
        if (q->rows != (side ? cols : rows) || q->cols != (side ? rows : cols))
            return fail(DPG_ERR_INVALID_ARG, "%s: %s is %lld x %lld, x %lld x %lld", who, name, (long long)q->rows,
                        (long long)q->cols, (long long)rows, (long long)cols);
        QuantSide& s = side ? a.col : a.row;
        s.codes = static_cast<unsigned char*>(q->codes);
        s.scales = static_cast<unsigned char*>(q->scales);
        s.pitch = fp4_pitch(q->cols);
        s.tiles = fp4_tiles(q->cols, q->format);
        s.vectors = (q->cols + 7) / 8;
    }
    if (by_row && by_col) {
        if (by_row->format != by_col->format)
            return fail(DPG_ERR_INVALID_ARG, "%s: by_row and by_col have different formats", who);
        if (rows > 0 && cols > 0 && (by_row->codes == by_col->codes || by_row->scales == by_col->scales))
            return fail(DPG_ERR_INVALID_ARG, "%s: by_row and by_col share a buffer", who);
    }
    const int st = strided_check(x, dtype, rows, cols, stride, "x", who);
    if (st != DPG_OK) return st;
    const dpg_fp4* first = by_row ? by_row : by_col;
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.stride = rows > 1 ? stride : cols;
    a.tiles_c = (cols + kQuantTile - 1) / kQuantTile;
    a.vec = aligned(x, 16) && (rows <= 1 || stride % (dtype == DPG_F32 ? 4 : 8) == 0);
    a.amax = first->amax;
    a.amax_copy = by_row && by_col && by_col->amax != by_row->amax ? by_col->amax : nullptr;
    if ((rows + kQuantTile - 1) / kQuantTile * a.tiles_c > 0x7FFFFFFF)
        return fail(DPG_ERR_INVALID_ARG, "%s: %lld x %lld elements in one call", who, (long long)rows, (long long)cols);
    return DPG_OK;
}

// Whether every buffer of n matrices lies apart from the others: a matrix quantised
// later would take the place of an earlier one's. (One matrix's two forms may have one
// amax: it is the same number.)
static int fp4_apart(const dpg_fp4* by_row, const dpg_fp4* by_col, int32_t n, const char* who) {
    struct Span {
        uintptr_t at, end;
        int32_t amax_of;               // -1: codes or scales
    };
    try {
        std::vector<Span> spans;
        spans.reserve(size_t(n) * 6);
        for (const dpg_fp4* side : {by_row, by_col})
            for (int32_t k = 0; side && k < n; ++k) {
                const dpg_fp4& q = side[k];
                const uintptr_t codes = reinterpret_cast<uintptr_t>(q.codes), scales = reinterpret_cast<uintptr_t>(q.scales),
                                amax = reinterpret_cast<uintptr_t>(q.amax);
                spans.push_back({codes, codes + uintptr_t(q.rows * fp4_pitch(q.cols)), -1});
                spans.push_back({scales, scales + uintptr_t((q.rows + kFp4TileRows - 1) / kFp4TileRows *
                                                            fp4_tiles(q.cols, q.format) * kFp4TileBytes), -1});
                if (q.format == DPG_NVFP4) spans.push_back({amax, amax + DPG_FP4_AMAX_FLOATS * sizeof(float), k});
            }
        std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.at < b.at; });
        for (size_t i = 1; i < spans.size(); ++i) {
            const Span &a = spans[i - 1], &b = spans[i];
            if (b.at < a.end && !(a.at == b.at && a.amax_of >= 0 && a.amax_of == b.amax_of))
                return fail(DPG_ERR_INVALID_ARG, "%s: two of the 4-bit matrices share a buffer", who);
        }
    } catch (const std::exception&) {
        return fail(DPG_ERR_OOM, "%s: out of host memory", who);
    }
    return DPG_OK;
}

template <bool F32, bool MX, bool SR>
static int launch_quant(const QuantArgs& a, int64_t tiles, cudaStream_t s, const char* who) {
    auto k = k_fp4_quantize<F32, MX, SR>;
    const int smem = quant_smem<F32>();
    static std::atomic<uint64_t> once{0};
    const int st = allow_smem(reinterpret_cast<const void*>(k), smem, once, who);
    if (st != DPG_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(tiles));
    cfg.blockDim = dim3(TileOf<F32, SR>::kThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (t_programmatic) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (!MX && !a.parts && tiles > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = unsigned(tiles);
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, a);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return fail(DPG_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    }
    return after_launch(who);
}

static int quantize(QuantArgs& a, int32_t dtype, int32_t format, cudaStream_t s, const char* who) {
    if (a.rows == 0 || a.cols == 0) return DPG_OK;
    const bool f32 = dtype == DPG_F32, mx = format == DPG_MXFP4;
    const int64_t tiles = (a.rows + kQuantTile - 1) / kQuantTile * a.tiles_c;
    // up to 8 tiles are one cluster, whose CTAs find the largest magnitude among themselves
    if (!mx && tiles > 8) {
        const int64_t n = a.rows * a.cols;
        const int per = f32 ? 4 : 8;
        const bool flat = a.stride == a.cols;
        const int64_t pieces = flat ? 0 : (a.cols + per - 1) / per + (a.vec ? 0 : 1);
        const int64_t want = (n + 16383) / 16384;
        a.parts = int32_t(want < kAmaxCtas ? want : kAmaxCtas);
        const int st = launch_k(f32 ? k_fp4_amax<true> : k_fp4_amax<false>, unsigned(a.parts), kAmaxThreads, s, who, a.x, a.rows,
                                a.cols, a.stride, pieces, reinterpret_cast<uint32_t*>(a.amax) + 1);
        if (st != DPG_OK) return st;
    }
    const int which = (f32 ? 4 : 0) + (mx ? 2 : 0) + (a.seed ? 1 : 0);
    switch (which) {
        case 0: return launch_quant<false, false, false>(a, tiles, s, who);
        case 1: return launch_quant<false, false, true>(a, tiles, s, who);
        case 2: return launch_quant<false, true, false>(a, tiles, s, who);
        case 3: return launch_quant<false, true, true>(a, tiles, s, who);
        case 4: return launch_quant<true, false, false>(a, tiles, s, who);
        case 5: return launch_quant<true, false, true>(a, tiles, s, who);
        case 6: return launch_quant<true, true, false>(a, tiles, s, who);
        default: return launch_quant<true, true, true>(a, tiles, s, who);
    }
}

}  // namespace dpg

using dpg::fail;

extern "C" {

int dpg_fp4_sizes(int64_t rows, int64_t cols, int32_t format, int64_t* code_bytes, int64_t* scale_bytes) {
    dpg::clear_error();
    const int st = dpg::fp4_shape(rows, cols, format, "the matrix", "dpg_fp4_sizes");
    if (st != DPG_OK) return st;
    if (code_bytes) *code_bytes = rows * dpg::fp4_pitch(cols);
    if (scale_bytes)
        *scale_bytes = (rows + dpg::kFp4TileRows - 1) / dpg::kFp4TileRows * dpg::fp4_tiles(cols, format) *
                       dpg::kFp4TileBytes;
    return DPG_OK;
}

int dpg_fp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t row_stride,
                     const int64_t* seed, const dpg_fp4* by_row, const dpg_fp4* by_col, void* stream) {
    dpg::clear_error();
    const dpg::Trace trace("dpg_fp4_quantize");
    dpg::QuantArgs a{};
    const int st = dpg::quant_args(x, x_dtype, rows, cols, row_stride, by_row, by_col, a, "dpg_fp4_quantize");
    if (st != DPG_OK) return st;
    if (seed && !dpg::aligned(seed, 8)) return fail(DPG_ERR_MISALIGNED, "dpg_fp4_quantize: seed misaligned");
    a.seed = seed;
    return dpg::quantize(a, x_dtype, (by_row ? by_row : by_col)->format, static_cast<cudaStream_t>(stream),
                         "dpg_fp4_quantize");
}

int dpg_fp4_dequantize(const dpg_fp4* q, void* out, int32_t out_dtype, int64_t row_stride, void* stream) {
    dpg::clear_error();
    const dpg::Trace trace("dpg_fp4_dequantize");
    if (!q) return fail(DPG_ERR_INVALID_ARG, "dpg_fp4_dequantize: q is NULL");
    int st = dpg::fp4_check(q, "q", "dpg_fp4_dequantize");
    if (st == DPG_OK)
        st = dpg::strided_check(out, out_dtype, q->rows, q->cols, row_stride, "out", "dpg_fp4_dequantize");
    if (st != DPG_OK) return st;
    if (q->rows == 0 || q->cols == 0) return DPG_OK;
    dpg::DequantArgs a{};
    a.codes = static_cast<const unsigned char*>(q->codes);
    a.scales = static_cast<const unsigned char*>(q->scales);
    a.amax = q->amax;
    a.rows = q->rows;
    a.cols = q->cols;
    a.pitch = dpg::fp4_pitch(q->cols);
    a.tiles = dpg::fp4_tiles(q->cols, q->format);
    a.stride = q->rows > 1 ? row_stride : q->cols;
    a.out = out;
    // one more where a row may start inside a piece
    const bool whole = dpg::aligned(out, out_dtype == DPG_F32 ? 64 : 32) && (q->rows <= 1 || row_stride % dpg::kPiece == 0);
    a.pieces = (q->cols + dpg::kPiece - 1) / dpg::kPiece + (whole ? 0 : 1);
    int grid = 0;
    st = dpg::grid_cover((a.rows * a.pieces + 255) / 256, &grid, "dpg_fp4_dequantize");
    if (st != DPG_OK) return st;
    const bool mx = q->format == DPG_MXFP4;
    auto k = out_dtype == DPG_F32 ? (mx ? dpg::k_fp4_dequantize<true, true> : dpg::k_fp4_dequantize<true, false>)
                                  : (mx ? dpg::k_fp4_dequantize<false, true> : dpg::k_fp4_dequantize<false, false>);
    return dpg::launch_k(k, unsigned(grid), 256, static_cast<cudaStream_t>(stream), "dpg_fp4_dequantize", a);
}

int dpg_allgather_params_fp4(const dpg_matrices_t* mats, const float* master, const int64_t* seed,
                             const dpg_fp4* by_row, const dpg_fp4* by_col, int32_t n, void* stream) {
    dpg::clear_error();
    const char* who = "dpg_allgather_params_fp4";
    const dpg::Trace trace(who);
    if (!mats) return fail(DPG_ERR_INVALID_ARG, "%s: mats is NULL", who);
    const dpg::Matrices& m = mats->m;
    if (n != m.n_matrices)
        return fail(DPG_ERR_INVALID_ARG, "%s: %d matrices, the object has %d", who, n, m.n_matrices);
    if (!by_row && !by_col) return fail(DPG_ERR_INVALID_ARG, "%s: by_row and by_col are NULL", who);
    if (n == 0) return DPG_OK;
    if (!master) return fail(DPG_ERR_INVALID_ARG, "%s: master is NULL", who);
    if (!dpg::aligned(master, 32)) return fail(DPG_ERR_MISALIGNED, "%s: master misaligned", who);
    if (seed && !dpg::aligned(seed, 8)) return fail(DPG_ERR_MISALIGNED, "%s: seed misaligned", who);
    for (int pass = 0; pass < 2; ++pass) {               // all are checked before the first is launched
        if (pass == 1) {
            const int st = dpg::fp4_apart(by_row, by_col, n, who);
            if (st != DPG_OK) return st;
        }
        int32_t k = 0;
        for (int32_t q = 0; q < m.n_params; ++q) {
            const int64_t r = m.rows[size_t(q)], c = m.cols[size_t(q)];
            for (int64_t e = 0; e < m.numels[size_t(q)]; e += r * c, ++k) {
                dpg::QuantArgs a{};
                const dpg_fp4 *br = by_row ? by_row + k : nullptr, *bc = by_col ? by_col + k : nullptr;
                int st = dpg::quant_args(master + m.param_offset[size_t(q)] + e, DPG_F32, r, c, c, br, bc, a, who);
                if (st != DPG_OK) return st;
                a.seed = seed;
                a.seed_plus = k;
                if (pass == 1)
                    st = dpg::quantize(a, DPG_F32, (br ? br : bc)->format, static_cast<cudaStream_t>(stream), who);
                if (st != DPG_OK) return st;
            }
        }
    }
    return DPG_OK;
}

}  // extern "C"
