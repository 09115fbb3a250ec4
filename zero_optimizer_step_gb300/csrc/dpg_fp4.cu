// dpg_fp4.cu -- quantisation to 4-bit floating point and back (see
// dpg_fp4_quantize, dpg_fp4_dequantize and dpg_allgather_params_fp4 in
// include/dpg.h).
//
// A block of 16 (or 32) elements x has the scale s = the least E4M3 (E8M0) value
// with max|x| <= 6 s, and the codes nearest to x / s on 0, .5, 1, 1.5, 2, 3, 4, 6.
// Every decision is exact:
//   * s by a product with 1/6 rounded up, then compared with its neighbours
//     through 6 s, which is exact;
//   * x / s for an E8M0 scale is a product with a power of two; for an E4M3 one
//     it is the correctly rounded quotient, from the reciprocal and one residual
//     (Markstein 1990).  A borderline m s has at most 7 bits, so a quotient whose
//     x is not on it rounds to something else than m, and ties stay ties.  The
//     product with the reciprocal alone is off by one unit for 11 of the 56
//     borderlines, and would round those ties up.
//   * stochastic: |x| - lo s and (2 u + 1) 2^-17 gap s are exact in fp32.
#include <cuda_fp4.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "dpg_fp4.h"
#include "dpg_host.h"
#include "dpg_ortho.h"

namespace dpg {

constexpr int kQuantThreads = 256;
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
    const float* amax;                  // where k_fp4_amax left it
    float* amax_copy;                   // the other side's (NULL: none)
    QuantSide row, col;
};

// ---------------------------------------------------------------------------
// Largest finite magnitude, as the bits of an fp32 number: these order like the
// numbers, and a maximum is the same in any order.
// ---------------------------------------------------------------------------
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
__global__ void __launch_bounds__(256) k_fp4_amax(const void* x, int64_t rows, int64_t cols, int64_t stride,
                                                  int32_t flat16, uint32_t* amax) {
    pdl_enter();
    uint32_t m = 0;
    const int64_t step = int64_t(gridDim.x) * 256, t = int64_t(blockIdx.x) * 256 + threadIdx.x;
    constexpr int kPer = F32 ? 4 : 8;   // elements of 16 bytes
    if (flat16) {                       // rows back to back, from a 16-byte boundary
        const int64_t n = rows * cols, vecs = n / kPer;
        const unsigned char* p = static_cast<const unsigned char*>(x);
        int64_t i = t;
        for (; i + 3 * step < vecs; i += 4 * step) {
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = *reinterpret_cast<const uint4*>(p + (i + u * step) * 16);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                m = max(max(m, max(magnitude_bits<F32>(v[u].x), magnitude_bits<F32>(v[u].y))),
                        max(magnitude_bits<F32>(v[u].z), magnitude_bits<F32>(v[u].w)));
        }
        for (; i < vecs; i += step) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + i * 16);
            m = max(max(m, max(magnitude_bits<F32>(v.x), magnitude_bits<F32>(v.y))),
                    max(magnitude_bits<F32>(v.z), magnitude_bits<F32>(v.w)));
        }
        for (int64_t j = vecs * kPer + t; j < n; j += step)
            m = max(m, F32 ? magnitude_bits<true>(static_cast<const uint32_t*>(x)[j])
                           : magnitude_bits<false>(static_cast<const uint16_t*>(x)[j]));
    } else {
        for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
            for (int64_t c = threadIdx.x; c < cols; c += 256)
                m = max(m, F32 ? magnitude_bits<true>(static_cast<const uint32_t*>(x)[r * stride + c])
                               : magnitude_bits<false>(static_cast<const uint16_t*>(x)[r * stride + c]));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0 && m) atomicMax(amax, m);
}

// ---------------------------------------------------------------------------
// One block
// ---------------------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011)
__device__ __forceinline__ uint4 philox(uint64_t n, uint32_t side, uint64_t key) {
    uint32_t x0 = uint32_t(n), x1 = uint32_t(n >> 32), x2 = side, x3 = 0, k0 = uint32_t(key),
             k1 = uint32_t(key >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint32_t a = __umulhi(0xD2511F53u, x0), b = 0xD2511F53u * x0;
        const uint32_t c = __umulhi(0xCD9E8D57u, x2), d = 0xCD9E8D57u * x2;
        x0 = c ^ x1 ^ k0;
        x2 = a ^ x3 ^ k1;
        x1 = d;
        x3 = b;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

// E4M3 value of a byte (0 .. 0x7E)
__device__ __forceinline__ float e4m3_value(int byte) {
    return byte < 8 ? float(byte) * 0.001953125f : __uint_as_float(uint32_t(byte + 960) << 20);
}

struct BlockScale {
    int byte;          // as stored
    float s, inv;      // its value, and about 1 / s (0 for s = 0); inv alone for E8M0
    bool bad;          // a NaN or an infinity in the block
};

// of a block whose largest magnitude has the bits `top`; `unit` = 2^-e (E4M3)
template <bool MX>
__device__ __forceinline__ BlockScale block_scale(uint32_t top, float unit) {
    BlockScale b;
    b.bad = top >= 0x7F800000u;
    if (MX) {
        const int e = int(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
        b.byte = b.bad ? 0xFF : e < 0 ? 0 : e;
        b.inv = b.bad ? 0.0f : __uint_as_float(uint32_t(254 - b.byte) << 23);
        b.s = __uint_as_float(b.byte == 0 ? 0x00400000u : uint32_t(b.byte) << 23);
        return b;
    }
    const float u = __uint_as_float(top) * unit;
    const float q = u * 0.166666672f;                   // 1/6 rounded up
    int k;
    if (q < 0.015625f)
        k = int(ceilf(q * 512.0f));
    else
        k = int((__float_as_uint(q) + 0xFFFFFu) >> 20) - 960;
    k = k > 0x7E ? 0x7E : k;
    if (k > 0 && 6.0f * e4m3_value(k - 1) >= u) --k;
    else if (k < 0x7E && 6.0f * e4m3_value(k) < u) ++k;
    b.s = e4m3_value(k);
    b.inv = b.bad || k == 0 ? 0.0f : 1.0f / b.s;
    b.byte = b.bad ? 0x7F : k;
    return b;
}

// two codes, x in the low half
__device__ __forceinline__ uint32_t nearest2(float x, float y) {
    return __nv_cvt_float2_to_fp4x2(make_float2(x, y), __NV_E2M1, cudaRoundNearest);
}

// code of v >= 0 (already times 2^-e), to the value above where the 16 bits u say so
template <bool MX>
__device__ __forceinline__ uint32_t stochastic(float v, const BlockScale& b, uint32_t u) {
    const float y = v * b.inv;
    // lo = y with one bit behind the point of its binade, in halves below 1
    const uint32_t bits = __float_as_uint(y);
    const bool small = y < 1.0f;
    const bool half = y >= 0.5f;
    const float lo = small ? (half ? 0.5f : 0.0f) : __uint_as_float(bits & 0xFFC00000u);
    const uint32_t code = small ? (half ? 1u : 0u) : (bits >> 22) - 252u;
    const float gap = y < 2.0f ? 0.5f : y < 4.0f ? 1.0f : 2.0f;
    const float t = (2.0f * float(u) + 1.0f) * 7.62939453125e-6f * gap;
    // an E8M0 scale: in units of s, exactly; else v - lo s and t s are exact.  (Where the rounding
    // of y took it to a neighbour of the right lo, the comparison still ends at the right code:
    // the distance to it is below or above every threshold.)
    return code + (MX ? y - lo > t : fmaf(-lo, b.s, v) > t * b.s ? 1u : 0u);
}

// N consecutive elements of a block (N a multiple of 8) to codes, 8 to a word.
// n0: number of the first group of 8 (random bits); x: values times 2^-e where
// E4M3.
template <bool MX, bool SR, int N>
__device__ __forceinline__ void encode(const float* x, const BlockScale& b, uint64_t n0, uint32_t side,
                                       uint64_t key, uint32_t* out) {
#pragma unroll
    for (int w = 0; w < N / 8; ++w) {
        const float* v = x + 8 * w;
        uint32_t word = 0;
        if (SR) {
            const uint4 r = philox(n0 + w, side, key);
            const uint32_t h[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = (j & 1) ? h[j >> 1] >> 16 : h[j >> 1] & 0xFFFFu;
                const uint32_t c = stochastic<MX>(fabsf(v[j]), b, u);
                word |= (c | (__float_as_uint(v[j]) >> 28 & 8u)) << (4 * j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y0 = v[2 * j] * b.inv, y1 = v[2 * j + 1] * b.inv;
                if (!MX) {
                    y0 = fmaf(fmaf(-y0, b.s, v[2 * j]), b.inv, y0);
                    y1 = fmaf(fmaf(-y1, b.s, v[2 * j + 1]), b.inv, y1);
                }
                word |= nearest2(y0, y1) << (8 * j);
            }
        }
        out[w] = b.bad ? 0u : word;
    }
}

// ---------------------------------------------------------------------------
// Both orientations from one read.  A CTA takes 128 x 128 elements: rows from
// registers as they were loaded, columns from shared memory.
// ---------------------------------------------------------------------------
template <bool F32>
struct TileOf {
    static constexpr int kPitch = F32 ? 132 : 68;          // words of a row in shared memory
    static constexpr int kBytes = kQuantTile * kPitch * 4;
};
constexpr int kColPitch = 80;                              // bytes of a column's codes in shared memory

template <bool F32, bool MX>
constexpr int quant_smem() { return TileOf<F32>::kBytes + kQuantTile * kColPitch; }

template <bool F32, bool MX, bool SR>
__global__ void __launch_bounds__(kQuantThreads) k_fp4_quantize(const __grid_constant__ QuantArgs a) {
    constexpr int B = MX ? 32 : 16;                        // elements of a block
    constexpr int kBlocks = kQuantTile / B;                // blocks of a tile's row
    constexpr int kTasks = kQuantTile * kBlocks / kQuantThreads;
    constexpr int kWords = B * (F32 ? 4 : 2) / 4;          // 32-bit words of a block
    constexpr int kTiles = kBlocks / 4;                    // scale tiles of a tile
    extern __shared__ __align__(16) uint32_t tile[];
    __shared__ __align__(16) unsigned char sc[2][kTiles * kFp4TileBytes];
    unsigned char* const out = reinterpret_cast<unsigned char*>(tile) + TileOf<F32>::kBytes;
    pdl_enter();
    const int64_t ti = blockIdx.x / a.tiles_c, tj = blockIdx.x % a.tiles_c;
    const int64_t r0 = ti * kQuantTile, c0 = tj * kQuantTile;
    const int tid = int(threadIdx.x);
    const bool by_row = a.row.codes != nullptr, by_col = a.col.codes != nullptr;
    float unit = 1.0f;
    if (!MX) {
        const float amax = __ldcg(a.amax);
        unit = __uint_as_float(uint32_t(127 - fp4_exponent(__float_as_uint(amax))) << 23);
        if (a.amax_copy && blockIdx.x == 0 && tid == 0) *a.amax_copy = amax;
    }
    const uint64_t key = SR ? uint64_t(__ldg(a.seed) + a.seed_plus) : 0;

    uint32_t raw[kTasks][kWords];
#pragma unroll
    for (int k = 0; k < kTasks; ++k) {
        const int task = k * kQuantThreads + tid, row = task / kBlocks, blk = task % kBlocks;
        const int64_t r = r0 + row, c = c0 + blk * B;
        const int64_t at = r * a.stride + c;
        if (r < a.rows && c + B <= a.cols && a.vec) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.x) + at * (F32 ? 4 : 2));
#pragma unroll
            for (int j = 0; j < kWords / 4; ++j) {
                const uint4 v = ld_grad_u4(p + j);
                raw[k][4 * j] = v.x;
                raw[k][4 * j + 1] = v.y;
                raw[k][4 * j + 2] = v.z;
                raw[k][4 * j + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                if (F32) {
                    raw[k][j] = r < a.rows && c + j < a.cols ? __ldg(static_cast<const uint32_t*>(a.x) + at + j) : 0u;
                } else {
                    const uint16_t* p = static_cast<const uint16_t*>(a.x) + at + 2 * j;
                    const uint32_t lo = r < a.rows && c + 2 * j < a.cols ? __ldg(p) : 0u;
                    const uint32_t hi = r < a.rows && c + 2 * j + 1 < a.cols ? __ldg(p + 1) : 0u;
                    raw[k][j] = lo | hi << 16;
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kTasks; ++k) {
        const int task = k * kQuantThreads + tid, row = task / kBlocks, blk = task % kBlocks;
        if (by_col) {
            uint4* p = reinterpret_cast<uint4*>(tile + row * TileOf<F32>::kPitch + blk * kWords);
#pragma unroll
            for (int j = 0; j < kWords / 4; ++j)
                p[j] = make_uint4(raw[k][4 * j], raw[k][4 * j + 1], raw[k][4 * j + 2], raw[k][4 * j + 3]);
        }
        if (!by_row) continue;
        const int64_t r = r0 + row, c = c0 + blk * B;
        float x[B];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            x[j] = F32 ? __uint_as_float(raw[k][j])
                       : __uint_as_float((j & 1) ? raw[k][j >> 1] & 0xFFFF0000u : raw[k][j >> 1] << 16);
            top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        }
        const BlockScale b = block_scale<MX>(top, unit);
        if (!MX) {
#pragma unroll
            for (int j = 0; j < B; ++j) x[j] *= unit;
        }
        uint32_t codes[B / 8];
        encode<MX, SR, B>(x, b, uint64_t(r) * a.row.vectors + uint64_t(c >> 3), 0, key, codes);
        if (r < a.rows && c < a.cols) {
            unsigned char* p = a.row.codes + r * a.row.pitch + (c >> 1);
            if (MX) *reinterpret_cast<uint4*>(p) = make_uint4(codes[0], codes[1], codes[B / 8 - 2], codes[B / 8 - 1]);
            else if ((blk & 1) == 0 && c + B >= a.cols) *reinterpret_cast<uint4*>(p) = make_uint4(codes[0], codes[1], 0, 0);
            else *reinterpret_cast<uint2*>(p) = make_uint2(codes[0], codes[1]);
        }
        sc[0][(blk >> 2) * kFp4TileBytes + (row & 31) * 16 + (row >> 5) * 4 + (blk & 3)] =
            static_cast<unsigned char>(r < a.rows && c < a.cols ? b.byte : 0);
    }
    __syncthreads();
    if (by_col) {
        // two neighbouring columns and one block of rows to a task
        constexpr int kColTasks = kQuantTile / 2 * kBlocks / kQuantThreads;
#pragma unroll 1
        for (int k = 0; k < kColTasks; ++k) {
            const int task = k * kQuantThreads + tid, pair = task % (kQuantTile / 2), blk = task / (kQuantTile / 2);
            const int64_t r = r0 + blk * B;
            float x[2][B];
            uint32_t top[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const uint32_t* p = tile + (blk * B + j) * TileOf<F32>::kPitch;
                if (F32) {
                    const uint2 v = *reinterpret_cast<const uint2*>(p + 2 * pair);
                    x[0][j] = __uint_as_float(v.x);
                    x[1][j] = __uint_as_float(v.y);
                } else {
                    widen2(p[pair], x[0][j], x[1][j]);
                }
                top[0] = max(top[0], __float_as_uint(x[0][j]) & 0x7FFFFFFFu);
                top[1] = max(top[1], __float_as_uint(x[1][j]) & 0x7FFFFFFFu);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = 2 * pair + h;
                const int64_t c = c0 + col;
                const BlockScale b = block_scale<MX>(top[h], unit);
                if (!MX) {
#pragma unroll
                    for (int j = 0; j < B; ++j) x[h][j] *= unit;
                }
                uint32_t codes[B / 8];
                encode<MX, SR, B>(x[h], b, uint64_t(c) * a.col.vectors + uint64_t(r >> 3), 1, key, codes);
                uint32_t* p = reinterpret_cast<uint32_t*>(out + col * kColPitch + blk * (B / 2));
#pragma unroll
                for (int j = 0; j < B / 8; ++j) p[j] = codes[j];
                sc[1][(blk >> 2) * kFp4TileBytes + (col & 31) * 16 + (col >> 5) * 4 + (blk & 3)] =
                    static_cast<unsigned char>(c < a.cols && r < a.rows ? b.byte : 0);
            }
        }
        __syncthreads();
        for (int k = tid; k < kQuantTile * 4; k += kQuantThreads) {      // 16 bytes: 32 rows of a column
            const int col = k >> 2, part = k & 3;
            if (c0 + col < a.cols && r0 + part * 32 < a.rows)
                *reinterpret_cast<uint4*>(a.col.codes + (c0 + col) * a.col.pitch + (r0 >> 1) + part * 16) =
                    *reinterpret_cast<const uint4*>(out + col * kColPitch + part * 16);
        }
    }
    for (int k = tid; k < 2 * kTiles * 32; k += kQuantThreads) {
        const int side = k / (kTiles * 32), t = k / 32 % kTiles, part = k % 32;
        const QuantSide& q = side ? a.col : a.row;
        const int64_t i = side ? tj : ti, j = (side ? ti : tj) * kTiles + t;
        if (q.codes && j < q.tiles)
            *reinterpret_cast<uint4*>(q.scales + (i * q.tiles + j) * kFp4TileBytes + part * 16) =
                *reinterpret_cast<const uint4*>(sc[side] + t * kFp4TileBytes + part * 16);
    }
}

// ---------------------------------------------------------------------------
// Values of a quantised matrix: a thread takes 32 elements of a row.
// ---------------------------------------------------------------------------
struct DequantArgs {
    const unsigned char* codes;
    const unsigned char* scales;
    const float* amax;
    int64_t rows, cols, pitch, tiles, stride, chunks;   // chunks: of 32 elements in a row
    void* out;
    int32_t vec;                                        // 16-byte stores are allowed
};

template <bool F32, bool MX>
__global__ void __launch_bounds__(256) k_fp4_dequantize(const __grid_constant__ DequantArgs a) {
    pdl_enter();
    const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t r = t / a.chunks, ch = t % a.chunks;
    if (r >= a.rows) return;
    const uint4 q = ld_grad_u4(a.codes + r * a.pitch + ch * 16);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const unsigned char* sp = a.scales + (r >> 7) * a.tiles * kFp4TileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
    float s[2];
    if (MX) {
        const int byte = __ldg(sp + (ch >> 2) * kFp4TileBytes + (ch & 3));
        s[0] = s[1] = byte == 0xFF ? __uint_as_float(0x7FC00000u)
                                   : __uint_as_float(byte == 0 ? 0x00400000u : uint32_t(byte) << 23);
    } else {
        const float unit = __uint_as_float(0x3F800000u + uint32_t(fp4_exponent(__float_as_uint(__ldg(a.amax)))) * 0x800000u);
        const uint32_t two = __ldg(reinterpret_cast<const unsigned short*>(sp + (ch >> 1) * kFp4TileBytes + (ch & 1) * 2));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int byte = int(two >> (8 * h)) & 0xFF;
            s[h] = byte == 0x7F ? __uint_as_float(0x7FC00000u) : e4m3_value(byte) * unit;
        }
    }
    const int n = int(min(int64_t(32), a.cols - ch * 32));
    const int64_t at = r * a.stride + ch * 32;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t c = w[g] >> (4 * j), m = c & 7u;
            // .5 m below 2 (0, .5, 1, 1.5), else (2 + low bit) 2^(m / 2 - 2)
            const float f = m < 2 ? 0.5f * float(m) : __uint_as_float((252u + m) << 22);
            v[j] = ((c & 8u) ? -f : f) * s[g >> 1];
        }
        if (F32) {
            float* p = static_cast<float*>(a.out) + at + 8 * g;
            if (a.vec && 8 * g + 8 <= n) {
                *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * g + j < n) p[j] = v[j];
            }
        } else {
            uint16_t* p = static_cast<uint16_t*>(a.out) + at + 8 * g;
            const uint4 h = narrow8(v);
            if (a.vec && 8 * g + 8 <= n) {
                st_u4(p, h);
            } else {
                const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * g + j < n) p[j] = uint16_t(hw[j >> 1] >> (16 * (j & 1)));
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

template <bool F32, bool MX>
static int launch_quant(const QuantArgs& a, cudaStream_t s, const char* who) {
    auto k = a.seed ? k_fp4_quantize<F32, MX, true> : k_fp4_quantize<F32, MX, false>;
    const int smem = a.col.codes ? quant_smem<F32, MX>() : 0;
    if (smem > 48 * 1024) DPG_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    const int64_t tiles = (a.rows + kQuantTile - 1) / kQuantTile * a.tiles_c;
    return launch_k(k, unsigned(tiles), kQuantThreads, size_t(smem), s, who, a);
}

static int quantize(const QuantArgs& a, int32_t dtype, int32_t format, cudaStream_t s, const char* who) {
    if (a.rows == 0 || a.cols == 0) return DPG_OK;
    if (format == DPG_NVFP4) {
        uint32_t* amax = reinterpret_cast<uint32_t*>(const_cast<float*>(a.amax));
        DPG_CUDA_TRY(cudaMemsetAsync(amax, 0, sizeof(uint32_t), s));
        int dev = 0, sms = 0;
        DPG_CUDA_TRY(cudaGetDevice(&dev));
        int st = sm_count(dev, &sms);
        if (st != DPG_OK) return st;
        const int64_t n = a.rows * a.cols;
        const int flat16 = a.stride == a.cols && aligned(a.x, 16);
        const int64_t want = flat16 ? (n + 8191) / 8192 : a.rows;
        const unsigned grid = unsigned(want < 1 ? 1 : want < 8 * sms ? want : 8 * sms);
        st = launch_k(dtype == DPG_F32 ? k_fp4_amax<true> : k_fp4_amax<false>, grid, 256, s, who, a.x, a.rows, a.cols,
                      a.stride, int32_t(flat16), amax);
        if (st != DPG_OK) return st;
    }
    if (dtype == DPG_F32)
        return format == DPG_MXFP4 ? launch_quant<true, true>(a, s, who) : launch_quant<true, false>(a, s, who);
    return format == DPG_MXFP4 ? launch_quant<false, true>(a, s, who) : launch_quant<false, false>(a, s, who);
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
    a.chunks = (q->cols + 31) / 32;
    a.stride = q->rows > 1 ? row_stride : q->cols;
    a.out = out;
    a.vec = dpg::aligned(out, 16) && (q->rows <= 1 || row_stride % (out_dtype == DPG_F32 ? 4 : 8) == 0);
    int grid = 0;
    st = dpg::grid_cover((a.rows * a.chunks + 255) / 256, &grid, "dpg_fp4_dequantize");
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
