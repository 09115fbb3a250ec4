// dpg_fp4_product.cu -- products of 4-bit quantised matrices on the tensor cores
// (see dpg_fp4_product in include/dpg.h).
//
// C = A B^T, both operands stored along the sum.  A tcgen05.mma of 4-bit kind
// takes 64 elements of each row (32 bytes) and their scales: 4 for blocks of 16,
// 2 for blocks of 32; codes come from shared memory (rows of 256 elements, 128
// bytes, 128-byte swizzle), scales from tensor memory, where tcgen05.cp brings
// a tile of 128 rows x 4 scales as it is stored (32 lanes x 16 bytes, copied to
// the four quarters of the lanes).  Sums are fp32 in tensor memory; the matrices'
// powers of two are applied to them at the end.
//
// Small products are bound by latency: 3.6 us for one tile of one stage (launch,
// tensor maps, tensor memory, first copy, results), 0.2 us for each further stage,
// and 1 to 2 us where CTAs exchange parts of a sum (8 x 14336 x 4096 6.7 us, 4.9 of
// them the weight's bytes; 4096 x 2304 x 768 7.5).  Large ones by what their ring of
// stages holds: see k_fp4_large.  Times in this file are of a loop over one set of
// operands, which lie in L2 where they fit; among other calls those two take 7.6 and 7.7,
// and 8192 x 14336 x 4096 takes 169 to 174 instead of 152.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <exception>
#include <map>
#include <mutex>
#include <utility>

#include "dpg_async.cuh"
#include "dpg_fp4.h"
#include "dpg_host.h"

namespace dpg {

constexpr int kProdDepth = 256;                  // elements of the sum in a stage
constexpr int kCodeRow = kProdDepth / 2;         // bytes of a row in a stage
constexpr int kRowTile = 128;                    // rows of an operand in a CTA
constexpr int kStoreBytes = 4096;                // of a storing warp: two boxes, or 32 x 32 sums
constexpr int kScaleBytes = 2048;                // room for the scales of 128 rows in a stage
constexpr uint64_t kProdWaitNs = 2000000000ull;  // bound of every wait, unless a test sets another

// Waits that ran out on this device since the library was loaded.  It only counts
// up: whoever asks compares it with what it saw before, so nothing that one stream
// reads, and no failure that comes meanwhile, is lost to another.
__device__ uint32_t g_fp4_failures;

struct ProductArgs {
    void* c;
    int64_t stride;
    const float* amax_a;         // DPG_NVFP4: of the operands
    const float* amax_b;
    int32_t m, n, k;
    int32_t c_f32, add;
    int32_t vec;                 // 16-byte accesses of C's rows are allowed
    int32_t boxes;               // bulk copies too: they write whole 16-byte pieces, also at a row's end
    int32_t wide;                // 32-byte stores, of whole pieces (not where C is added to)
    int32_t rows, cols;          // of the product as it is computed (its transpose if `swap`)
    int32_t tiles_r, tiles_c;
    int32_t swap;                // rows are C's columns
    int32_t split;               // CTAs (of one cluster) that share a sum
    uint64_t wait_ns;
    int64_t skip;                // test only: the first CTA leaves out this stage's first copy (-1: none)
};

struct ProductMaps {
    CUtensorMap codes_r, codes_c, scales_r, scales_c;
    CUtensorMap result;          // C, where `boxes`
};

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ void give_up(volatile int* abort) {
    *abort = 1;
    atomicAdd(&g_fp4_failures, 1u);
}
// true once the phase of `parity` completed; false when the bound ran out or
// another role of the CTA gave up
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t ns) {
    const uint32_t at = smem_u32(bar);
    if (try_wait(at, parity)) return true;
    const uint64_t until = global_ns() + ns;
    while (!try_wait(at, parity)) {
        if (*abort) return false;
        if (global_ns() > until) {
            give_up(abort);
            return false;
        }
    }
    return true;
}
// One lane of a warp.  What the warp computes before it stays in uniform
// registers, where the instructions want their operands: under `lane == 0` each
// was moved there on its own, 74 cycles to a copy of scales.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void copy_tile(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// 128-byte rows y .. of row of tiles z
__device__ __forceinline__ void copy_scale_rows(uint32_t dst, const CUtensorMap* map, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void copy_scale_rows_pair(uint32_t dst, const CUtensorMap* map, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar) : "memory");
}
// `bar` may be the other CTA's of the pair
__device__ __forceinline__ void copy_tile_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// rows of 128 bytes with a 128-byte swizzle, 8 rows every 1024 bytes
__device__ __forceinline__ uint64_t codes_desc(uint32_t addr) {
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// 32 rows of 16 bytes, 8 rows every 128 bytes
__device__ __forceinline__ uint64_t scales_desc(uint32_t addr) {
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
}
// E2M1 operands by rows, rows x cols sums, E8M0 (MX) or E4M3 scales; `id`: which
// two of the four scales (E8M0)
template <bool MX>
__device__ __forceinline__ uint32_t product_shape(int rows, int cols, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | (uint32_t(cols >> 3) << 17) | (MX ? 1u << 23 : 0u) |
           (uint32_t(rows >> 7) << 27) | (id << 29);
}
template <bool MX, bool PAIR>
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, uint32_t sa, uint32_t sb,
                                         bool add) {
#define DPG_MMA(group, kind)                                                                       \
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n tcgen05.mma.cta_group::" group      \
                 ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n}"                             \
                 :: "r"(d), "l"(a), "l"(b), "r"(shape), "r"(sa), "r"(sb), "r"(add ? 1u : 0u) : "memory")
    if (MX) {
        if (PAIR) DPG_MMA("2", "mxf4.block_scale.scale_vec::2X");
        else DPG_MMA("1", "mxf4.block_scale.scale_vec::2X");
    } else {
        if (PAIR) DPG_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
        else DPG_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    }
#undef DPG_MMA
}
// 512 bytes of scales to four columns of tensor memory
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t smem) {
    if (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(smem) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(smem) : "memory");
}
// arrives at `bar` once everything issued so far is done (PAIR: in both CTAs)
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     :: "r"(smem_u32(bar)), "h"(uint16_t(3)) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     :: "r"(smem_u32(bar)) : "memory");
}

// One stage's products: `steps` of 64 elements, scales first.  `at`: the stage
// (codes of the rows, of the columns, scales of the rows, of the columns), COLS:
// columns of the instruction, CODES: bytes of the columns' codes in this CTA.
template <bool MX, bool PAIR, int COLS, int CODES, int STEPS>
__device__ __forceinline__ void multiply_steps(uint32_t at, uint32_t d, uint32_t sf, bool fresh) {
    constexpr int kColTiles = COLS > 128 ? 2 : 1, kTiles = MX ? (STEPS + 1) / 2 : STEPS;
    constexpr int kSr = kRowTile * kCodeRow + CODES, kSc = kSr + kScaleBytes;
    const uint32_t tr = sf, tc = sf + 16;            // columns: 4 a tile of the rows, 4 or 8 of the columns
    const uint64_t scales = scales_desc(at), a = codes_desc(at);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        copy_scales<PAIR>(tr + 4 * t, scales + (kSr + t * kFp4TileBytes) / 16);
#pragma unroll
        for (int q = 0; q < kColTiles; ++q)
            copy_scales<PAIR>(tc + 4 * (kColTiles * t + q), scales + (kSc + (q * (MX ? 2 : 4) + t) * kFp4TileBytes) / 16);
    }
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const int t = MX ? k >> 1 : k;
        multiply<MX, PAIR>(d, a + 2 * k, a + kRowTile * kCodeRow / 16 + 2 * k,
                           product_shape<MX>(PAIR ? 256 : 128, COLS, MX ? 2u * uint32_t(k & 1) : 0u), tr + 4 * t,
                           tc + 4 * kColTiles * t, !fresh || k > 0);
    }
}
template <bool MX, bool PAIR, int COLS, int CODES>
__device__ __forceinline__ void multiply_stage(uint32_t at, uint32_t d, uint32_t sf, int steps, bool fresh) {
    if (steps >= 4) multiply_steps<MX, PAIR, COLS, CODES, 4>(at, d, sf, fresh);
    else if (steps == 3) multiply_steps<MX, PAIR, COLS, CODES, 3>(at, d, sf, fresh);
    else if (steps == 2) multiply_steps<MX, PAIR, COLS, CODES, 2>(at, d, sf, fresh);
    else multiply_steps<MX, PAIR, COLS, CODES, 1>(at, d, sf, fresh);
}

// ---------------------------------------------------------------------------
// results
// ---------------------------------------------------------------------------
// the operands' powers of two, as two factors (their product may leave fp32's range)
struct ProductScale {
    float f[2];
};
template <bool MX>
__device__ __forceinline__ ProductScale product_scale(const ProductArgs& a) {
    ProductScale s;
    s.f[0] = s.f[1] = 1.0f;
    if (!MX) {
        const int e = fp4_exponent(__float_as_uint(__ldg(a.amax_a))) + fp4_exponent(__float_as_uint(__ldg(a.amax_b)));
        const int h = e >> 1;      // -126 .. 117
        s.f[0] = __uint_as_float(uint32_t(127 + h) << 23);
        s.f[1] = __uint_as_float(uint32_t(127 + e - h) << 23);
    }
    return s;
}

// Four neighbouring results at `at` (elements of C), `n` of them inside C.
__device__ __forceinline__ float4 held_four(const ProductArgs& a, int64_t at, int n) {
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* p = static_cast<const float*>(a.c) + at;
    if (a.vec && n >= 4) return *reinterpret_cast<const float4*>(p);
    if (n > 0) o.x = p[0];
    if (n > 1) o.y = p[1];
    if (n > 2) o.z = p[2];
    if (n > 3) o.w = p[3];
    return o;
}
__device__ __forceinline__ void store_four(const ProductArgs& a, int64_t at, int n, float4 y) {
    if (a.c_f32) {
        float* p = static_cast<float*>(a.c) + at;
        if (a.vec && n >= 4) {
            *reinterpret_cast<float4*>(p) = y;
        } else {
            if (n > 0) p[0] = y.x;
            if (n > 1) p[1] = y.y;
            if (n > 2) p[2] = y.z;
            if (n > 3) p[3] = y.w;
        }
        return;
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.c) + at;
    if (a.vec && n >= 4) {
        *reinterpret_cast<uint2*>(p) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
        if (n > 0) p[0] = lo.x;
        if (n > 1) p[1] = lo.y;
        if (n > 2) p[2] = hi.x;
        if (n > 3) p[3] = hi.y;
    }
}

// Sums leave tensor memory a row to a lane; stored so, each access of a warp is
// 32 lines of memory (4 us for a tile of 128 x 256 where its products take 4 at
// k = 4096).  They go through shared memory, rows of COLS values in 16-byte
// pieces whose order within the row goes by the row, so that both a column of
// pieces and a row of them lie in different banks.
template <int COLS>
__device__ __forceinline__ int piece_at(int row, int piece) {
    constexpr int kMask = COLS >= 32 ? 7 : 3;
    return row * COLS + ((piece ^ ((COLS >= 32 ? row : row >> 1) & kMask)) << 2);
}

// A warp's 32 x 32 results (lane: row) by bulk copies: boxes of 32 rows x 64
// bytes with a 64-byte swizzle, in two halves of the warp's 4 KB in turn.  (One box
// of 128 bytes at a time: 4096 x 2304 x 768 9.3 us instead of 7.3.)
__device__ __forceinline__ void store_boxes(const ProductArgs& a, const CUtensorMap* map, uint32_t smem, int lane, int r,
                                            int c, const float* v, uint32_t& boxes) {
    const int n = a.c_f32 ? 2 : 1, width = a.c_f32 ? 16 : 32;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h >= n || c + h * width >= a.n) break;
        const uint32_t at = smem + (boxes++ & 1) * (kStoreBytes / 2), row = at + uint32_t(lane) * 64;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");   // what it held is on its way
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t to = row + (uint32_t(j) ^ (uint32_t(lane) >> 1 & 3u)) * 16;
            const uint4 w = a.c_f32 ? make_uint4(__float_as_uint(v[16 * h + 4 * j]), __float_as_uint(v[16 * h + 4 * j + 1]),
                                                 __float_as_uint(v[16 * h + 4 * j + 2]), __float_as_uint(v[16 * h + 4 * j + 3]))
                                    : narrow8(v + 8 * j);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(to), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            if (a.add)
                asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];"
                             :: "l"(map), "r"(c + h * width), "r"(r), "r"(at) : "memory");
            else
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                             :: "l"(map), "r"(c + h * width), "r"(r), "r"(at) : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
}
// 32 x 32 results singly, four columns of four rows to a lane group, any alignment
__device__ __forceinline__ void store_singly(const ProductArgs& a, float* box, int lane, int r, int c, const float* v) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(box + piece_at<32>(lane, j >> 2)) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    __syncwarp();
    const int row0 = lane >> 3, piece = lane & 7, n = a.n - c - 4 * piece, rows = a.m - r - row0;
    const int64_t at = int64_t(r + row0) * a.stride + c + 4 * piece, step = 4 * a.stride;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {           // four rows' old values at a time
        float4 o[4];
        if (a.add) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (16 * half + 4 * i < rows) o[i] = held_four(a, at + (4 * half + i) * step, n);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (16 * half + 4 * i < rows) {
                float4 y = *reinterpret_cast<const float4*>(box + piece_at<32>(16 * half + i * 4 + row0, piece));
                if (a.add) y.x += o[i].x, y.y += o[i].y, y.z += o[i].z, y.w += o[i].w;
                store_four(a, at + (4 * half + i) * step, n, y);
            }
    }
}

// A lane's 32 results to its own row, 32 bytes at a time.  That each access is 32
// lines of memory costs less than the way through shared memory, which operands and
// products fill (8192 x 14336 x 4096 151 us, by boxes 155; 4096 x 8192 x 2048 29.2 and
// 30.9; stores of 16 bytes were slower than boxes).
__device__ __forceinline__ void store_wide(const ProductArgs& a, int lane, int r, int c, const float* v) {
    if (r + lane >= a.m) return;
    const int64_t at = int64_t(r + lane) * a.stride + c;
    if (a.c_f32) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            F8 f;
#pragma unroll
            for (int i = 0; i < 8; ++i) f.v[i] = v[j + i];
            if (c + j < a.n) st_f8(static_cast<float*>(a.c) + at + j, f);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
            const uint4 x = narrow8(v + j), y = narrow8(v + j + 8);
            const F8 f = {{__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w),
                           __uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w)}};
            if (c + j < a.n) st_f8(reinterpret_cast<float*>(static_cast<__nv_bfloat16*>(a.c) + at + j), f);
        }
    }
}

// 32 columns of a warp's 32 rows from row r, column c on, scaled, into C
__device__ __forceinline__ void store_columns(const ProductArgs& a, const CUtensorMap* map, const ProductScale& scale, float* box,
                                              int lane, int r, int c, float* v, uint32_t& boxes) {
    if (r >= a.m || c >= a.n) return;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = v[j] * scale.f[0] * scale.f[1];
    if (a.wide) store_wide(a, lane, r, c, v);
    else if (a.boxes) store_boxes(a, map, smem_u32(box), lane, r, c, v, boxes);
    else store_singly(a, box, lane, r, c, v);
}

// ---------------------------------------------------------------------------
// Small products: 128 x COLS sums to a CTA.  Where there are few tiles, the CTAs
// of a cluster share the sum, leave their parts in shared memory and add them in
// the order of their ranks, each a share of the rows (or, where C's rows run along
// the tile's columns, of the columns).
//
// Two CTAs fit an SM and hold at most 256 of its 512 columns of tensor memory
// each; beside the CTAs of the large product and of the orthogonalisation
// no other fits.  So no CTA of a cluster ever waits for tensor memory that a CTA
// which waits for another cluster's holds.
//
//   warp 0  copies operands     warp 1  issues the products     warps 2..5  store
// ---------------------------------------------------------------------------
constexpr int kSmallThreads = 192;
template <int COLS>
struct SmallShape {
    static constexpr int kCodes = COLS * kCodeRow;
    static constexpr int kStage = kRowTile * kCodeRow + kCodes + 2 * kScaleBytes;
    static constexpr int kStages = COLS <= 32 ? 4 : COLS == 64 ? 4 : 3;
    static constexpr int kScaleColumn = COLS < 32 ? 32 : COLS;             // of tensor memory
    static constexpr int kColumns = kScaleColumn + 64 <= 128 ? 128 : 256;
    static constexpr int kSmem = kStages * kStage + 256;
    static_assert(kStage % 1024 == 0, "the swizzle's boundary");
    static_assert(kSmem > 77 * 1024 && 2 * (kSmem + 1024) <= 228 * 1024, "two CTAs to an SM, not three");
    static_assert(COLS * kRowTile * 4 <= kStages * kStage, "room for the sums");
};
struct SmallShared {
    uint64_t full[4], empty[4], done;
    uint32_t tmem;
    volatile int abort;
};

// The cluster's parts of a tile added up, this CTA's share of its rows: a thread
// keeps to four columns.  What C holds and the parts of kBatch rows are on their way
// at a time.
template <int COLS, int SPLIT>
__device__ __forceinline__ void join_rows(const ProductArgs& a, const ProductScale& scale, uint32_t part, int rank, int r0, int c0) {
    constexpr int kPer = COLS / 4, kStep = kSmallThreads / kPer, kBatch = SPLIT == 8 ? 2 : 4;
    constexpr int kShare = kRowTile / SPLIT;
    const int piece = int(threadIdx.x) % kPer, row0 = int(threadIdx.x) / kPer;
    const int n = a.n - c0 - 4 * piece, rows = min(kShare, a.m - r0 - rank * kShare);
    uint32_t from[SPLIT];
#pragma unroll
    for (int q = 0; q < SPLIT; ++q) from[q] = map_to(part, uint32_t(q));
    for (int i = row0; i < rows; i += kBatch * kStep) {
        const int64_t at = int64_t(r0 + rank * kShare + i) * a.stride + c0 + 4 * piece;
        float4 o[kBatch], y[kBatch][SPLIT];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i + u * kStep >= rows) continue;
            if (a.add) o[u] = held_four(a, at + u * kStep * a.stride, n);
            const uint32_t off = uint32_t(piece_at<COLS>(rank * kShare + i + u * kStep, piece)) * 4;
#pragma unroll
            for (int q = 0; q < SPLIT; ++q)
                asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(y[u][q].x), "=f"(y[u][q].y), "=f"(y[u][q].z), "=f"(y[u][q].w)
                             : "r"(from[q] + off) : "memory");
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i + u * kStep >= rows) continue;
            float4 x = y[u][0];
#pragma unroll
            for (int q = 1; q < SPLIT; ++q) x.x += y[u][q].x, x.y += y[u][q].y, x.z += y[u][q].z, x.w += y[u][q].w;
            x = make_float4(x.x * scale.f[0] * scale.f[1], x.y * scale.f[0] * scale.f[1], x.z * scale.f[0] * scale.f[1],
                            x.w * scale.f[0] * scale.f[1]);
            if (a.add) x.x += o[u].x, x.y += o[u].y, x.z += o[u].z, x.w += o[u].w;
            store_four(a, at + u * kStep * a.stride, n, x);
        }
    }
}
// The same where C's rows run along the tile's columns: this CTA's share of those,
// a thread to a row of the tile.
template <int COLS, int SPLIT>
__device__ __forceinline__ void join_columns(const ProductArgs& a, const ProductScale& scale, uint32_t part, int rank, int r0,
                                             int c0) {
    constexpr int kShare = COLS / SPLIT, kBatch = kShare < 4 ? kShare : 4;
    const int row = int(threadIdx.x), c = c0 + rank * kShare;
    if (row >= kRowTile || r0 + row >= a.n) return;
    uint32_t from[SPLIT];
#pragma unroll
    for (int q = 0; q < SPLIT; ++q) from[q] = map_to(part, uint32_t(q)) + uint32_t(rank * kShare * kRowTile + row) * 4;
#pragma unroll 1
    for (int j = 0; j < kShare && c + j < a.m; j += kBatch) {
        float x[kBatch], y[kBatch][SPLIT];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t at = int64_t(c + j + u) * a.stride + r0 + row;
            x[u] = a.add && c + j + u < a.m ? static_cast<const float*>(a.c)[at] : 0.0f;
#pragma unroll
            for (int q = 0; q < SPLIT; ++q)
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y[u][q]) : "r"(from[q] + uint32_t(j + u) * kRowTile * 4) : "memory");
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (c + j + u >= a.m) continue;
            const int64_t at = int64_t(c + j + u) * a.stride + r0 + row;
            float t = y[u][0];
#pragma unroll
            for (int q = 1; q < SPLIT; ++q) t += y[u][q];
            t = x[u] + t * scale.f[0] * scale.f[1];
            if (a.c_f32) static_cast<float*>(a.c)[at] = t;
            else static_cast<__nv_bfloat16*>(a.c)[at] = __float2bfloat16_rn(t);
        }
    }
}
template <int COLS, int SPLIT>
__device__ __forceinline__ void join_parts(const ProductArgs& a, const ProductScale& scale, uint32_t part, int rank, int r0, int c0) {
    if constexpr (COLS < 128) {                             // (128: never swapped, see product)
        if (a.swap) return join_columns<COLS, SPLIT>(a, scale, part, rank, r0, c0);
    }
    join_rows<COLS, SPLIT>(a, scale, part, rank, r0, c0);
}

template <bool MX, int COLS>
__global__ void __launch_bounds__(kSmallThreads, 2) k_fp4_small(const __grid_constant__ ProductArgs a,
                                                             const __grid_constant__ ProductMaps maps) {
    using S = SmallShape<COLS>;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(1024) unsigned char dyn[];
    SmallShared& sh = *reinterpret_cast<SmallShared*>(dyn + kStages * S::kStage);
    const uint32_t stage0 = smem_u32(dyn);
    const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = int(threadIdx.x & 31);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        mbar_init(&sh.done, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&sh.tmem)), "n"(S::kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    pdl_enter();
    const uint32_t tmem = sh.tmem;
    const int rank = a.split > 1 ? int(cluster_rank()) : 0;
    const int tile = int(blockIdx.x) / a.split;
    const int r0 = tile % a.tiles_r * kRowTile, c0 = tile / a.tiles_r * COLS;
    // this CTA's stages of the sum
    const int all = (a.k + kProdDepth - 1) / kProdDepth;
    const int first = int(int64_t(all) * rank / a.split), last = int(int64_t(all) * (rank + 1) / a.split);

    if (warp == 0 && lane == 0) {
        int s = 0;
        uint32_t par = 1;
        for (int k = first; k < last; ++k) {
            if (!wait_phase(&sh.empty[s], par, &sh.abort, a.wait_ns)) break;
            const uint32_t at = stage0 + uint32_t(s) * S::kStage, bar = smem_u32(&sh.full[s]);
            mbar_expect(&sh.full[s], kRowTile * kCodeRow + S::kCodes + 2 * (MX ? 1024 : 2048));
            if (blockIdx.x != 0 || k - first != a.skip) copy_tile(at, &maps.codes_r, k * kCodeRow, r0, bar);
            copy_tile(at + kRowTile * kCodeRow, &maps.codes_c, k * kCodeRow, c0, bar);
            const uint32_t sf = at + kRowTile * kCodeRow + S::kCodes;
            copy_scale_rows(sf, &maps.scales_r, k * (MX ? 8 : 16), r0 / kFp4TileRows, bar);
            copy_scale_rows(sf + kScaleBytes, &maps.scales_c, k * (MX ? 8 : 16), c0 / kFp4TileRows, bar);
            if (++s == kStages) {
                s = 0;
                par ^= 1;
            }
        }
    } else if (warp == 1) {
        const bool mine = elect_one();
        int s = 0;
        uint32_t par = 0;
        bool ok = true;
        for (int k = first; k < last; ++k) {
            ok = wait_phase(&sh.full[s], par, &sh.abort, a.wait_ns);
            if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const int left = a.k - k * kProdDepth, steps = left >= kProdDepth ? 4 : (left + 63) >> 6;
            if (mine) {
                multiply_stage<MX, false, COLS, S::kCodes>(stage0 + uint32_t(s) * S::kStage, tmem,
                                                           tmem + S::kScaleColumn + 32 * (k & 1), steps, k == first);
                commit<false>(&sh.empty[s]);
            }
            __syncwarp();
            if (++s == kStages) {
                s = 0;
                par ^= 1;
            }
        }
        if (ok && mine) commit<false>(&sh.done);
    }
    __syncwarp();
    float* const part = reinterpret_cast<float*>(dyn);
    const ProductScale scale = product_scale<MX>(a);
    if (warp >= 2) {
        const int row0 = (warp & 3) * 32, row = row0 + lane;
        const bool ok = __all_sync(0xFFFFFFFFu, wait_phase(&sh.done, 0, &sh.abort, a.wait_ns));
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t sums = tmem + (uint32_t(row0) << 16);
        constexpr int kGroup = COLS < 32 ? COLS : 32;
        if (ok) {                                           // the stages are free: every product is done
            if (COLS == 128 && a.split == 1) {              // whole sums: each warp stores its rows
                float* box = part + row0 * (kStoreBytes / 128);
                uint32_t boxes = 0;
#pragma unroll 1
                for (int c = 0; c < COLS; c += 32) {
                    float v[32];
                    load_acc32(sums + c, v);
                    store_columns(a, &maps.result, scale, box, lane, r0 + row0, c0 + c, v, boxes);
                }
                if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            } else {
#pragma unroll 1
                for (int c = 0; c < COLS; c += 32) {
                    float v[32];
                    load_acc32(sums + c, v);                // (COLS = 16: with 16 unused columns)
                    if (COLS < 128 && a.swap) {
#pragma unroll
                        for (int j = 0; j < kGroup; ++j) part[(c + j) * kRowTile + row] = v[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < kGroup; j += 4)
                            *reinterpret_cast<float4*>(part + piece_at<COLS>(row, (c + j) >> 2)) =
                                make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    }
                }
            }
        }
    }
    if (sh.abort) {   // the copies this CTA has in flight land within this time
        const uint64_t until = global_ns() + 2000000ull;
        while (global_ns() < until) {}
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (a.split > 1) cluster_sync();
    if (!sh.abort) {
        const uint32_t at = smem_u32(part);
        if (a.split == 8) join_parts<COLS, 8>(a, scale, at, rank, r0, c0);
        else if (a.split == 4) join_parts<COLS, 4>(a, scale, at, rank, r0, c0);
        else if (a.split == 2) join_parts<COLS, 2>(a, scale, at, rank, r0, c0);
        else if (COLS < 128) join_parts<COLS, 1>(a, scale, at, rank, r0, c0);
    }
    if (a.split > 1) cluster_sync();                        // the others have read this CTA's part
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(S::kColumns) : "memory");
}

// ---------------------------------------------------------------------------
// Large products: 256 x 256 sums to a pair of CTAs on two SMs, pairs that stay
// and take tile after tile.  CTA r holds rows 128 r .. of both operands; the
// pair's products read both halves, and each CTA's tensor memory holds the scales
// of its own rows and of all columns.
//
// Tensor memory: sums of even tiles in columns 0 .. 255, of odd ones in 160 ..
// 415, two sets of a stage's scales behind them.  The next tile's products start
// when the 96 columns that both sums have are read, which is done first.
//
// 8192 x 14336 x 4096 takes 152 us (6.3 PFLOP/s, 0.55 of six times the measured bf16
// rate), 8192 x 8192 x 8192 152 to 160.  Products alone, without copies of codes, take
// 124, copies alone 121 (18 TB/s into the SMs, 57 bytes a clock each), all but the
// stores 125: a stage is filled again 0.9 to 1.25 us after it was taken, and five stages
// are 0.9 us of products (four: 168, three: 203).  Stages of half the depth, of which
// ten fit, with rows of 64 bytes: 250; operands prefetched to L2 six or twelve stages
// ahead: 175, 167.
//
//   warp 0  copies operands     warp 1  of CTA 0: issues the products
//   warps 2..9  store (warp w: lanes 32 (w mod 4) .., every other 32 columns)
// ---------------------------------------------------------------------------
constexpr int kLargeStages = 5;
constexpr int kLargeCodes = kRowTile * kCodeRow;
constexpr int kLargeStage = 2 * kLargeCodes + 3 * kScaleBytes;
constexpr int kLargeEpiWarps = 8;
constexpr int kLargeThreads = 32 * (2 + kLargeEpiWarps);
constexpr int kLargeTile = 256;
constexpr int kOverlap = 96;
struct LargeShared {
    uint64_t full[kLargeStages], empty[kLargeStages], done[2], clear;
    uint32_t tmem;
    volatile int abort;
};
constexpr int kLargeSmem = kLargeStages * kLargeStage + kLargeEpiWarps * kStoreBytes + int(sizeof(LargeShared));
static_assert(kLargeStage % 1024 == 0, "the swizzle's boundary");
static_assert(kLargeSmem <= 227 * 1024 && kLargeSmem + 78 * 1024 > 228 * 1024, "alone on its SM");

// tile t of the queue: 8 rows of tiles at a time, column after column, so that
// the tiles in work at one time share operands
__device__ __forceinline__ void large_tile(const ProductArgs& a, int t, int& r0, int& c0) {
    const int per = 8 * a.tiles_c, g = t / per, in = t - g * per;
    const int high = min(8, a.tiles_r - 8 * g);
    r0 = (8 * g + in % high) * kLargeTile;
    c0 = in / high * kLargeTile;
}

template <bool MX>
__global__ void __cluster_dims__(2) __launch_bounds__(kLargeThreads, 1)
k_fp4_large(const __grid_constant__ ProductArgs a, const __grid_constant__ ProductMaps maps) {
    extern __shared__ __align__(1024) unsigned char dyn[];
    LargeShared& sh =
        *reinterpret_cast<LargeShared*>(dyn + kLargeStages * kLargeStage + kLargeEpiWarps * kStoreBytes);
    const uint32_t stage0 = smem_u32(dyn);
    const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = int(threadIdx.x & 31);
    const uint32_t rank = cluster_rank();
    const int pair = int(blockIdx.x >> 1), pairs = int(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kLargeStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        mbar_init(&sh.done[0], 1);
        mbar_init(&sh.done[1], 1);
        mbar_init(&sh.clear, 2 * kLargeEpiWarps);
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
    const int tiles = a.tiles_r * a.tiles_c, stages = (a.k + kProdDepth - 1) / kProdDepth;

    if (warp == 0 && lane == 0) {
        const uint32_t full0 = map_to(smem_u32(&sh.full[0]), 0);
        constexpr int kScales = MX ? 1024 : 2048;
        int s = 0;
        int64_t skip = blockIdx.x == 0 ? a.skip : -1;
        uint32_t par = 1;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            int r0, c0;
            large_tile(a, t, r0, c0);
            for (int k = 0; k < stages; ++k) {
                if (!(ok = wait_phase(&sh.empty[s], par, &sh.abort, a.wait_ns))) break;
                const uint32_t at = stage0 + uint32_t(s) * kLargeStage, bar = full0 + uint32_t(s) * 8;
                if (rank == 0) mbar_expect(&sh.full[s], 2 * (2 * kLargeCodes + 3 * kScales));
                if (skip-- != 0) copy_tile_pair(at, &maps.codes_r, k * kCodeRow, r0 + int(rank) * kRowTile, bar);
                copy_tile_pair(at + kLargeCodes, &maps.codes_c, k * kCodeRow, c0 + int(rank) * kRowTile, bar);
                const uint32_t sf = at + 2 * kLargeCodes;
                copy_scale_rows_pair(sf, &maps.scales_r, k * (MX ? 8 : 16), r0 / kFp4TileRows + int(rank), bar);
                copy_scale_rows_pair(sf + kScaleBytes, &maps.scales_c, k * (MX ? 8 : 16), c0 / kFp4TileRows, bar);
                if (++s == kLargeStages) {
                    s = 0;
                    par ^= 1;
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        const bool mine = elect_one();
        int s = 0, it = 0;
        uint32_t par = 0, set = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs, ++it) {
            if (it > 0) ok = wait_phase(&sh.clear, uint32_t(it - 1) & 1u, &sh.abort, a.wait_ns);
            if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + uint32_t(it & 1) * (kLargeTile - kOverlap);
            for (int k = 0; k < stages; ++k, set ^= 1) {
                ok = wait_phase(&sh.full[s], par, &sh.abort, a.wait_ns);
                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const int left = a.k - k * kProdDepth, steps = left >= kProdDepth ? 4 : (left + 63) >> 6;
                if (mine) {
                    multiply_stage<MX, true, kLargeTile, kLargeCodes>(stage0 + uint32_t(s) * kLargeStage, d,
                                                                      tmem + 2 * kLargeTile - kOverlap + 48 * set,
                                                                      steps, k == 0);
                    commit<true>(&sh.empty[s]);
                }
                __syncwarp();
                if (++s == kLargeStages) {
                    s = 0;
                    par ^= 1;
                }
            }
            if (ok && mine) commit<true>(&sh.done[it & 1]);
        }
    } else if (warp >= 2) {
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const ProductScale scale = product_scale<MX>(a);
        const uint32_t clear = map_to(smem_u32(&sh.clear), 0);
        float* const box = reinterpret_cast<float*>(dyn + kLargeStages * kLargeStage + (warp - 2) * kStoreBytes);
        uint32_t boxes = 0;
        int it = 0;
        for (int t = pair; t < tiles; t += pairs, ++it) {
            int r0, c0;
            large_tile(a, t, r0, c0);
            const int r = r0 + int(rank) * kRowTile + quad * 32;
            const bool ok = wait_phase(&sh.done[it & 1], uint32_t(it >> 1) & 1u, &sh.abort, a.wait_ns);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t sums = tmem + uint32_t(it & 1) * (kLargeTile - kOverlap) + (uint32_t(quad * 32) << 16);
            // in groups of 32 columns: the three that the next tile's sums take first
            const int before = (it & 1) ? 0 : kLargeTile - kOverlap;
#pragma unroll 1
            for (int g = half; g < kLargeTile / 32; g += 2) {
                const int c = (before + g * 32) & (kLargeTile - 1);
                float v[32];
                load_acc32(sums + uint32_t(c), v);
                if (g + 2 >= kOverlap / 32 && g < kOverlap / 32) {    // this warp's last of the three
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(clear) : "memory");
                }
                store_columns(a, &maps.result, scale, box, lane, r, c0 + c, v, boxes);   // (r: the warp's first row)
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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

// k = 0: zeros, or what C held
__global__ void __launch_bounds__(256) k_fp4_zero(const __grid_constant__ ProductArgs a) {
    pdl_enter();
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= int64_t(a.m) * a.n) return;
    const int64_t at = i / a.n * a.stride + i % a.n;
    if (a.c_f32) static_cast<float*>(a.c)[at] = 0.0f;
    else static_cast<uint16_t*>(a.c)[at] = 0;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static int encoder(EncodeTiled* out, const char* who) {
    static std::atomic<EncodeTiled> known{nullptr};
    EncodeTiled fn = known.load(std::memory_order_acquire);
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        DPG_CUDA_TRY(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found));
        if (found != cudaDriverEntryPointSuccess || !p)
            return fail(DPG_ERR_CUDA, "%s: the driver has no tensor maps", who);
        fn = reinterpret_cast<EncodeTiled>(p);
        known.store(fn, std::memory_order_release);
    }
    *out = fn;
    return DPG_OK;
}

// codes: boxes of 256 elements x box_rows; scales: boxes of a stage's tiles x
// box_tiles rows of tiles.  What lies outside is zero.
static int encode_operand(const dpg_fp4* q, int box_rows, int box_tiles, CUtensorMap* codes, CUtensorMap* scales,
                          const char* who) {
    EncodeTiled fn = nullptr;
    const int st = encoder(&fn, who);
    if (st != DPG_OK) return st;
    const cuuint32_t step[2] = {1, 1};
    const cuuint64_t dims[2] = {cuuint64_t(q->cols + 1) / 2, cuuint64_t(q->rows)};
    const cuuint64_t pitch[1] = {cuuint64_t(fp4_pitch(q->cols))};
    const cuuint32_t box[2] = {kCodeRow, cuuint32_t(box_rows)};
    CUresult e = fn(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q->codes, dims, pitch, box, step,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (e == CUDA_SUCCESS) {
        // as 128-byte rows, four to a tile
        const int64_t tiles = fp4_tiles(q->cols, q->format);
        const cuuint64_t sdims[3] = {128, cuuint64_t(tiles) * 4, cuuint64_t((q->rows + kFp4TileRows - 1) / kFp4TileRows)};
        const cuuint64_t spitch[2] = {128, cuuint64_t(tiles) * kFp4TileBytes};
        const cuuint32_t sbox[3] = {128, q->format == DPG_MXFP4 ? 8u : 16u, cuuint32_t(box_tiles)}, sstep[3] = {1, 1, 1};
        e = fn(scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, q->scales, sdims, spitch, sbox, sstep,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    return e == CUDA_SUCCESS ? DPG_OK : fail(DPG_ERR_CUDA, "%s: tensor map error %d", who, int(e));
}

// C in boxes of 32 rows x 64 bytes, if its rows start and end on 16-byte boundaries
static int encode_result(const ProductArgs& a, CUtensorMap* map, const char* who) {
    if (!a.boxes || a.wide) return DPG_OK;
    EncodeTiled fn = nullptr;
    const int st = encoder(&fn, who);
    if (st != DPG_OK) return st;
    const int size = a.c_f32 ? 4 : 2;
    const cuuint64_t dims[2] = {cuuint64_t(a.n), cuuint64_t(a.m)};
    const cuuint64_t pitch[1] = {cuuint64_t(a.stride) * size};
    const cuuint32_t box[2] = {cuuint32_t(64 / size), 32}, step[2] = {1, 1};
    const CUresult e = fn(map, a.c_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.c, dims,
                          pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return e == CUDA_SUCCESS ? DPG_OK : fail(DPG_ERR_CUDA, "%s: tensor map error %d", who, int(e));
}

template <bool MX, int COLS>
static int launch_small(ProductArgs a, const dpg_fp4* r, const dpg_fp4* c, int sms, cudaStream_t s, const char* who) {
    using S = SmallShape<COLS>;
    a.tiles_r = (a.rows + kRowTile - 1) / kRowTile;
    a.tiles_c = (a.cols + COLS - 1) / COLS;
    const int64_t tiles = int64_t(a.tiles_r) * a.tiles_c;
    const int stages = (a.k + kProdDepth - 1) / kProdDepth;
    // CTAs share a sum where it is long enough for the exchange (two or more 128 columns wide cost 1
    // to 2 us, a stage 0.2) and there is an SM for each, for clusters of eight two.  us with 1, 2, 4, 8:
    // 512 x 2048 x 2048 4.9, 7.0, 8.6, 16.9; 1024 x 1024 x 8192 10.7, 10.2, 11.5, 19.8; 384 x 1024 x 16384
    // 17.9, 13.3, 9.9, 12.1; 200 x 200 x 16384 18.4, 13.0, 9.3, 7.4; 64 x 4096 x 4096 8.8, 7.4, 5.9, 6.9;
    // 8 x 14336 x 4096 6.7, 6.9, 9.9, 16.3.  Rows of C that start anywhere are written by all threads
    // only then: 1111 x 777 x 512, added, 11.5 and 7.5.
    const int least = COLS < 128 ? 8 : a.boxes ? 16 : 2;
    a.split = stages < least ? 1 : tiles * 8 <= sms / 2 && stages >= 16 ? 8 : tiles * 4 <= sms && stages >= 8 ? 4 : tiles * 2 <= sms ? 2 : 1;
    if (tiles * a.split > 0x7FFFFFFF) return fail(DPG_ERR_INVALID_ARG, "%s: %lld tiles", who, (long long)tiles);
    ProductMaps maps;
    int st = encode_operand(r, kRowTile, 1, &maps.codes_r, &maps.scales_r, who);
    if (st == DPG_OK) st = encode_operand(c, COLS, 1, &maps.codes_c, &maps.scales_c, who);
    if (st == DPG_OK && COLS == 128 && a.split == 1) st = encode_result(a, &maps.result, who);
    if (st != DPG_OK) return st;
    auto k = k_fp4_small<MX, COLS>;
    static std::atomic<uint64_t> once{0};
    st = allow_smem(reinterpret_cast<const void*>(k), S::kSmem, once, who);
    if (st != DPG_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(tiles * a.split));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (a.split > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = unsigned(a.split);
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (t_programmatic) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = unsigned(n);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, a, maps);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return fail(DPG_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    }
    return after_launch(who);
}

template <bool MX>
static int launch_large(ProductArgs a, const dpg_fp4* r, const dpg_fp4* c, int sms, cudaStream_t s, const char* who) {
    a.tiles_r = (a.rows + kLargeTile - 1) / kLargeTile;
    a.tiles_c = (a.cols + kLargeTile - 1) / kLargeTile;
    a.split = 1;
    const int64_t tiles = int64_t(a.tiles_r) * a.tiles_c;
    if (tiles > 0x3FFFFFFF) return fail(DPG_ERR_INVALID_ARG, "%s: %lld tiles", who, (long long)tiles);
    ProductMaps maps;
    int st = encode_operand(r, kRowTile, 1, &maps.codes_r, &maps.scales_r, who);
    if (st == DPG_OK) st = encode_operand(c, kRowTile, 2, &maps.codes_c, &maps.scales_c, who);
    if (st != DPG_OK) return st;
    st = encode_result(a, &maps.result, who);
    if (st != DPG_OK) return st;
    const int pairs = int(tiles < sms / 2 ? tiles : sms / 2);
    static std::atomic<uint64_t> once{0};
    st = allow_smem(reinterpret_cast<const void*>(k_fp4_large<MX>), kLargeSmem, once, who);
    if (st != DPG_OK) return st;
    return launch_k(k_fp4_large<MX>, unsigned(2 * pairs), kLargeThreads, size_t(kLargeSmem), s, who, a, maps);
}

template <bool MX>
static int product(const dpg_fp4* x, const dpg_fp4* w, ProductArgs a, cudaStream_t s, const char* who) {
    int dev = 0, sms = 0;
    DPG_CUDA_TRY(cudaGetDevice(&dev));
    int st = sm_count(dev, &sms);
    if (st != DPG_OK) return st;
    const int64_t large = (int64_t(a.m) + kLargeTile - 1) / kLargeTile * ((int64_t(a.n) + kLargeTile - 1) / kLargeTile);
    a.rows = a.m;
    a.cols = a.n;
    const int few = a.m < a.n ? a.m : a.n;
    // Pairs where there is a tile of 256 x 256 for each, for longer sums for half of them (us with pairs
    // and without: 2560 x 2560 x 1024, 100 tiles, 7.4 and 9.3; 1536 x 2048 x 8192, 48, 14.1 and 16.9; 2048
    // x 2048 x 512, 64, 5.0 and 4.6; 1536 x 1536 x 4096, 36, 8.8 and 7.3).  A side of 128 or less would
    // leave half of each such tile empty.
    if (few > kRowTile && (large >= sms / 2 || (large >= sms / 4 && a.k > 2048))) return launch_large<MX>(a, x, w, sms, s, who);
    if (few > 64) return launch_small<MX, 128>(a, x, w, sms, s, who);
    // The shorter side in the columns of the sums, of which there may be 16, 32 or 64: 16 x 4096 x 4096
    // 4.6 us, 64 rows 5.9, 128 rows, in tiles of 128 x 128, 7.1.
    a.swap = a.m < a.n;
    if (a.swap) {
        a.rows = a.n;
        a.cols = a.m;
    }
    const dpg_fp4 *r = a.swap ? w : x, *c = a.swap ? x : w;
    if (few <= 16) return launch_small<MX, 16>(a, r, c, sms, s, who);
    if (few <= 32) return launch_small<MX, 32>(a, r, c, sms, s, who);
    return launch_small<MX, 64>(a, r, c, sms, s, who);
}

}  // namespace dpg

using dpg::fail;

extern "C" {

int dpg_fp4_product(const dpg_fp4* x, const dpg_fp4* w, void* c, int32_t c_dtype, int64_t row_stride,
                    int32_t accumulate, void* stream) {
    dpg::clear_error();
    const char* who = "dpg_fp4_product";
    const dpg::Trace trace(who);
    if (!x) return fail(DPG_ERR_INVALID_ARG, "%s: a is NULL", who);
    if (!w) return fail(DPG_ERR_INVALID_ARG, "%s: b is NULL", who);
    int st = dpg::fp4_check(x, "a", who);
    if (st == DPG_OK) st = dpg::fp4_check(w, "b", who);
    if (st != DPG_OK) return st;
    if (x->format != w->format) return fail(DPG_ERR_INVALID_ARG, "%s: a and b have different formats", who);
    if (x->cols != w->cols)
        return fail(DPG_ERR_INVALID_ARG, "%s: sums over %lld and %lld elements", who, (long long)x->cols,
                    (long long)w->cols);
    if (c_dtype != DPG_BF16 && c_dtype != DPG_F32)
        return fail(DPG_ERR_INVALID_ARG, "%s: dtype %d of c unknown", who, c_dtype);
    if (accumulate && c_dtype != DPG_F32) return fail(DPG_ERR_INVALID_ARG, "%s: only an fp32 c is added to", who);
    dpg::ProductArgs a{};
    if (x->rows == 0 || w->rows == 0) return DPG_OK;
    if (!c) return fail(DPG_ERR_INVALID_ARG, "%s: c is NULL", who);
    if (!dpg::aligned(c, c_dtype == DPG_BF16 ? 2 : 4)) return fail(DPG_ERR_MISALIGNED, "%s: c misaligned", who);
    if (x->rows > 1 && (row_stride < w->rows || row_stride > (int64_t(1) << 40)))
        return fail(DPG_ERR_INVALID_ARG, "%s: row stride %lld of c, which has %lld columns", who, (long long)row_stride,
                    (long long)w->rows);
    a.c = c;
    a.stride = x->rows > 1 ? row_stride : w->rows;
    a.amax_a = x->amax;
    a.amax_b = w->amax;
    a.m = int32_t(x->rows);
    a.n = int32_t(w->rows);
    a.k = int32_t(x->cols);
    a.c_f32 = c_dtype == DPG_F32;
    a.add = accumulate != 0;
    a.vec = dpg::aligned(c, 16) && (x->rows <= 1 || row_stride % (a.c_f32 ? 4 : 8) == 0);
    a.boxes = a.vec && w->rows % (a.c_f32 ? 4 : 8) == 0;
    const int piece = a.c_f32 ? 8 : 16;
    a.wide = !a.add && dpg::aligned(c, 32) && w->rows % piece == 0 && (x->rows <= 1 || row_stride % piece == 0);
    a.wait_ns = dpg::t_staged_timeout_ns > 0 ? uint64_t(dpg::t_staged_timeout_ns) : dpg::kProdWaitNs;
    a.skip = dpg::t_staged_skip;
    dpg::t_staged_skip = -1;
    dpg::t_staged_timeout_ns = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.k == 0) {
        if (a.add) return DPG_OK;
        int grid = 0;
        st = dpg::grid_cover((int64_t(a.m) * a.n + 255) / 256, &grid, who);
        return st != DPG_OK ? st : dpg::launch_k(dpg::k_fp4_zero, unsigned(grid), 256, s, who, a);
    }
    return x->format == DPG_MXFP4 ? dpg::product<true>(x, w, a, s, who) : dpg::product<false>(x, w, a, s, who);
}

int dpg_fp4_status(void* stream) {
    dpg::clear_error();
    const char* who = "dpg_fp4_status";
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int dev = 0;
    unsigned long long id = 0;       // of the stream: handles are used again, and one stands for each thread's own
    void* word = nullptr;
    uint32_t now = 0;
    DPG_CUDA_TRY(cudaGetDevice(&dev));
    DPG_CUDA_TRY(cudaStreamGetId(s, &id));
    DPG_CUDA_TRY(cudaGetSymbolAddress(&word, dpg::g_fp4_failures));
    DPG_CUDA_TRY(cudaMemcpyAsync(&now, word, sizeof now, cudaMemcpyDeviceToHost, s));
    DPG_CUDA_TRY(cudaStreamSynchronize(s));
    if (now == 0) return DPG_OK;     // (nothing is kept for streams until a wait has run out)
    try {
        // what each stream was told of last
        static std::mutex mu;
        static std::map<std::pair<int, unsigned long long>, uint32_t> told;
        std::lock_guard<std::mutex> g(mu);
        uint32_t& before = told[{dev, id}];
        if (before == now) return DPG_OK;
        before = now;
    } catch (const std::exception&) {
        // no room to remember it: the stream is told again the next time
    }
    return fail(DPG_ERR_DEVICE_TIMEOUT, "%s: a wait of a product on the device ran out; its results are incomplete", who);
}

}  // extern "C"
