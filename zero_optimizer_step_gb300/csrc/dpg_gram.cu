// dpg_gram.cu -- orthogonalisation of matrices whose shorter side is at most
// kGramSide, or kSmallSide where choose_paths sends them here (see
// dpg_orthogonalize in include/dpg.h).
//
// Every Newton-Schulz step multiplies X from the left by a polynomial of its
// Gram matrix, Q_k = aI + bA_k + cA_k^2 with A_k = X_k X_k^T, and all of these
// are polynomials of A_0: they commute, and
//     A_{k+1} = Q_k A_k Q_k,     X_n = (Q_{n-1} ... Q_1 Q_0) X_0.
// So the steps run on m x m matrices alone, between one pass over U that sums
// its Gram matrix (which also gives the norm: its trace) and one that
// multiplies U by the product P of the Q_k: 3 m^2 n flops and a few m^3 per
// step instead of 3 m^2 n per step, and three launches' latency instead of
// three dependent tile products per step.
//
// Everything is binary32.  An error e in A_k moves the small eigenvalues l by
// e / l relative, so the 11-bit operands of the large matrices' tensor-core
// products would lose the directions that the steps are there to bring up;
// with 24 bits the result of five default steps is within 1e-6 (Gaussian) to
// 7e-4 (rank one) of the exact one.  A step multiplies e by up to a^2, and what
// e made negative is never brought back: twelve steps on one A_0 ended in NaN
// for low ranks.  Longer schedules are therefore cut into phases (gram_phases):
// P is applied to the copy of X, and the Gram matrix is summed anew, which is
// as good as the iteration on X itself.
//
// Times (128 x 6000, five steps): sum 18 us, steps 67 us, application 12 us;
// the steps alone 12, 17, 30, 62 us at 16, 32, 64, 128 rows.  A step of 128
// rows takes 12 us: four products of 16 x 128 x 128 per CTA of about 2 us
// (half the fp32 rate; two warps per scheduler feed it from shared memory) and
// two exchanges of rows of about 1.2 us (64 KB out of and into every CTA).
// Long matrices (4 of 128 x 50000) are bound by the fp32 rate of the two
// passes over the columns: 222 and 147 us, 30 and 45 TFLOP/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dpg_host.h"
#include "dpg_ortho.h"

namespace dpg {

struct GramArgs {
    const SmallDesc* mats;
    const void* update;
    uint16_t* out;           // flat bf16
    float* copy;             // U, or X after a phase, 32 columns at a time: [block][padded rows][32]
    float* part;             // per Gram item: partial sum, [padded rows]^2
    int32_t* part_exp;       // per Gram item: its values are U 2^-exp
    float* prod;             // per matrix: the product of the Q_k, [padded rows]^2
    int32_t* exp;            // per matrix: prod is for U 2^-exp
    int32_t* status;         // 0, or the error of the first wait that ran out
    uint64_t wait_ns;        // bound of every wait
    int32_t leave_out;       // test only: 0: the first CTA does not send its first values (-1: none)
    double eps;
    int32_t first;           // the copy holds U, to be divided by its norm; else X as it is
    int32_t n_steps;         // of this phase
    float a[DPG_MAX_NS_STEPS], b[DPG_MAX_NS_STEPS], c[DPG_MAX_NS_STEPS];
};

constexpr int kGramThreads = 256;

// 2^k for any k that occurs here, exactly
__device__ __forceinline__ float pow2(int k) {
    return k < -126 ? 0.0f : __int_as_float((k > 127 ? 127 : k) + 127 << 23);
}

// ---------------------------------------------------------------------------
// Partial Gram matrices.  One CTA sums the outer products of up to `width`
// columns, 32 at a time through shared memory; each thread holds a T x T block
// of the sum (T = padded rows / 16).  U's range may exceed what fp32 squares
// can hold, so columns are scaled by the power of two of the largest value so
// far, and the sum with them when that grows.
// ---------------------------------------------------------------------------
enum : int { kFromBf16 = 0, kFromF32 = 1, kFromCopy = 2 };   // what is summed

template <int MP, int FROM>
__device__ __forceinline__ void gram_item(const GramArgs& a, const SmallDesc& d, const SmallItem& it, float* sm) {
    constexpr int T = MP / 16, P = MP + 4, kPer = MP * 32 / kGramThreads;
    float* tile = sm;                    // [32][P]
    float* red = sm + 32 * P;            // 8 + 1
    const int tx = int(threadIdx.x) & 15, ty = int(threadIdx.x) >> 4;
    // a thread's columns: four neighbours in each 64, so that the lanes' reads
    // are contiguous
    auto col = [&](int j) { return T >= 4 ? (j >> 2) * 64 + tx * 4 + (j & 3) : tx * T + j; };
    constexpr int kTwo = (T + 1) / 2;    // a thread's columns in pairs (at 16: one and a zero)
    uint64_t acc[T][kTwo];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < kTwo; ++j) acc[i][j] = 0;
    int e = -1000;
    float x[kPer];
    const bool tall = FROM != kFromCopy && d.tall;   // (the copy holds X's rows)
    // all loads before any use (a load under its own branch would be waited
    // for there, one memory latency per value): out of range ones read U's
    // first element
    auto fetch = [&](int c0) {
        if (FROM == kFromCopy) {           // whole blocks, zeros past the matrix
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                x[i] = __ldg(a.copy + d.copy + int64_t(c0 >> 5) * (MP * 32) + int(threadIdx.x) + i * kGramThreads);
            return;
        }
        uint32_t raw[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int q = int(threadIdx.x) + i * kGramThreads;
            const int r = tall ? q % MP : q >> 5, c = c0 + (tall ? q / MP : q & 31);
            const int64_t at = d.off + (r < d.m && c < d.n
                                            ? (tall ? int64_t(c) * d.m + r : int64_t(r) * d.n + c) : 0);
            raw[i] = FROM == kFromF32 ? __ldg(static_cast<const uint32_t*>(a.update) + at)
                                      : uint32_t(__ldg(static_cast<const uint16_t*>(a.update) + at)) << 16;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int q = int(threadIdx.x) + i * kGramThreads;
            const int r = tall ? q % MP : q >> 5, c = c0 + (tall ? q / MP : q & 31);
            x[i] = r < d.m && c < d.n ? __uint_as_float(raw[i]) : 0.0f;
        }
    };
    fetch(it.c0);
    for (int c0 = it.c0; c0 < it.c1; c0 += 32) {
        float top = 0.0f;
        float* copy = a.copy + d.copy + int64_t(c0 >> 5) * (MP * 32);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int q = int(threadIdx.x) + i * kGramThreads;
            const int r = tall ? q % MP : q >> 5, c = tall ? q / MP : q & 31;
            if (FROM != kFromCopy) copy[r * 32 + c] = x[i];
            top = fmaxf(top, fabsf(x[i]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
        __syncthreads();                 // also: the tile before is used up
#pragma unroll
        for (int w = 0; w < 8; ++w) top = fmaxf(top, red[w]);
        // |u| < 2^(te + 1); an infinity keeps its own scale and poisons the sum
        const int te = top > 0.0f && top < 3.0e38f ? ilogbf(top) : (top > 0.0f ? 127 : -1000);
        if (te > e) {
            const float k = pow2(2 * (e - te));
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int j = 0; j < kTwo; ++j) acc[i][j] = mul2(acc[i][j], pair_of(k, k));
            e = te;
        }
        // 2^-e in two factors: either may leave fp32's range alone
        const float s0 = e > -1000 ? pow2(-(e >> 1)) : 0.0f, s1 = e > -1000 ? pow2(-(e - (e >> 1))) : 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int q = int(threadIdx.x) + i * kGramThreads;
            const int r = tall ? q % MP : q >> 5, c = tall ? q / MP : q & 31;
            tile[c * P + r] = x[i] * s0 * s1;
        }
        __syncthreads();
        if (c0 + 32 < it.c1) fetch(c0 + 32);
#pragma unroll 4
        for (int k = 0; k < 32; ++k) {
            float u[T], v[2 * kTwo] = {};
#pragma unroll
            for (int i = 0; i < T; ++i) {
                u[i] = tile[k * P + ty * T + i];
                v[i] = tile[k * P + col(i)];
            }
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int j = 0; j < kTwo; ++j)
                    acc[i][j] = fma2(pair_of(u[i], u[i]), pair_of(v[2 * j], v[2 * j + 1]), acc[i][j]);
        }
    }
    float* out = a.part + it.part;
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j)
            out[(ty * T + i) * MP + col(j)] = j % 2 ? halves_of(acc[i][j / 2]).y : halves_of(acc[i][j / 2]).x;
    if (threadIdx.x == 0) a.part_exp[it.index] = e;
}

template <int FROM>
__global__ void __launch_bounds__(kGramThreads) k_gram_sum(const __grid_constant__ GramArgs a,
                                                          const SmallItem* items) {
    __shared__ __align__(16) float sm[32 * (kSmallSide + 4) + 16];
    pdl_enter();
    const SmallItem it = items[blockIdx.x];
    const SmallDesc d = a.mats[it.mat];
    switch (d.mp) {
        case 16: return gram_item<16, FROM>(a, d, it, sm);
        case 32: return gram_item<32, FROM>(a, d, it, sm);
        case 64: return gram_item<64, FROM>(a, d, it, sm);
        default: return gram_item<128, FROM>(a, d, it, sm);
    }
}

// ---------------------------------------------------------------------------
// The steps on the Gram matrix.  A cluster of MP / 16 CTAs per matrix; each
// holds A and Q whole and owns 16 rows of every product, which it writes into
// the other CTAs' copies (distributed shared memory).  Per step
//     Q = aI + bA + cA^2,   P <- P Q,   A <- (A Q) Q
// with two exchanges, Q's rows and A's.  The writes count their bytes at a
// barrier in the CTA that they go to; a CTA that has all MP^2 values goes on,
// and knows with them that every CTA is through with what it overwrites next:
// a CTA sends rows of Q only after its products with A, rows of A only after
// its products with Q (a product ends with a CTA barrier).  A cluster barrier
// per exchange instead took 23.3 us against 22.1 for 64 x 32 and 32 x 10, 70
// against 66 for 1000 of 16 x 64, and as long at 64 and 128 rows, where the
// bytes are the exchange.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void gram_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// After a wait that ran out: what others sent without being waited for lands
// within this time.  (Not inlined: the code would be fetched in every call.)
__device__ __noinline__ void linger() {
    uint64_t since, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(since));
    do asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
    while (now - since < 2000000ull);
}

// 16 rows times MP x MP.  The CTA's threads split K into R parts; within one, a
// thread holds R rows by MP / 16 columns (four rows where there are columns
// enough: half the shared-memory reads per multiply-add of two).  The parts
// then exchange their sums, and each thread keeps one row: row() and col(j).
template <int MP>
struct RowProduct {
    static constexpr int kCols = MP / 16, R = MP >= 64 ? 4 : 2;
    static constexpr int kGroup = kGramThreads / R;              // threads of a part
    static constexpr int kExchange = R * R * kCols * kGroup;     // floats of shared memory
    float v[kCols];
    __device__ __forceinline__ static int tx() { return int(threadIdx.x) & 15; }
    __device__ __forceinline__ static int ty() { return int(threadIdx.x) % kGroup >> 4; }
    __device__ __forceinline__ static int part() { return int(threadIdx.x) / kGroup; }
    __device__ __forceinline__ static int row() { return R * ty() + part(); }
    __device__ __forceinline__ static int col(int j) {
        return kCols >= 4 ? (j >> 2) * 64 + tx() * 4 + (j & 3) : tx() * kCols + j;
    }
    __device__ __forceinline__ void run(const float* left, const float* right, float* exchange) {
        constexpr int kTwo = (kCols + 1) / 2;                    // columns in pairs (at 16: one and a zero)
        uint64_t two[R][kTwo];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < kTwo; ++j) two[i][j] = 0;
        left += R * ty() * MP;
#pragma unroll 2
        for (int k = part() * (MP / R); k < (part() + 1) * (MP / R); k += 4) {
            float l[R][4];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(left + i * MP + k);
                l[i][0] = q.x;
                l[i][1] = q.y;
                l[i][2] = q.z;
                l[i][3] = q.w;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint64_t r[kTwo];
                const float* from = right + (k + u) * MP;
                if constexpr (kCols >= 4) {
#pragma unroll
                    for (int g = 0; g < kCols / 4; ++g) {
                        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(from + g * 64 + tx() * 4);
                        r[2 * g] = q.x;
                        r[2 * g + 1] = q.y;
                    }
                } else if constexpr (kCols == 2) {
                    r[0] = *reinterpret_cast<const uint64_t*>(from + tx() * 2);
                } else {
                    r[0] = pair_of(from[tx()], 0.0f);
                }
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const uint64_t l2 = pair_of(l[i][u], l[i][u]);
#pragma unroll
                    for (int j = 0; j < kTwo; ++j) two[i][j] = fma2(l2, r[j], two[i][j]);
                }
            }
        }
        float s[R][kCols];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < kCols; ++j) s[i][j] = j % 2 ? halves_of(two[i][j / 2]).y : halves_of(two[i][j / 2]).x;
        float* e = exchange + int(threadIdx.x) % kGroup;         // [part][row][column][thread]
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i != part())
#pragma unroll
                for (int j = 0; j < kCols; ++j) e[((part() * R + i) * kCols + j) * kGroup] = s[i][j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            float t = 0.0f;
#pragma unroll
            for (int p = 0; p < R; ++p) t += p == part() ? s[p][j] : e[((p * R + part()) * kCols + j) * kGroup];
            v[j] = t;
        }
    }
};

template <int W>
struct Width {
    static constexpr int value = W;
};

template <int MP>
__device__ void gram_steps(const GramArgs& a, int mat, int rank, float* sm) {
    constexpr int C = MP / 16;           // CTAs of the cluster that hold rows
    if (rank >= C) {                     // the others only meet the barriers
        gram_cluster_sync();
        gram_cluster_sync();
        return;
    }
    float* A = sm;                       // [MP][MP]
    float* Q = A + MP * MP;              // [MP][MP]
    float* P = Q + MP * MP;              // [16][MP], own rows
    float* S = P + 16 * MP;              // [16][MP], own rows: A Q
    float* exchange = S + 16 * MP;
    __shared__ double den_sh;
    __shared__ float scale_sh;
    __shared__ uint64_t all_of[2];       // A's rows, Q's rows
    const SmallDesc d = a.mats[mat];
    const int t = int(threadIdx.x), row0 = rank * 16;

    // writes W neighbouring values to the own rows (row, col ..) of `dst` in
    // every CTA of the cluster: 16 bytes at a time where there are as many (one
    // value at a time, the writes took longer than the products)
    bool ok = true;                      // after a wait ran out: waits no more, the result is worthless
    auto spread = [&](float* dst, uint64_t* bar, int row, int col, const float* v, auto width) {
        constexpr int W = decltype(width)::value;
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(dst + (row0 + row) * MP + col));
        const uint32_t bar_at = static_cast<uint32_t>(__cvta_generic_to_shared(bar));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t to, bar_to;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(c));
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar_to) : "r"(bar_at), "r"(c));
            if constexpr (W == 4)
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1,%2,%3,%4}, [%5];"
                             :: "r"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(bar_to) : "memory");
            else if constexpr (W == 2)
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1,%2}, [%3];"
                             :: "r"(to), "f"(v[0]), "f"(v[1]), "r"(bar_to) : "memory");
            else
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];"
                             :: "r"(to), "f"(v[0]), "r"(bar_to) : "memory");
        }
    };
    // expects one exchange (thread 0, before any wait for it, after the last one ended), and
    // waits for the n-th
    auto expect_all = [&](uint64_t* bar) {
        if (t == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                         :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(bar))), "r"(MP * MP * 4) : "memory");
    };
    auto wait_all = [&](uint64_t* bar, int n) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(bar));
        uint64_t since = 0;
        for (uint32_t polls = 0; ok; ++polls) {
            uint32_t done;
            asm volatile("{\n .reg .pred p;\n"
                         " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                         " selp.u32 %0, 1, 0, p;\n}"
                         : "=r"(done) : "r"(at), "r"(uint32_t(n & 1)) : "memory");
            if (done) return;
            if ((polls & 255) == 0) {
                uint64_t now;
                asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
                if (polls == 0) since = now;
                if (now - since > a.wait_ns) {
                    ok = false;
                    atomicCAS(a.status, 0, DPG_ERR_DEVICE_TIMEOUT);
                }
            }
        }
    };
    if (t == 0) {
        for (int k = 0; k < 2; ++k)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;"
                         :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(all_of + k))) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    expect_all(all_of);

    // the partial sums under one scale, own rows
    int e = -1000;
    for (int k = 0; k < d.n_items; ++k) e = max(e, __ldg(a.part_exp + d.item0 + k));
    gram_cluster_sync();                 // every CTA has started: its memory may be written
    const int leave_out = blockIdx.x == 0 ? a.leave_out : -1;
    for (int q = t; q < 4 * MP; q += kGramThreads) {
        const float4* p = reinterpret_cast<const float4*>(a.part + d.part + row0 * MP) + q;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < d.n_items; k += 16) {
            float4 v[16];
            int pe[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int it = min(k + u, d.n_items - 1);
                v[u] = __ldg(p + int64_t(it) * (MP * MP / 4));
                pe[u] = __ldg(a.part_exp + d.item0 + it);
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const float w = k + u < d.n_items ? pow2(2 * (pe[u] - e)) : 0.0f;
                if (k + u < d.n_items) {
                    s[0] = fmaf(v[u].x, w, s[0]);
                    s[1] = fmaf(v[u].y, w, s[1]);
                    s[2] = fmaf(v[u].z, w, s[2]);
                    s[3] = fmaf(v[u].w, w, s[3]);
                }
            }
        }
        if (q != leave_out)
            spread(A, all_of, q / (MP / 4), (q % (MP / 4)) * 4, s, Width<4>());
    }
    wait_all(all_of, 0);
    if (t < 32) {                        // trace: the squared norm of U 2^-e
        double s = 0.0;
        for (int r = t; r < MP; r += 32) s += double(A[r * MP + r]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (t == 0) {
            // divisor of U 2^-e: max(norm, eps) 2^-e; of X 2^-e: 2^-e (a.eps is 1)
            double den = sqrt(a.first ? s : 0.0);
            if (e > -1000) den = fmax(den, scalbn(a.eps, -e));
            const bool ok = s < 3.0e38;  // a NaN or an infinity in the matrix: NaN everywhere
            if (!(den > 0.0)) den = 1.0; // a zero matrix stays zero
            den_sh = ok ? den : __longlong_as_double(0x7FF8000000000000ll);
            scale_sh = float(1.0 / (den_sh * den_sh));
        }
    }
    __syncthreads();

    // step 0 takes A as scale * (the sum in memory)
    float scale = scale_sh;
    RowProduct<MP> y;
    constexpr int kCols = RowProduct<MP>::kCols, W = kCols < 4 ? kCols : 4;
    const int row = y.row();
    for (int step = 0; step < a.n_steps; ++step) {
        expect_all(all_of + 1);
        y.run(A + row0 * MP, A, exchange);
        const float ca = a.a[step], cb = a.b[step] * scale, cc = a.c[step] * scale * scale;
#pragma unroll
        for (int g = 0; g < kCols; g += W) {
            const int col = y.col(g);
            float q[W];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                q[j] = fmaf(cc, y.v[g + j], cb * A[(row0 + row) * MP + col + j]);
                if (col + j == row0 + row) q[j] += ca;
            }
            spread(Q, all_of + 1, row, col, q, Width<W>());
        }
        wait_all(all_of + 1, step);
        const bool last = step + 1 == a.n_steps;
        if (step == 0) {
            for (int q = t; q < 16 * MP; q += kGramThreads) P[q] = Q[row0 * MP + q];
        } else {
            y.run(P, Q, exchange);       // (its barrier: every thread has read P)
#pragma unroll
            for (int j = 0; j < kCols; ++j) P[row * MP + y.col(j)] = y.v[j];
        }
        if (last) break;
        // the exchange is free again; and a CTA that waited in vain ends here: it expects nothing
        // on top of what never came, and sends at most the rows of one more exchange, whose bytes
        // a barrier can count unexpected
        if (__syncthreads_or(!ok)) break;
        expect_all(all_of);
        y.run(A + row0 * MP, Q, exchange);
#pragma unroll
        for (int j = 0; j < kCols; ++j) S[row * MP + y.col(j)] = y.v[j] * scale;
        __syncthreads();
        y.run(S, Q, exchange);
#pragma unroll
        for (int g = 0; g < kCols; g += W) spread(A, all_of, row, y.col(g), &y.v[g], Width<W>());
        scale = 1.0f;
        wait_all(all_of, step + 1);
    }
    __syncthreads();
    const float inv = float(1.0 / den_sh);
    for (int q = t; q < 16 * MP; q += kGramThreads) a.prod[d.prod + row0 * MP + q] = P[q] * inv;
    if (rank == 0 && t == 0) a.exp[mat] = e;
    if (!ok) linger();
    __syncwarp();
    gram_cluster_sync();                 // no CTA leaves while others write to it
}

// All matrices of one padded side, in clusters of its size.
template <int MP>
__global__ void __launch_bounds__(kGramThreads) k_gram_steps(const __grid_constant__ GramArgs a,
                                                            const int32_t* which) {
    extern __shared__ __align__(16) float gram_sm[];
    pdl_enter();
    gram_steps<MP>(a, which[blockIdx.x / (MP / 16)], int(blockIdx.x) % (MP / 16), gram_sm);
}

// Matrices of any padded sides, in clusters of eight.
__global__ void __launch_bounds__(kGramThreads) k_gram_steps_mixed(const __grid_constant__ GramArgs a) {
    extern __shared__ __align__(16) float gram_sm[];
    pdl_enter();
    const int mat = int(blockIdx.x) / 8, rank = int(blockIdx.x) % 8;
    switch (a.mats[mat].mp) {
        case 16: return gram_steps<16>(a, mat, rank, gram_sm);
        case 32: return gram_steps<32>(a, mat, rank, gram_sm);
        case 64: return gram_steps<64>(a, mat, rank, gram_sm);
        default: return gram_steps<128>(a, mat, rank, gram_sm);
    }
}

template <int MP>
constexpr int gram_steps_smem() {
    return (2 * MP * MP + 32 * MP + RowProduct<MP>::kExchange) * 4;
}
constexpr int kMixedMost = 15;   // clusters of eight that are resident at once

// ---------------------------------------------------------------------------
// O = P U, 64 columns per CTA: a thread holds MP / 16 rows by 4 columns.
// BACK: not the end, the new X goes back into the copy (a CTA has all of its
// columns in shared memory by then, and no other one reads them).
// ---------------------------------------------------------------------------
constexpr int kProdCols = 64;
constexpr int gram_apply_smem(int mp) { return (mp * (mp + 4) + mp * kProdCols) * 4; }

template <int MP, bool BACK>
__device__ __forceinline__ void apply_item(const GramArgs& a, const SmallDesc& d, const SmallItem& it, float* sm) {
    constexpr int T = MP / 16, PP = MP + 4;
    float* P = sm;                       // [MP][PP]
    float* X = sm + MP * PP;             // [MP][64]
    const int t = int(threadIdx.x), tx = t & 15, ty = t >> 4;
    const int e = a.exp[it.mat];
    const float s0 = e > -1000 ? pow2(-(e >> 1)) : 0.0f, s1 = e > -1000 ? pow2(-(e - (e >> 1))) : 0.0f;
    constexpr int kP = (MP * MP / 4 + kGramThreads - 1) / kGramThreads, kX = MP * kProdCols / 4 / kGramThreads;
    float4 p[kP], x[kX];
    // the copy holds whole blocks of 32 columns, and one more is never far: a
    // second block past the end is read from the first instead
#pragma unroll
    for (int i = 0; i < kX; ++i) {
        const int q = t + i * kGramThreads, blk = it.c0 + q / (MP * 8) * 32 < d.n ? q / (MP * 8) : 0;
        const float4* from =
            reinterpret_cast<const float4*>(a.copy + d.copy + int64_t((it.c0 >> 5) + blk) * (MP * 32)) + q % (MP * 8);
        x[i] = BACK ? *from : __ldg(from);
    }
#pragma unroll
    for (int i = 0; i < kP; ++i)
        p[i] = __ldg(reinterpret_cast<const float4*>(a.prod + d.prod) + min(t + i * kGramThreads, MP * MP / 4 - 1));
#pragma unroll
    for (int i = 0; i < kX; ++i) {
        const int q = t + i * kGramThreads, blk = q / (MP * 8), r = q / 8 % MP, c = q % 8 * 4;
        const float k = it.c0 + blk * 32 < d.n ? 1.0f : 0.0f;
        *reinterpret_cast<float4*>(X + r * kProdCols + blk * 32 + c) =
            make_float4(x[i].x * s0 * s1 * k, x[i].y * s0 * s1 * k, x[i].z * s0 * s1 * k, x[i].w * s0 * s1 * k);
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) {
        const int q = t + i * kGramThreads;
        if (q < MP * MP / 4) *reinterpret_cast<float4*>(P + (q / (MP / 4)) * PP + (q % (MP / 4)) * 4) = p[i];
    }
    __syncthreads();
    uint64_t acc[T][2];
#pragma unroll
    for (int i = 0; i < T; ++i) acc[i][0] = acc[i][1] = 0;
    const int kend = (d.m + 3) & ~3;
#pragma unroll 1
    for (int k = 0; k < kend; k += 4) {
        ulonglong2 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const ulonglong2*>(X + (k + u) * kProdCols + tx * 4);
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const float4 p4 = *reinterpret_cast<const float4*>(P + (ty * T + i) * PP + k);
            const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                acc[i][0] = fma2(pair_of(p[u], p[u]), x[u].x, acc[i][0]);
                acc[i][1] = fma2(pair_of(p[u], p[u]), x[u].y, acc[i][1]);
            }
        }
    }
    const bool vec = !d.tall && ((d.off | d.n) & 3) == 0;
#pragma unroll
    for (int i = 0; i < T; ++i) {
        const int r = ty * T + i, c = it.c0 + tx * 4;
        if (r >= d.m) continue;
        const float2 o01 = halves_of(acc[i][0]), o23 = halves_of(acc[i][1]);
        const float o[4] = {o01.x, o01.y, o23.x, o23.y};
        if (BACK) {
            if (c < d.n)                 // (a started block is whole in the copy)
                *reinterpret_cast<float4*>(a.copy + d.copy + int64_t(c >> 5) * (MP * 32) + r * 32 + (c & 31)) =
                    make_float4(o[0], c + 1 < d.n ? o[1] : 0.0f, c + 2 < d.n ? o[2] : 0.0f, c + 3 < d.n ? o[3] : 0.0f);
        } else if (vec && c < d.n) {
            const __nv_bfloat162 u = __floats2bfloat162_rn(o[0], o[1]);
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[2], o[3]);
            *reinterpret_cast<uint2*>(a.out + d.off + int64_t(r) * d.n + c) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < d.n)
                    a.out[d.off + (d.tall ? int64_t(c + j) * d.m + r : int64_t(r) * d.n + c + j)] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(o[j]));
        }
    }
}

template <bool BACK>
__global__ void __launch_bounds__(kGramThreads) k_gram_apply(const __grid_constant__ GramArgs a,
                                                            const SmallItem* items) {
    extern __shared__ __align__(16) float gram_sm[];
    pdl_enter();
    const SmallItem it = items[blockIdx.x];
    const SmallDesc d = a.mats[it.mat];
    switch (d.mp) {
        case 16: return apply_item<16, BACK>(a, d, it, gram_sm);
        case 32: return apply_item<32, BACK>(a, d, it, gram_sm);
        case 64: return apply_item<64, BACK>(a, d, it, gram_sm);
        default: return apply_item<128, BACK>(a, d, it, gram_sm);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int gram_prepare() {
    DPG_CUDA_TRY(cudaFuncSetAttribute(k_gram_steps<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      gram_steps_smem<64>()));
    DPG_CUDA_TRY(cudaFuncSetAttribute(k_gram_steps<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      gram_steps_smem<128>()));
    DPG_CUDA_TRY(cudaFuncSetAttribute(k_gram_steps_mixed, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      gram_steps_smem<128>()));
    DPG_CUDA_TRY(cudaFuncSetAttribute(k_gram_apply<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      gram_apply_smem(kSmallSide)));
    DPG_CUDA_TRY(cudaFuncSetAttribute(k_gram_apply<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      gram_apply_smem(kSmallSide)));
    return DPG_OK;
}

template <typename... P, typename... A>
static int launch_clusters(void (*k)(P...), int n, int ctas, int smem, cudaStream_t s, const char* who,
                           const A&... args) {
    if (n == 0) return DPG_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(n) * unsigned(ctas));
    cfg.blockDim = dim3(kGramThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = t_programmatic ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return fail(DPG_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    }
    return after_launch(who);
}

// arguments of steps [k0, k1) of hp
static GramArgs gram_args(const Matrices& m, const void* update, const dpg_muon_hparams* hp, int k0, int k1,
                          void* out) {
    GramArgs a{};
    a.wait_ns = kOrthoWaitNs;
    a.mats = m.d_small;
    a.update = update;
    a.out = static_cast<uint16_t*>(out);
    a.copy = reinterpret_cast<float*>(m.ws + m.o_small_copy);
    a.part = reinterpret_cast<float*>(m.ws + m.o_small_part);
    a.part_exp = reinterpret_cast<int32_t*>(m.ws + m.o_small_exp);
    a.exp = a.part_exp + m.gram_items.size();
    a.prod = reinterpret_cast<float*>(m.ws + m.o_small_prod);
    a.status = reinterpret_cast<int32_t*>(m.ws + m.o_status);
    a.eps = k0 == 0 ? hp->eps : 1.0;
    a.first = k0 == 0;
    a.n_steps = k1 - k0;
    for (int k = k0; k < k1; ++k) {
        a.a[k - k0] = float(hp->coeffs[k][0]);
        a.b[k - k0] = float(hp->coeffs[k][1]);
        a.c[k - k0] = float(hp->coeffs[k][2]);
    }
    return a;
}

int gram_read(const Matrices& m, const void* update, int32_t update_dtype, const dpg_muon_hparams* hp,
              void* out, cudaStream_t s, const char* who) {
    if (m.small.empty()) return DPG_OK;
    return launch_k(update_dtype == DPG_F32 ? k_gram_sum<kFromF32> : k_gram_sum<kFromBf16>,
                    unsigned(m.gram_items.size()), kGramThreads, s, who, gram_args(m, update, hp, 0, 0, out),
                    static_cast<const SmallItem*>(m.d_gram_items));
}

static int launch_gram_steps(const Matrices& m, const GramArgs& a, cudaStream_t s, const char* who) {
    const int32_t *w = m.d_small_order, *n = m.small_count;
    int st = DPG_OK;
    if ((n[0] > 0) + (n[1] > 0) + (n[2] > 0) + (n[3] > 0) > 1 && int(m.small.size()) <= kMixedMost) {
        // one launch side by side instead of one per padded side: sides of 16, 32, 64 and 128 took
        // 11, 15, 30 and 75 us one after the other.  With more matrices than clusters of eight fit,
        // the smaller sides would wait for places as large as the largest needs.
        const int smem = n[3] ? gram_steps_smem<128>() : n[2] ? gram_steps_smem<64>() : gram_steps_smem<32>();
        st = launch_clusters(k_gram_steps_mixed, int(m.small.size()), 8, smem, s, who, a);
    } else {
        st = launch_clusters(k_gram_steps<16>, n[0], 1, gram_steps_smem<16>(), s, who, a, w);
        if (st == DPG_OK)
            st = launch_clusters(k_gram_steps<32>, n[1], 2, gram_steps_smem<32>(), s, who, a, w + n[0]);
        if (st == DPG_OK)
            st = launch_clusters(k_gram_steps<64>, n[2], 4, gram_steps_smem<64>(), s, who, a, w + n[0] + n[1]);
        if (st == DPG_OK)
            st = launch_clusters(k_gram_steps<128>, n[3], 8, gram_steps_smem<128>(), s, who, a,
                                 w + n[0] + n[1] + n[2]);
    }
    return st;
}

int gram_finish(const Matrices& m, const void* update, const dpg_muon_hparams* hp, const OrthoSchedule& sch,
                const WaitFault& fault, void* out, cudaStream_t s, const char* who) {
    if (m.small.empty()) return DPG_OK;
    const int mp = m.small_count[3] ? 128 : m.small_count[2] ? 64 : m.small_count[1] ? 32 : 16;
    int st = DPG_OK;
    for (int p = 0; p < sch.n_phases && st == DPG_OK; ++p) {
        const bool last = p + 1 == sch.n_phases;
        GramArgs a = gram_args(m, update, hp, p ? sch.phase_end[p - 1] : 0, sch.phase_end[p], out);
        a.wait_ns = fault.wait_ns;
        a.leave_out = fault.skip >= 0 ? 0 : -1;
        st = launch_gram_steps(m, a, s, who);
        if (st == DPG_OK)
            st = launch_k(last ? k_gram_apply<false> : k_gram_apply<true>, unsigned(m.prod_items.size()), kGramThreads,
                          size_t(gram_apply_smem(mp)), s, who, a, static_cast<const SmallItem*>(m.d_prod_items));
        if (st == DPG_OK && !last)
            st = launch_k(k_gram_sum<kFromCopy>, unsigned(m.gram_items.size()), kGramThreads, s, who, a,
                          static_cast<const SmallItem*>(m.d_gram_items));
    }
    return st;
}

}  // namespace dpg
