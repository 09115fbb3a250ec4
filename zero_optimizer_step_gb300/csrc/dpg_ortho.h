// dpg_ortho.h -- the matrices of a plan and their Newton-Schulz workspace:
// declarations shared by the host tables (dpg_matrices.cpp), the
// orthogonalisation (dpg_ortho.cu) and the momentum / apply passes
// (dpg_muon.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <vector>

#include "dpg_internal.h"

namespace dpg {

// Workspace matrices are stored as blocks of 128 rows x 64 columns of fp16,
// 16 KB each: row r of a block is 128 bytes, whose eight 16-byte chunks are
// permuted by chunk ^ (r mod 8).  That is the shared-memory image the tensor
// cores read with a 128-byte swizzle, both as rows of K (a block of 128 rows,
// 64 deep) and as columns (64 columns, 128 -- or 64 -- deep), so a block
// moves between HBM and shared memory as one contiguous copy and the same
// stored X serves X X^T and B X.  Rows are padded to 256 and columns to 256
// with zeros: an output tile of 256 x 256 always exists.
constexpr int kBlkRows = 128;
constexpr int kBlkCols = 64;
constexpr int64_t kBlkBytes = int64_t(kBlkRows) * kBlkCols * 2;
constexpr int kOrthoTile = 256;

struct MatDesc {
    int64_t off;          // first element in the flat buffer
    int32_t rows, cols;   // as stored by the user
    int32_t m, n;         // shorter and longer side: X is m x n
    int32_t tall;         // rows > cols: X is the transpose of the stored matrix
    int32_t kn, km;       // 64-deep blocks of a sum over n, over m
    int32_t cbx, cba;     // 64-column blocks in a row of X, of A
    int64_t x[2], lo;     // first block of the two X buffers and of X's low part
    int64_t a, b;         // first block of A and of bA + cA^2 (off-diagonal parts)
    int64_t lo2, blo;     // first block of X's other low part, of B's low part: in the second
                          // workspace, or in the first if `both`
    int32_t both;         // all steps take both halves (see lay_out)
    int64_t diag;         // first entry of the per-row vectors (see OrthoArgs)
    int64_t rowsq;        // first entry of X's row sums of squares, [cbx][padded rows]
    int32_t rows_pad;     // rows of X padded to 256
    int32_t norm0, norm1; // its items in the norm table
    int32_t tiles[3];     // output tiles of each product (see lay_queue), each part counted
    int32_t group0;       // its first group of parts
    int32_t groups;       // A tiles that are summed in parts (0: none)
};

// One output tile of one product of one matrix: 256 rows from 256 i, 64 blocks
// columns from 64 blocks j.  A tile of A may be summed in parts: the pairs of
// the parts each take a share of the sum's length, leave one another their
// sums, and each finishes its share of the columns.
struct alignas(16) OrthoTile {
    int32_t mat;
    int32_t group;        // which tile in parts, of all
    int16_t i, j;
    uint8_t prod, blocks; // blocks: 4 or 2
    uint8_t part, split;  // split: log2 of the number of parts
};
static_assert(sizeof(OrthoTile) == 16, "one load");

// Matrices whose shorter side is at most kGramSide take the steps on their Gram
// matrices (dpg_gram.cu) and none of the tiles, those of up to kSmallSide where that
// is faster (see choose_paths).
constexpr int kGramSide = 64;
constexpr int kSmallSide = 128;
struct SmallDesc {
    int64_t off;          // first element in the flat buffer
    int32_t m, n, tall;   // as in MatDesc
    int32_t mp;           // m padded to 16, 32, 64 or 128
    int64_t copy, part, prod;   // first floats of its copy, partial Gram matrices, product
    int32_t item0, n_items;     // its Gram items
};
// columns [c0, c1) of a small matrix
struct SmallItem {
    int32_t mat, c0, c1, index;
    int64_t part;
};

// Items of the norm and conversion passes and of the weight update.
struct NormItem {
    int32_t mat, count;   // elements [start, start + count) of the matrix
    int64_t start;
};
struct ConvItem {
    int32_t mat, i, j, pad;   // blocks (i, 2 j) and (i, 2 j + 1) of X
};
struct ApplyItem {
    int64_t off;          // flat offset, a multiple of 8
    int32_t count;        // <= kApplyChunk elements of one parameter
    int32_t param;
};
constexpr int kNormChunk = 16384;
constexpr int kApplyChunk = 1024;

// Products of a step, in order: A = X X^T, B = bA + cA^2, X' = aX + BX.
enum : int { kProdA = 0, kProdB = 1, kProdX = 2 };

constexpr uint64_t kOrthoWaitNs = 2000000000ull;   // bound of every wait, unless a test sets another
// what a test does to one call
struct WaitFault {
    int64_t skip;         // >= 0: one copy or exchange is left out
    uint64_t wait_ns;
};

constexpr float kLoScale = 2048.0f;   // of X's low half

// Constants of one Newton-Schulz step.  Stored fp16 values are the true ones
// times a power of two that keeps the largest the step can produce below 2^15.
struct OrthoStep {
    float a, b, c;
    float inv_sx;      // 1 / scale of X (step 0: the matrix's own, on the device)
    float sx_next;     // scale of the new X
    float sa, inv_sa;  // scale of A
    float sb, inv_sb;  // scale of bA + cA^2
};

// The steps of a call, and where the Gram path sums its matrices anew.
struct OrthoSchedule {
    OrthoStep st[DPG_MAX_NS_STEPS];
    int32_t both_steps;                    // the first so many take both halves (see both_halves)
    int32_t n_phases;                      // of the Gram path (see gram_phases)
    int32_t phase_end[DPG_MAX_NS_STEPS];   // the step after each
};

struct Matrices {
    int64_t total_padded = 0;
    int32_t n_params = 0;
    std::vector<int64_t> param_offset, numels;
    std::vector<MatDesc> mats;
    std::vector<OrthoTile> queue;      // tiles of a step, pair after pair (see lay_queue)
    std::vector<int32_t> queue_first;  // pairs + 1
    int32_t pairs = 0;
    std::vector<SmallDesc> small;
    std::vector<SmallItem> gram_items, prod_items;
    std::vector<int32_t> small_order;  // small matrices by padded side
    int32_t small_count[4] = {0, 0, 0, 0};
    int32_t n_matrices = 0;
    std::vector<NormItem> norm_items;
    std::vector<ConvItem> conv_items;
    std::vector<ApplyItem> apply_items;
    std::vector<double> scales;        // 2 per parameter: spectral, rms
    bool any_both = false;             // one of mats is `both`
    int64_t n_low_blocks = 0;          // of the second workspace
    int64_t n_blocks = 0, n_diag = 0, n_rowsq = 0, n_groups = 0;
    int64_t n_small_copy = 0, n_small_part = 0, n_small_prod = 0;   // floats
    int64_t workspace_bytes = 0;
    // byte offsets in the workspace
    int64_t o_diag = 0, o_rowsq = 0, o_part = 0, o_scal = 0, o_count = 0, o_done = 0, o_join = 0, o_status = 0;
    int64_t o_small_copy = 0, o_small_part = 0, o_small_exp = 0, o_small_prod = 0;

    std::mutex mu;
    int device = -1;
    unsigned char* ws = nullptr;       // workspace_bytes
    unsigned char* ws_low = nullptr;   // n_low_blocks blocks, from the first call that needs them on
    unsigned char* d_tables = nullptr; // one allocation, sections below
    unsigned char* d_update_tables = nullptr;   // apply_items and scales
    MatDesc* d_mats = nullptr;
    OrthoTile* d_queue = nullptr;
    int32_t* d_queue_first = nullptr;
    SmallDesc* d_small = nullptr;
    SmallItem *d_gram_items = nullptr, *d_prod_items = nullptr;
    int32_t* d_small_order = nullptr;
    NormItem* d_norm_items = nullptr;
    ConvItem* d_conv_items = nullptr;
    ApplyItem* d_apply_items = nullptr;
    double* d_scales = nullptr;
    // tensor maps of the workspace (128 and 64 rows a copy) and of the second one
    alignas(64) unsigned char maps[4][128];
};

// fills queue, queue_first and pairs for a device that holds `clusters` CTA pairs
void lay_queue(Matrices& m, int clusters);
// device side (dpg_ortho.cu)
int upload_matrices(Matrices& m, bool both);   // both: steps that take both halves follow
int upload_for_update(Matrices& m);   // only what dpg_muon_apply needs
void release_matrices(Matrices& m);
int check_matrices(Matrices& m, void* stream);
// validates hp for the orthogonalisation and fills the schedule
int ortho_steps(const dpg_muon_hparams* hp, OrthoSchedule* sch, const char* who);
int ortho_launch(Matrices& m, const void* update, int32_t update_dtype, const dpg_muon_hparams* hp,
                 const OrthoSchedule& sch, void* out, void* stream, const char* who);

// The small matrices' part (dpg_gram.cu): gram_read is the only one that reads
// `update`, gram_finish the only one that writes `out`.
int gram_prepare();
int gram_read(const Matrices& m, const void* update, int32_t update_dtype, const dpg_muon_hparams* hp,
              void* out, cudaStream_t s, const char* who);
int gram_finish(const Matrices& m, const void* update, const dpg_muon_hparams* hp, const OrthoSchedule& sch,
                const WaitFault& fault, void* out, cudaStream_t s, const char* who);

}  // namespace dpg

struct dpg_matrices {
    dpg::Matrices m;
};
