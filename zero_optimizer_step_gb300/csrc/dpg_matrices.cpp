// dpg_matrices.cpp -- host tables of a plan's matrices (shapes, workspace
// layout, tiles, work items) and the constants of the Newton-Schulz steps.
#include <algorithm>
#include <cmath>
#include <exception>
#include <functional>
#include <new>
#include <queue>
#include <utility>

#include "dpg_ortho.h"

namespace dpg {

constexpr int64_t kMaxMatrices = 1 << 20;   // of one object

static int64_t ceil_div(int64_t x, int64_t d) { return (x + d - 1) / d; }
static int padded_side(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128; }

// Columns of a small matrix's Gram items: about 64 groups of whole 32-column
// blocks (every further group is a partial sum to write and to read again; very
// long matrices get one per 1024 columns, up to 128).
static int64_t gram_width(int64_t n) {
    const int64_t blocks = ceil_div(n, 32);
    const int64_t groups = std::min<int64_t>(blocks, std::max<int64_t>(64, std::min<int64_t>(128, n / 1024)));
    return ceil_div(blocks, groups) * 32;
}

// Items of a small matrix: Gram sums, products of 64 columns.
static void small_items(Matrices& M, const MatDesc& d) {
    SmallDesc s{};
    s.off = d.off;
    s.m = d.m;
    s.n = d.n;
    s.tall = d.tall;
    s.mp = padded_side(d.m);
    const int32_t mat = int32_t(M.small.size());
    const int64_t blocks = ceil_div(d.n, 32);
    s.copy = M.n_small_copy;
    M.n_small_copy += blocks * 32 * s.mp;
    s.prod = M.n_small_prod;
    M.n_small_prod += int64_t(s.mp) * s.mp;
    const int64_t width = gram_width(d.n);
    s.part = M.n_small_part;
    s.item0 = int32_t(M.gram_items.size());
    for (int64_t c = 0; c < d.n; c += width) {
        M.gram_items.push_back({mat, int32_t(c), int32_t(std::min<int64_t>(c + width, d.n)),
                                int32_t(M.gram_items.size()), M.n_small_part});
        M.n_small_part += int64_t(s.mp) * s.mp;
    }
    s.n_items = int32_t(M.gram_items.size()) - s.item0;
    for (int64_t c = 0; c < d.n; c += 64)
        M.prod_items.push_back({mat, int32_t(c), int32_t(std::min<int64_t>(c + 64, d.n)), 0, 0});
    M.small.push_back(s);
}

// How many parts an A tile's sum may have: the parts' sums (256 KB each) are
// left in the buffer of the next X, which is free while A is built.
static int most_parts(const MatDesc& d) {
    const int tm = d.cba / 4, tn = d.cbx / 4;
    return tn >= 4 * (tm + 1) ? 4 : tn >= 2 * (tm + 1) ? 2 : 1;
}

static int64_t up256(int64_t x) { return ceil_div(x, 256) * 256; }

// Which matrices of at most kSmallSide rows take the Gram path.  From 2 to 64 rows
// all do: the tiles, padded to 256, were 10 to 900 us slower, except for one to four
// short ones of 32 and 64 rows beside larger matrices, 10 to 25 us faster, and use
// up to eight times the memory.
//
// Those of 65 to 128 rows: where five default steps of all of them are estimated to
// take no longer so.  The Gram path is three launches of its own: its
// steps take 62 us for as many matrices as have their clusters resident, its two
// passes over the columns 2 ns per column, and nothing else runs beside it.  The
// tiles' fifteen products follow one another and take both halves of their operands
// (see lay_out), but as many tiles as there are pairs run at once, and beside larger
// matrices they mostly fill gaps.  Measured, Gram path and tiles (us):
//     1 of 128 x 128      74   127      beside 4 of 768 x 768 (146)   223   152
//     1 of 128 x 1000     79   181                                   227   213
//     16 of 128 x 1000   166   204                                   316   231
//     16 of 128 x 600    152   181                                   299   203
//     64 of 128 x 600    405   274                                   557   358
//     30 of 100 x 100    144   145                                   292   261
//     4 of 128 x 6000    121   268                                   270   280
// (In 48 such sets, alone and beside five lists, the rule picks the slower path
// twice, by 15 and 26 us of 700 and 2080.)  The numbers in the rule (76 pairs, 15
// clusters, times) are this GPU's; with long schedules both paths' times grow alike.
// Where the tiles would take more than 16 GB, the path of less memory is taken.
//
// Single rows have no off-diagonal parts that would need both halves.  A few beside
// matrices on the tiles stay there and save the Gram path's launches (1 x 777 beside
// four of 517 to 1031 rows: 175 against 185 us).
struct Paths {
    bool gram_rows;    // single rows take the Gram path
    bool gram_large;   // 65 to 128 rows do
    bool gram(int64_t m) const {
        return m == 1 ? gram_rows : m <= kGramSide || (m <= kSmallSide && gram_large);
    }
};
static Paths choose_paths(const Plan& p, const int64_t* rows, const int64_t* cols) {
    int64_t count = 0, columns = 0, longest = 0, blocks = 0, floats = 0;
    double tiles = 0, single = 0, single_sum = 0;
    bool larger = false;
    for (int32_t q = 0; q < p.n_params; ++q) {
        const int64_t m = std::min(rows[q], cols[q]), n = std::max(rows[q], cols[q]);
        const int64_t k = p.numels[q] / (rows[q] * cols[q]);
        if (k == 0) continue;
        larger = larger || m > kSmallSide;
        const double deep = double(ceil_div(n, kBlkCols)), wide = double(ceil_div(n, kOrthoTile));
        if (m == 1) {
            single += double(k) * 5.0 * (std::max(0.3 * deep, 3.0) + 3.0 + 3.0 * wide) / 76.0;
            single_sum = std::max(single_sum, 0.3 * deep);
        }
        if (m <= kGramSide || m > kSmallSide) continue;
        count += k;
        columns += k * n;
        longest = std::max(longest, n);
        blocks += k * 8 * (4 * ceil_div(n, kOrthoTile) + 3);   // as lay_out counts them
        floats += k * (ceil_div(n, 32) * 32 * kSmallSide +     // as small_items
                       (ceil_div(n, gram_width(n)) + 1) * kSmallSide * kSmallSide);
        // in units of a pair's time: three sums each, or the finish of a block in 1, 2 or 3 visits
        tiles += double(k) * 5.0 * (std::max(0.9 * deep, 5.0) + 9.0 + 6.0 * wide) / 76.0;
    }
    Paths out;
    if (blocks * kBlkBytes > (int64_t(16) << 30)) {
        out.gram_large = floats * int64_t(sizeof(float)) < blocks * kBlkBytes;
    } else {
        const double deep = double(ceil_div(longest, kBlkCols));
        out.gram_large = 62.0 * double(ceil_div(count, 15)) + 10.0 + 2e-3 * double(columns) <=
                         (larger ? 10.0 + deep : 120.0 + 2.0 * deep) + tiles;
    }
    const bool on_tiles = larger || (count > 0 && !out.gram_large);
    // (the Gram path's launches take about 13 us; a tile's sum may take as long as others' do)
    out.gram_rows = !on_tiles || single > 10.0 || single_sum > 10.0;
    return out;
}

// Lays the matrices out; false when an index would leave its type.
static bool lay_out(const Plan& p, const int64_t* rows, const int64_t* cols, Matrices& M) {
    M.total_padded = p.total_padded;
    M.n_params = p.n_params;
    M.param_offset = p.param_offset;
    M.numels = p.numels;
    M.scales.assign(2 * size_t(p.n_params), 1.0);
    int64_t count = 0;
    for (int32_t q = 0; q < p.n_params; ++q)
        if ((count += p.numels[q] / (rows[q] * cols[q])) > kMaxMatrices) return false;
    // Items of the norm pass: as long as leaves about four per SM (each costs a fence and an
    // atomic besides its loads)
    const Paths paths = choose_paths(p, rows, cols);
    int64_t tiled = 0;
    for (int32_t q = 0; q < p.n_params; ++q)
        if (!paths.gram(std::min(rows[q], cols[q]))) tiled += p.numels[q];
    const int64_t norm_chunk = kNormChunk * std::clamp<int64_t>(ceil_div(tiled, 608 * int64_t(kNormChunk)), 1, 8);
    for (int32_t q = p.n_params - 1; q >= 0; --q) {   // flat order
        const double r = double(rows[q]), c = double(cols[q]);
        M.scales[2 * size_t(q)] = std::sqrt(std::max(1.0, r / c));
        M.scales[2 * size_t(q) + 1] = 0.2 * std::sqrt(std::max(r, c));
        const int64_t numel = p.numels[q];
        for (int64_t e = 0; e < numel; e += kApplyChunk)
            M.apply_items.push_back({p.param_offset[q] + e,
                                     int32_t(std::min<int64_t>(kApplyChunk, numel - e)), q});
        const int64_t one = rows[q] * cols[q];
        for (int64_t e = 0; e < numel; e += one) {
            MatDesc d{};
            d.off = p.param_offset[q] + e;
            d.rows = int32_t(rows[q]);
            d.cols = int32_t(cols[q]);
            d.tall = rows[q] > cols[q];
            d.m = int32_t(std::min(rows[q], cols[q]));
            d.n = int32_t(std::max(rows[q], cols[q]));
            ++M.n_matrices;
            if (paths.gram(d.m)) {
                small_items(M, d);
                continue;
            }
            d.kn = int32_t(ceil_div(d.n, kBlkCols));
            d.km = int32_t(ceil_div(d.m, kBlkCols));
            const int64_t tm = ceil_div(d.m, kOrthoTile), tn = ceil_div(d.n, kOrthoTile);
            if (tm > 0x3FFF || tn > 0x3FFF) return false;
            const int64_t rb = tm * (kOrthoTile / kBlkRows);
            d.cbx = int32_t(tn * (kOrthoTile / kBlkCols));
            d.cba = int32_t(tm * (kOrthoTile / kBlkCols));
            const int64_t xb = rb * d.cbx, ab = rb * d.cba;
            d.x[0] = M.n_blocks;
            d.x[1] = d.x[0] + xb;
            d.lo = d.x[1] + xb;
            d.a = d.lo + xb;
            d.b = d.a + ab;
            M.n_blocks = d.b + ab;
            // Few rows average little of the rounding that fp16 off-diagonal parts
            // leave: five default steps on rank one end 5 % off at 2 to 4 rows, 1 % at
            // 16, 5e-3 at 32, and every row twice 4e-3 at 128.  Both halves in all
            // steps leave 1e-4; their blocks are few.
            d.both = d.m > 1 && d.m <= kSmallSide;
            M.any_both = M.any_both || d.both;
            int64_t& low = d.both ? M.n_blocks : M.n_low_blocks;
            d.lo2 = low;
            d.blo = d.lo2 + xb;
            low = d.blo + ab;              // (n_low_blocks stays below n_blocks)
            // a block's first 128-byte row is a 32-bit coordinate of the copies
            if (M.n_blocks * kBlkRows > 0x7FFFFFFFll) return false;
            d.diag = M.n_diag;
            d.rows_pad = int32_t(tm * kOrthoTile);
            M.n_diag += d.rows_pad;
            d.rowsq = M.n_rowsq;
            M.n_rowsq += int64_t(d.rows_pad) * d.cbx;
            if (tm * tn > 0x1FFFFFF) return false;   // counts of a call stay in 32 bits
            if (most_parts(d) > 1) {
                d.group0 = int32_t(M.n_groups);
                M.n_groups += tm * (tm + 1);         // A tiles of 128 columns
                if (M.n_groups > 0x3FFFFFF) return false;
            }
            const int32_t mat = int32_t(M.mats.size());
            d.norm0 = int32_t(M.norm_items.size());
            for (int64_t s = 0; s < one; s += norm_chunk)
                M.norm_items.push_back({mat, int32_t(std::min(norm_chunk, one - s)), s});
            d.norm1 = int32_t(M.norm_items.size());
            for (int64_t i = 0; i < rb; ++i)
                for (int64_t j = 0; j < d.cbx / 2; ++j)
                    M.conv_items.push_back({mat, int32_t(i), int32_t(j), 0});
            M.mats.push_back(d);
        }
    }
    int64_t o = M.n_blocks * kBlkBytes;
    M.o_diag = o;   // three vectors: diagonals of A, of B, and the part of B's that X's low half sees
    o += up256(3 * M.n_diag * int64_t(sizeof(float)));
    M.o_rowsq = o;
    o += up256(M.n_rowsq * int64_t(sizeof(float)));
    M.o_part = o;
    o += up256(int64_t(M.norm_items.size()) * int64_t(sizeof(double)));
    M.o_scal = o;   // per matrix: power-of-two scale of X, 1 / (norm times it)
    o += up256(int64_t(M.mats.size()) * 2 * int64_t(sizeof(float)));
    M.o_count = o;  // per matrix: arrivals of its norm items
    o += up256(int64_t(M.mats.size()) * int64_t(sizeof(int32_t)));
    M.o_done = o;   // per matrix and product: tiles finished in this call
    o += up256(int64_t(M.mats.size()) * 3 * int64_t(sizeof(int32_t)));
    M.o_join = o;   // per group of parts, CTA and warp: parts left in this call
    o += up256(M.n_groups * 16 * int64_t(sizeof(int32_t)));
    M.o_status = o;
    o += 256;
    for (int c = 0; c < 4; ++c)
        for (size_t k = 0; k < M.small.size(); ++k)
            if (M.small[k].mp == 16 << c) {
                M.small_order.push_back(int32_t(k));
                ++M.small_count[c];
            }
    M.o_small_copy = o;
    o += up256(M.n_small_copy * int64_t(sizeof(float)));
    M.o_small_part = o;
    o += up256(M.n_small_part * int64_t(sizeof(float)));
    M.o_small_prod = o;
    o += up256(M.n_small_prod * int64_t(sizeof(float)));
    M.o_small_exp = o;   // per Gram item, then per matrix
    o += up256(int64_t(M.gram_items.size() + M.small.size()) * int64_t(sizeof(int32_t)));
    M.workspace_bytes = o;
    return M.gram_items.size() < 0x7FFFFFFF && M.prod_items.size() < 0x7FFFFFFF &&
           M.small.size() < 0x7FFFFFF && M.norm_items.size() < 0x7FFFFFFF && M.conv_items.size() < 0x7FFFFFFF &&
           M.apply_items.size() < 0x7FFFFFFF;
}

// How the products of a step are cut: blocks of 64 columns in a tile of each,
// and the most parts of an A tile.
struct Cut {
    int blocks[3], parts;
};
// A deal of one step's tiles to the pairs.
struct Deal {
    std::vector<std::vector<OrthoTile>> mine;   // pair by pair
    int64_t end = 0;                            // modelled time of the step
};

static int parts_of(const MatDesc& d, const Cut& c) { return std::min(c.parts, most_parts(d)); }

// The tiles of one step -- A tiles, B tiles, X tiles of all matrices, larger
// matrices first -- dealt out to the pairs in this order, each to the pair that
// could start it first.  The parts of a tile wait for one another, so they go
// to different pairs and stand next to one another in the order.  The model
// behind "first" (units of 25 ns): a tile holds its pair for 0.3 us per 64 of
// its sum, or for its finish (3 us) where that is longer, and starts 1.5 us
// after the last of its matrix's tiles of the product before.  At 128 columns
// the finish is 1.75 us and the sum of A and B 0.225 us per 64; that of X is no
// shorter than at 256, as its stored rows of X are read and written beside it.
// Parts take 3 us to join.  It only balances the queues; the kernel waits for
// what has really happened.
static Deal deal(const Matrices& M, const std::vector<int32_t>& order, const Cut& cut, int pairs) {
    Deal out;
    out.mine.resize(size_t(pairs));
    using Free = std::pair<int64_t, int32_t>;
    std::priority_queue<Free, std::vector<Free>, std::greater<Free>> idle;   // {time, pair}
    for (int32_t p = 0; p < pairs; ++p) idle.push({0, p});
    std::vector<int64_t> ready(M.mats.size(), 0), next(M.mats.size(), 0);
    for (int prod = 0; prod < 3; ++prod) {
        const int blocks = cut.blocks[prod], per = 4 / blocks;
        const int64_t stage = per == 1 || prod == kProdX ? 12 : 9, finish = per == 1 ? 120 : 70, signal = 60;
        for (int32_t k : order) {
            const MatDesc& d = M.mats[size_t(k)];
            const int parts = prod == kProdA ? parts_of(d, cut) : 1;
            const int64_t sum = stage * ((prod == kProdA ? d.kn : d.km) + parts - 1) / parts;
            const int64_t join = parts > 1 ? 120 : 0;
            const int tm = d.cba / 4, tn = (prod == kProdX ? d.cbx : d.cba) / 4;
            int32_t group = d.group0;
            for (int i = 0; i < tm; ++i)
                for (int j = prod == kProdX ? 0 : i * per; j < tn * per; ++j, ++group) {
                    Free f[4];
                    for (int s = 0; s < parts; ++s) {
                        f[s] = idle.top();
                        idle.pop();
                    }
                    for (int s = 0; s < parts; ++s) {
                        const int64_t start = std::max(f[s].first, ready[size_t(k)]);
                        // (a part holds its pair until the last one is there)
                        const int64_t held = std::max(f[parts - 1].first, start) + std::max(sum, finish) + join;
                        const int64_t done = held - std::max(sum, finish) + sum + finish + signal;
                        next[size_t(k)] = std::max(next[size_t(k)], done);
                        out.end = std::max(out.end, done);
                        out.mine[size_t(f[s].second)].push_back({k, group, int16_t(i), int16_t(j), uint8_t(prod),
                                                                 uint8_t(blocks), uint8_t(s), uint8_t(parts >> 1)});
                        idle.push({held, f[s].second});
                    }
                }
        }
        ready = next;
    }
    return out;
}

// Tiles of a product are 256 columns wide or, where that lets the step end
// earlier in the model, 128: with few tiles, more pairs work at a product and
// each has half the finish.  Where rows are long, A's sums are also cut into
// two or four parts.  Measured with all three products at 256; A and B at 128;
// all at 128; A at 256 in four parts (two where the rows allow no more) and B
// at 128 (us, 76 pairs):
//     4 of 768 x 2304, 4 of 768 x 768   257   246   263   250
//     4 of 768 x 768                    186   168   156     -
//     4 of 2048 x 2048                  591   673   816     -
//     4 of 1024 x 4096                  395   369   454   355
//     6 of 300 x 5000                   345   323   334   286
//     200 x 10000                       343   328   335   198
// (Later steps made all of them 2 to 4 % faster.)  For these, and for ten of
// twelve other sets, the model picks the fastest of
// the mixtures; for the two (512 x 2048, 768 x 3000) one that is 2 % behind.
void lay_queue(Matrices& M, int clusters) {
    std::vector<int32_t> order(M.mats.size());
    for (size_t k = 0; k < order.size(); ++k) order[k] = int32_t(k);
    std::stable_sort(order.begin(), order.end(), [&](int32_t x, int32_t y) {
        const MatDesc &u = M.mats[size_t(x)], &v = M.mats[size_t(y)];
        return u.m != v.m ? u.m > v.m : u.n > v.n;
    });
    int64_t wide = 0;   // X tiles of 256 columns
    for (const MatDesc& d : M.mats) wide += int64_t(d.cba / 4) * (d.cbx / 4);
    Deal best;
    Cut cut{};
    for (int c = 0; c < 20; ++c) {
        // A: whole at 256, whole at 128, in two or four parts at 256, in two at 128
        static const int a_blocks[5] = {4, 2, 4, 4, 2}, a_parts[5] = {1, 1, 2, 4, 2};
        const Cut u{{a_blocks[c >> 2], c & 1 ? 2 : 4, c & 2 ? 2 : 4}, a_parts[c >> 2]};
        if (u.parts > clusters) continue;
        Deal d = deal(M, order, u, clusters);
        if (c == 0 || d.end < best.end) {
            best = std::move(d);
            cut = u;
        }
        if (wide > 16 * int64_t(clusters)) break;   // enough tiles for every pair as they are
    }
    for (MatDesc& d : M.mats) {
        const int64_t tm = d.cba / 4, tn = d.cbx / 4;
        const int parts = parts_of(d, cut);
        for (int prod = 0; prod < 3; ++prod)
            d.tiles[prod] = int32_t((prod == kProdX ? tm * tn : tm * (tm + 1) / 2) * (4 / cut.blocks[prod]) *
                                    (prod == kProdA ? parts : 1));
        d.groups = parts > 1 ? d.tiles[kProdA] / parts : 0;
    }
    // pairs without a tile come last: none is given one before an idle pair
    while (!best.mine.empty() && best.mine.back().empty()) best.mine.pop_back();
    M.pairs = int32_t(best.mine.size());
    M.queue.clear();
    M.queue_first.assign(1, 0);
    for (const auto& q : best.mine) {
        M.queue.insert(M.queue.end(), q.begin(), q.end());
        M.queue_first.push_back(int32_t(M.queue.size()));
    }
}

// Largest |a s + b s^3 + c s^5| for s in [0, hi]: at an end or where the
// derivative a + 3 b l + 5 c l^2, l = s^2, vanishes.  Coefficients are divided
// by the largest, and each root is a quotient that does not cancel (for a tiny
// c the textbook formula gives 0 in place of the root -a / 3 b).
static double largest_odd(double a, double b, double c, double hi) {
    const double size = std::max(std::fabs(a), std::max(std::fabs(b), std::fabs(c)));
    if (size == 0.0) return 0.0;
    a /= size;
    b /= size;
    c /= size;
    auto p = [&](double s) { return std::fabs(s * (a + s * s * (b + c * s * s))); };
    double best = p(hi);
    const double A = 5.0 * c, B = 3.0 * b, disc = B * B - 4.0 * A * a;
    if (disc >= 0.0) {
        const double q = -0.5 * (B + std::copysign(std::sqrt(disc), B));   // roots q / A and a / q
        for (const double l : {A != 0.0 ? q / A : 0.0, q != 0.0 ? a / q : 0.0})
            if (l > 0.0 && l < hi * hi) best = std::max(best, p(std::sqrt(l)));
    }
    return best * size;
}

// Largest |b l + c l^2| for l in [0, hi].
static double largest_quad(double b, double c, double hi) {
    double best = std::fabs(b * hi + c * hi * hi);
    if (c != 0.0) {
        const double l = -b / (2.0 * c);
        if (l > 0.0 && l < hi) best = std::max(best, std::fabs(b * l + c * l * l));
    }
    return best;
}

// The power of two that maps values up to `most` below 2^15 with a factor of
// two to spare for rounding (fp16 ends at 65504).
static float scale_for(double most) {
    int e = 0;
    std::frexp(std::max(most, 1e-12), &e);   // most < 2^e
    return float(std::ldexp(1.0, 14 - e));
}

// How much a step may enlarge an error in an eigenvalue l of the Gram matrix:
// the largest slope of l (a + b l + c l^2)^2 over [0, hi], at least 1.  It is
// a^2 at 0, and there it counts: an eigenvalue that rounding made negative
// meets a factor that grows with its size, so nothing brings it back.
static double gram_growth(double a, double b, double c, double hi) {
    double most = 1.0;
    for (int i = 0; i <= 4; ++i) {
        const double l = hi * i / 4.0, q = a + l * (b + l * c);
        most = std::max(most, std::fabs(q * (q + 2.0 * l * (b + 2.0 * c * l))));
    }
    return most;
}

// Cuts the steps into phases; the Gram path applies a phase's product to X and
// sums the Gram matrix of the new X before the next one.  growth: of each step.
// The sum's rounding (1e-8 to 1e-7 of the largest eigenvalue) times the growth
// of a phase is what a phase adds to the result.  Five default steps (2.4e5) as
// one phase: up to 7e-4 for a matrix of rank one, three launches.  Whatever
// grows by more is cut at 2000 (three default steps), where the phases together
// leave no more than the iteration on X in binary32 does (1e-5 to 2e-4): each
// phase is three launches more, and cut at 2.4e5 too they left up to 2e-3.
static void gram_phases(const double* growth, int n_steps, bool precise, OrthoSchedule* sch) {
    constexpr double kOnePhase = 2.4e5, kEach = 2000.0;
    double all = 1.0, phase = 1.0;
    for (int k = 0; k < n_steps; ++k) all *= growth[k];
    sch->n_phases = 0;
    for (int k = 0; k < n_steps; ++k) {
        if (k > 0 && phase * growth[k] > kEach && (all > kOnePhase || precise)) {
            sch->phase_end[sch->n_phases++] = k;
            phase = 1.0;
        }
        phase *= growth[k];
    }
    sch->phase_end[sch->n_phases++] = n_steps;
}

// Which steps of the tiles take both halves of their operands.  In directions
// that X lacks, what a step's roundings leave there is multiplied by the a_k of
// the steps after it.  With fp16 halves alone (3e-4 a step) five default steps
// end within 2.7e-3 for 256 rows and more whatever the matrix (4e-3 for 129), six
// at 6e-3 and eight at 7e-2 (every row twice, or rank m / 2).  Where the a_k multiply to more than those five
// (485), the steps with more than 4 still to come -- all but the last two of
// default ones -- take both: the end is within 1.3e-3 again.  Such a step takes
// two to three times as long (eight GPT-2-small attention matrices 88 us
// against 41, a 1B model's layer 1.1 ms against 0.34).
static void both_halves(const dpg_muon_hparams* hp, OrthoSchedule* sch) {
    double all = 1.0, to_come = 1.0;
    for (int k = 0; k < hp->n_steps; ++k) all *= std::max(1.0, std::fabs(hp->coeffs[k][0]));
    sch->both_steps = hp->precise ? hp->n_steps : 0;
    for (int k = hp->n_steps - 1; k >= 0 && all > 490.0 && !hp->precise; --k) {
        if (to_come > 4.0) {
            sch->both_steps = k + 1;
            break;
        }
        to_come *= std::max(1.0, std::fabs(hp->coeffs[k][0]));
    }
}

int ortho_steps(const dpg_muon_hparams* hp, OrthoSchedule* sch, const char* who) {
    if (!hp) return fail(DPG_ERR_INVALID_ARG, "%s: hparams is NULL", who);
    if (hp->n_steps < 1 || hp->n_steps > DPG_MAX_NS_STEPS)
        return fail(DPG_ERR_INVALID_ARG, "%s: n_steps %d outside [1, %d]", who, hp->n_steps,
                    DPG_MAX_NS_STEPS);
    if (!(hp->eps >= 1e-30) || !std::isfinite(hp->eps))
        return fail(DPG_ERR_INVALID_ARG, "%s: eps must be finite and >= 1e-30", who);
    // Every entry of a matrix is at most its largest singular value, which is
    // at most 1 for X_0 and at most largest_odd() of the previous bound after
    // a step; the entries of A and of bA + cA^2 follow.  The 1% covers what
    // the roundings of a step can add.
    double top = 1.0, growth[DPG_MAX_NS_STEPS];
    float sx = 0.0f;
    for (int k = 0; k < hp->n_steps; ++k) {
        const double a = hp->coeffs[k][0], b = hp->coeffs[k][1], c = hp->coeffs[k][2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
            return fail(DPG_ERR_INVALID_ARG, "%s: coeffs[%d] not finite", who, k);
        growth[k] = gram_growth(a, b, c, top * top);
        OrthoStep& s = sch->st[k];
        s.a = float(a);
        s.b = float(b);
        s.c = float(c);
        s.inv_sx = k == 0 ? 0.0f : 1.0f / sx;
        s.sa = scale_for(top * top);
        s.inv_sa = 1.0f / s.sa;
        s.sb = scale_for(largest_quad(b, c, top * top));
        s.inv_sb = 1.0f / s.sb;
        top = std::max(largest_odd(a, b, c, top) * 1.01, 1e-6);
        if (!(top <= 32.0))
            return fail(DPG_ERR_INVALID_ARG, "%s: after step %d singular values may reach %g", who, k, top);
        s.sx_next = sx = scale_for(top);
    }
    gram_phases(growth, hp->n_steps, hp->precise != 0, sch);
    both_halves(hp, sch);
    return DPG_OK;
}

}  // namespace dpg

using dpg::fail;

extern "C" {

int dpg_plan_matrices(const dpg_plan_t* plan, const int64_t* rows, const int64_t* cols,
                      dpg_matrices_t** out) {
    dpg::clear_error();
    if (!out) return fail(DPG_ERR_INVALID_ARG, "dpg_plan_matrices: out is NULL");
    *out = nullptr;
    if (!plan) return fail(DPG_ERR_INVALID_ARG, "dpg_plan_matrices: plan is NULL");
    const dpg::Plan& p = plan->p;
    if (p.n_params > 0 && (!rows || !cols))
        return fail(DPG_ERR_INVALID_ARG, "dpg_plan_matrices: rows or cols is NULL");
    for (int32_t q = 0; q < p.n_params; ++q) {
        if (rows[q] < 1 || cols[q] < 1 || rows[q] > (1 << 23) || cols[q] > (1 << 23))
            return fail(DPG_ERR_INVALID_ARG, "dpg_plan_matrices: parameter %d: shape outside [1, 2^23]", q);
        if (p.numels[q] % (rows[q] * cols[q]) != 0)
            return fail(DPG_ERR_INVALID_ARG,
                        "dpg_plan_matrices: parameter %d: %lld elements are no stack of %lld x %lld", q,
                        (long long)p.numels[q], (long long)rows[q], (long long)cols[q]);
    }
    dpg_matrices* h = new (std::nothrow) dpg_matrices();
    if (!h) return fail(DPG_ERR_OOM, "dpg_plan_matrices: out of host memory");
    bool ok = false;
    try {
        ok = dpg::lay_out(p, rows, cols, h->m);
    } catch (const std::exception&) {
        delete h;
        return fail(DPG_ERR_OOM, "dpg_plan_matrices: out of host memory");
    }
    if (!ok) {
        delete h;
        return fail(DPG_ERR_INVALID_ARG, "dpg_plan_matrices: matrices too large for one object");
    }
    *out = h;
    return DPG_OK;
}

void dpg_matrices_destroy(dpg_matrices_t* mats) {
    if (!mats) return;
    dpg::release_matrices(mats->m);
    delete mats;
}

int dpg_matrices_info(const dpg_matrices_t* mats, int32_t* n_matrices, int64_t* workspace_bytes) {
    dpg::clear_error();
    if (!mats) return fail(DPG_ERR_INVALID_ARG, "dpg_matrices_info: mats is NULL");
    if (n_matrices) *n_matrices = mats->m.n_matrices;
    if (workspace_bytes) *workspace_bytes = mats->m.workspace_bytes;
    return DPG_OK;
}

int dpg_matrices_status(dpg_matrices_t* mats, void* stream) {
    dpg::clear_error();
    if (!mats) return fail(DPG_ERR_INVALID_ARG, "dpg_matrices_status: mats is NULL");
    return dpg::check_matrices(mats->m, stream);
}

int dpg_matrices_upload(dpg_matrices_t* mats) {
    dpg::clear_error();
    if (!mats) return fail(DPG_ERR_INVALID_ARG, "dpg_matrices_upload: mats is NULL");
    return dpg::upload_matrices(mats->m, false);
}

}  // extern "C"
