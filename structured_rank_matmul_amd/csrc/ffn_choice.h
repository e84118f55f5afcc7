// Which kernel a feed-forward call runs, from its sizes alone: host code without
// HIP, so that a test on the CPU can list the variants and see that each is
// tested.  Sizes are of the argument checks' ranges; `elem` is the bytes of an
// operand's element (1, 2 or 4).
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace dyra {

// ------------------------------------------------------------------ linear layer, gated pair

// Up to this many tokens the weights are streamed (skinny_linear.h).
constexpr int64_t kSkinnyTokens = 32;
// Whether X is streamed and the weights' rows take the tokens' part (launch_narrow):
// few features, one unit of 16 tokens a CU; float32, where the tiles are bound by their
// MFMAs, up to four with one block of features and two with two.  Tiles | narrow,
// us: bf16 2048 x 4096 -> 32 13.4 | 8.9, 2048 x 7168 -> 8 21.2 | 7.9, 8192 x 4096 -> 32
// 14.2 | 18.7; float32 1589 x 9184 -> 32 105 | 30, 16384 x 768 -> 10 16.8 | 11.5, 8000 x 2048
// -> 32 26.3 | 20.1, 16384 x 768 -> 32 17.0 | 18.4.
inline bool takes_narrow(int elem, bool gated, int64_t M, int64_t N) {
    const int blocks = gated || N > 16 ? 2 : 1;
    return N <= (gated ? 16 : 32) && M <= 16 * 256 * (elem == 4 ? 4 / blocks : 1);
}

// Few tokens: slabs of K that a wavefront's registers hold of each of `blocks` of 16
// tokens (skinny_kernel), or 0 where the tokens go through the ring.
struct FewTokens {
    int slabs, blocks;
};
inline int64_t few_token_units(bool gated, int64_t N) { return (N + (gated ? 7 : 15)) / (gated ? 8 : 16); }
inline FewTokens few_tokens(bool gated, int64_t M, int64_t N, int64_t row_bytes) {
    // registers hold a wavefront's slabs of the tokens (8 a slab and block of 16)
    // up to 24 slabs of one block or 12 of two; they pay from the third unit of a
    // workgroup on (two blocks: the second)
    const int64_t units = few_token_units(gated, N), slabs = (row_bytes + 1023) / 1024;  // of 128 bytes, in 8 wavefronts
    if (M <= 16 && units > 512 && slabs <= 24)
        return {slabs <= 2 ? 2 : slabs <= 4 ? 4 : slabs <= 8 ? 8 : slabs <= 16 ? 16 : 24, 1};
    if (M > 16 && M <= 32 && units > 256 && slabs <= 12) return {slabs <= 4 ? 4 : slabs <= 8 ? 8 : 12, 2};
    return {0, 1};
}

// Tile shapes by tokens and weight rows (gated: gate and up rows together), and the
// time of a round of one tile per CU: per slab in bf16 and in float32 (ns; a slab is 64
// bf16 or 32 floats of K), and for the start and the epilogue.  From whole calls of one
// and of four full rounds at K = 1024 and 4096, plain and gated, reads from memory
// included; taken again, bf16: 174 to 196, 193 to 282, 290 to 342, 512 to 605, 854 to
// 892, 1092 to 1142, 1190 to 1231, 1332 to 1338; float32: 345 to 369, 492 to 563, 995 to
// 1093, 1861 to 1955.  The first stays at 150: with 185, 40 random shapes whose choice
// that changes (64 x 64 for 32 x 64) ran 10 % slower.  What every tile reads alike, the
// operands once, is left out: at 64 x 4096 -> 2 x 14336 that is half of the time.  What the
// choice is worth, us by tile (128 x 256 | 192 | 224 | 256 x 256): 448 363 333 336 at
// 14336 x 4096 -> 4096, 388 307 306 276 at 12288, 237 212 173 181 at 25728 x 4096 ->
// 1024, 62 62 65 71 at 2048 x 4096 -> 4096 (the library's product: 330, 265, 166, 55).
enum Tile { T32x64, T64x64, T64x128, T128x128, T128x256, T192x256, T224x256, T256x256 };
struct TileCost {
    int bm, bn;
    double slab, slab_f32, once;
};
constexpr TileCost kTiles[] = {{32, 64, 150, 345, 2500},    {64, 64, 230, 520, 2500},  {64, 128, 305, 1015, 3500},
                               {128, 128, 550, 1905, 4000}, {128, 256, 870, 0, 5500},  {192, 256, 1110, 0, 4000},
                               {224, 256, 1220, 0, 5000},   {256, 256, 1340, 0, 6000}};

// Start and epilogue of a tile.  Large tiles of 8-bit operands have half the slabs of bf16, and
// scales: fitted anew, by the bytes of their results (in bf16), to 64 products of 300 to 32768
// tokens, each with bf16 and float32 results.  The choice is 0.8 % behind the best tile of
// all on average; with bf16's times 3.2, as 192 | 256 x 256 us 137 | 130 at 25728 x 1024 -> 4096, 414
// | 363 at gated 12093 x 1104 -> 11776, 128 x 256 | 192 x 256 12.9 | 19.1 at 2109 x 272 -> 2944.
inline double tile_once(int elem, bool gated, int tile) {
    const TileCost &t = kTiles[tile];
    return elem == 1 && tile >= T128x256 ? 2400.0 + 0.035 * t.bm * t.bn * (gated ? 1 : 2) : t.once;
}
// The shape with the smallest estimated time.
inline Tile pick_tile(int elem, bool gated, int64_t M, int64_t N, int64_t row_bytes) {
    const double rows = (double)N * (gated ? 2 : 1), slabs = std::ceil((double)row_bytes / 128.0);
    Tile best = T32x64;
    double cost = 1e300;
    for (int i = T32x64; i <= (elem != 4 ? T256x256 : T128x128); ++i) {
        if (elem == 1 && i == T224x256) continue;  // not made: its epilogue does not fit the registers
        const TileCost &t = kTiles[i];
        const double rounds = std::ceil(std::ceil((double)M / t.bm) * std::ceil(rows / t.bn) / 256.0);
        const double c = rounds * (slabs * (elem != 4 ? t.slab : t.slab_f32) + tile_once(elem, gated, i));
        if (c < cost) {
            cost = c;
            best = (Tile)i;
        }
    }
    return best;
}

// 8-bit operands, whose sums are exact: K in `parts` that a product's tiles are made of by
// as many workgroups each, joined by a second kernel.  It pays for long rows and few tiles;
// the second kernel and the workspace cost 6 us.  The times of the tiles above are
// those of short rows: over long ones the smaller tiles took up to 1.5 times as long, parts of
// them 1.2 times (a fit to 90 products of 33 to 8000 tokens).  67 products that this splits took
// 0.62 of the whole's time on average, 0.98 at worst.  us, inputs past the caches, whole | split:
// 186 x 12416 -> 188 22.6 | 11.3, 64 x 14336 -> 4096 29.1 | 20.6, 185 x 11072 -> 1600 25.7 | 20.6,
// gated 1102 x 10288 -> 456 48.3 | 33.7, 166 x 10320 -> 3968 40.3 | 37.1, 583 x 5808 -> 3957 43.8 |
// 39.1; left whole: 64 x 4096 -> 4096 11.0 | 11.7, 256 x 4096 -> 4096 13.1 | 18.6, 512 x 4096 ->
// 4096 19.2 | 26.9, and, which it should split, gated 51 x 5584 -> 854 20.2 | 14.1.  The whole is
// priced with `once`, as in the fit: with tile_once() 14 products of rows of 37000 to 46000, which
// take 0.79 of the time split (gated 1597 x 40400 -> 1290 366 | 280), would be left whole.
struct Split {
    Tile tile;
    int parts;   // 1: no split
    int slabs;   // of a part (the last may have fewer)
};
// Sums of a row in the workspace, and what one call may take of it.
constexpr int64_t split_row(int64_t N) { return (N + 7) / 8 * 8; }
constexpr int64_t kSplitBytesMost = int64_t{64} << 20;
inline int64_t split_bytes(bool gated, int64_t M, int64_t N, int parts) {
    return parts > 1 ? (int64_t)parts * (gated ? 2 : 1) * M * split_row(N) * 4 : 0;
}
inline Split pick_split(bool gated, int64_t M, int64_t N, int64_t row_bytes) {
    const double rows = (double)N * (gated ? 2 : 1), slabs = std::ceil((double)row_bytes / 128.0);
    const Tile whole = pick_tile(1, gated, M, N, row_bytes);
    const double count = std::ceil((double)M / kTiles[whole].bm) * std::ceil(rows / kTiles[whole].bn);
    Split best{whole, 1, (int)slabs};
    if (whole > T128x256) return best;  // tiles enough; and a gelu that does not depend on the workspace (gelu_table.h)
    double cost = 0.9 * std::ceil(count / 256.0) * (slabs * kTiles[whole].slab * (whole <= T128x128 ? 1.5 : 1.0) + kTiles[whole].once);
    for (int i = T64x64; i <= T128x256; ++i) {
        const TileCost &t = kTiles[i];
        const double tiles = std::ceil((double)M / t.bm) * std::ceil(rows / t.bn);
        for (int want = 2; want <= 16; ++want) {
            // whole stages of up to two slabs; at least 8 slabs a part
            const int per = 2 * (int)std::ceil(slabs / want / 2.0), parts = (int)std::ceil(slabs / per);
            if (per < 8 || parts < 2) break;
            const int64_t bytes = split_bytes(gated, M, N, parts);
            if (bytes > kSplitBytesMost) break;
            const double c = std::ceil(tiles * parts / 256.0) * (per * t.slab * 1.2 + t.once) + 6000.0 + (double)bytes / 4000.0;
            if (c < cost) {
                cost = c;
                best = {(Tile)i, parts, per};
            }
        }
    }
    return best;
}

// ------------------------------------------------------------------ expert layer

// Pairs (token, place) and experts that one call takes.
constexpr int kMoeMaxPairs = 1024;
constexpr int kMoeMaxExperts = 1024;
// Of split sums, a token: at most 256 workgroups of 8 features in float32.
constexpr int kMoePartBytes = 256 * 8 * 4;
// Pairs of one moe_down workgroup: 16 KB of sums.
constexpr int down_pairs(int rows) { return 4096 / rows; }

// Slabs of c in a wavefront's registers (moe_up_kernel).
inline int up_slabs(int64_t row_bytes) {
    const int64_t slabs = (row_bytes + 1023) / 1024;
    return slabs <= 2 ? 2 : slabs <= 4 ? 4 : slabs <= 8 ? 8 : 12;
}

// Features and pairs of a slot of moe_down_kernel.
struct Down {
    int rows, slot;
};
inline Down down_kernel(int T, int k, int experts, int64_t c) {
    // 8 rows a workgroup while that gives no more workgroups than CUs (each takes
    // one), or where 16 would read the weights for a second chunk of tokens; else
    // 16: 8 tokens, 32 experts, 4 places, 2880 x 1024 72 us against 86.  Slots of 8
    // where experts have 6 pairs on average or less
    const int pairs = T * k;
    return {c <= 8 * 256 || pairs > down_pairs(16) ? 8 : 16, T <= 8 || pairs <= 6 * experts ? 8 : 16};
}
// Workgroups that share the slabs of the same features (1: none do); `parts` whether
// the workspace has room for their sums, `rest` whether H has two parts.
inline int down_splits(Down d, int elem, int T, int k, int experts, int64_t c, int64_t f, bool parts, bool rest) {
    // One workgroup streams about 50 bytes a ns.  The slabs are shared by as many as
    // there are CUs for, down to 150 KB each, where that saves 8 us: the join takes 5
    // and a launch more of the host.  57 tokens, 9 experts, 4 places, 360 x 5432: 98 ->
    // 29 + 5 us; 10 tokens, 17 experts, 8 places, 296 x 1064: 15 -> 11 + 4.
    const int chunk = std::min(T, down_pairs(d.rows) / k);
    const int64_t rows = (c + d.rows - 1) / d.rows, chunks = (T + chunk - 1) / chunk;
    const int64_t bytes = std::min<int64_t>((int64_t)chunk * k, experts) * f * elem * (d.rows + (rest ? 2 : 1) * d.slot);
    const int64_t splits = std::min(256 / (rows * chunks), bytes / 150000);
    return splits > 1 && parts && splits * c * 4 <= kMoePartBytes && (double)bytes * (1 - 1.0 / (double)splits) > 400e3
               ? (int)splits : 1;
}

}  // namespace dyra
