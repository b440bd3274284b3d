// How the 16-bit products (zero_matmul.cu) divide their work: shared memory and stages of
// their blocks, splits of the columns c, tile widths.  Host arithmetic and
// constants, without CUDA, so that it is tested by itself.
#pragma once

#include <atomic>
#include <cstdint>

#ifdef __CUDACC__
#define ZGB_BOTH __host__ __device__
#else
#define ZGB_BOTH
#endif

namespace zgb {

constexpr int kSmemSm = 233472;      // shared memory of an SM
constexpr int kSmemBlock = 231424;   // dynamic shared memory that leaves room for no other block

namespace product {

constexpr int kDepth = 64;                       // columns c of a stage: 128 bytes
constexpr int kLine = 128;
constexpr int kHalf = 128 * kLine;               // 128 rows of an operand in a stage

constexpr int kOneWarps = 8;                     // of results, before copies and products
constexpr int kOneThreads = (kOneWarps + 2) * 32;
constexpr int kMostBlocks = 2;                   // of an SM

constexpr int kStagePad = 33;                    // floats of a row that changes places
constexpr int kPitch = 132;                  // a lane a row: no two of eight on one bank

// Floats of shared memory that a split's block needs.
ZGB_BOTH constexpr int split_floats(int span, int splits)
{
    return (span + (splits > 1 ? splits * ((span + splits - 1) / splits) : 0)) * kPitch;
}

constexpr int staged_floats() { return kOneThreads / 32 * 32 * kStagePad; }

// A block of matmul_kernel, with nt rows of A in a tile.
struct Tile {
    static constexpr int kStages = 8;                       // at most
    static ZGB_BOTH constexpr int stage(int nt) { return kHalf + nt * kLine; }
    static ZGB_BOTH constexpr int tmem(int nt)
    {
        return nt <= 32 ? 32 : nt <= 64 ? 64 : nt <= 128 ? 128 : 256;
    }
    // A block's share of an SM's shared memory is at least its share of the tensor
    // memory, so that no block waits for tensor memory that another one
    // holds: two that wait for their cluster peers so would wait forever.
    static constexpr int smem(int stages, int nt, int splits, bool staged)
    {
        // the sums, when they are done, a split's shares of them, and room to reorder
        const int part = (split_floats(nt, splits) + (staged ? staged_floats() : 0)) * 4;
        const int ring = stages * stage(nt) > part ? stages * stage(nt) : part;
        const int share = (kSmemSm / (512 / tmem(nt)) + 127) / 128 * 128;
        return ring + 1024 > share ? ring + 1024 : share;
    }
    // Stages of the longest ring.
    static constexpr int most(int nt)
    {
        return (kSmemBlock - 1024) / stage(nt) < kStages ? (kSmemBlock - 1024) / stage(nt)
                                                         : kStages;
    }
};

// A block of matmul_mid_kernel.
constexpr int kMidStages = 7;

ZGB_BOTH constexpr int mid_stage(int wide) { return kHalf + wide * kLine; }
ZGB_BOTH constexpr int mid_gated_stage(int nt, int wide) { return (nt + 2 * wide) * kLine; }

constexpr int mid_smem(int stages, int wide, int splits, bool staged)
{
    const int ring = stages * mid_stage(wide);
    const int part = ((splits > 1 ? split_floats(128, splits) : 0) +
                      (staged ? staged_floats() : 0)) * 4;
    return (ring > part ? ring : part) + 1024;
}
static_assert(mid_smem(kMidStages, 128, 8, true) <= kSmemBlock, "one block's shared memory");

// (its share of an SM's at least, half, as its tensor memory is: see Tile)
constexpr int mid_gated_smem(int stages, int nt, int wide)
{
    const int ring = stages * mid_gated_stage(nt, wide);
    const int most = ring > staged_floats() * 4 ? ring : staged_floats() * 4;
    return most + 1024 > kSmemSm / 2 ? most + 1024 : kSmemSm / 2;
}

// Rows of A in each of `tiles_m` tiles, as equal as multiples of 16 can be.
inline int width(int64_t m, int64_t tiles_m)
{
    return (int)((m + tiles_m * 16 - 1) / (tiles_m * 16) * 16);
}

// How many clusters of `splits` blocks of a kernel find a place at once: fewer than
// the SMs' number says, because a cluster's blocks share a group of SMs.  Asked for once
// for each device (of the first sixteen), split and ring length.
struct Room {
    static constexpr int kDevices = 16, kRing = 8;       // kRing: stages of the longest ring
    std::atomic<int16_t> known[kDevices][9][kRing + 1] = {};
    // ask(splits, smem, found): whether the device answers, and what
    template <class Ask> int of(int device, int splits, int stages, int smem, Ask ask)
    {
        const bool kept = device >= 0 && device < kDevices;
        std::atomic<int16_t> &at = known[kept ? device : 0][splits][stages];
        const int n = kept ? at.load(std::memory_order_relaxed) : 0;
        if (n) return n - 1;
        int found = 0;
        if (!ask(splits, smem, found)) return 0;         // no answer: asked again next time
        if (kept) at.store((int16_t)(found < 32766 ? found + 1 : 32767), std::memory_order_relaxed);
        return found;
    }
};
static_assert(Tile::kStages <= Room::kRing && kMidStages <= Room::kRing, "the table's last entry");

// A split, the ring's length, and the stages of the fullest SM.
struct Cut {
    int splits, stages;
    int64_t least;
};

// The split that leaves the fullest SM the fewest of the kt stages, a join
// counting as kJoin of them, as long as all clusters find a place at once.
// `smem(stages, splits)`: a block's shared memory; `most`: stages of the longest ring;
// `room(splits, stages, smem)`: clusters that find a place.
template <class Smem, class Place>
Cut choose_split(int64_t kt, int64_t tiles, int sms, int most, int blocks_sm, Smem smem,
                 Place room)
{
    constexpr int kJoin = 4;
    auto ring = [&](int splits, int per_sm) {
        const int64_t rounds = (kt + splits - 1) / splits;
        int st = rounds < 1 ? 1 : rounds < most ? (int)rounds : most;
        // (a block has what its kernel is allowed, blocks together what the SM has)
        while (st > 0 && (smem(st, splits) > kSmemBlock ||
                          (smem(st, splits) + 1024) * per_sm > kSmemSm))
            --st;
        return st;
    };
    const int64_t deep = (tiles + sms - 1) / sms;        // whole tiles of the fullest SM
    Cut c = {1, ring(1, deep < blocks_sm ? (int)deep : blocks_sm), deep * kt};
    for (int n = 2; n <= 8 && kt >= 2 * n; ++n) {
        const int64_t per_sm = (tiles * n + sms - 1) / sms;
        if (per_sm > blocks_sm) break;
        const int64_t rounds = (kt + n - 1) / n, cost = per_sm * rounds + kJoin;
        if (cost >= c.least) continue;
        // (blocks that share an SM want three stages at least to keep their copies coming)
        const int st = ring(n, (int)per_sm);
        if (st < 1 || (st < 3 && st < rounds) || room(n, st, smem(st, n)) < tiles) continue;
        c = {n, st, cost};
    }
    return c;
}

// How matmul_pair_kernel goes over an m by n result.
struct PairShape {
    int half;                            // rows of B that either block brings, at most 128
    int cut;                             // parts of a tile from tile `whole` on
    int64_t tiles_m, tiles_n, whole, steps;
};

inline PairShape pair_shape(int64_t m, int64_t n, int sms, bool gated)
{
    PairShape g;
    // The tile's width that leaves the pairs the least columns to go through, one after
    // the other: with few tiles a pair, 256 can leave most of them idle at the end.
    // (6400 x 1600 over 8192 columns c, 76 pairs: 175 tiles of 256 go three deep, and so
    // do 225 of 192.)
    // A narrower tile reads A more often: it has to save an eighth.
    g.tiles_m = (m + 255) / 256;
    int64_t least = 0;
    for (int half = 128; half >= 64; half -= gated ? 32 : 16) {   // blocks of 32 stay whole
        const int64_t wide = gated ? half : 2 * half, across = (n + wide - 1) / wide;
        const int64_t deep = (across * g.tiles_m + sms / 2 - 1) / (sms / 2) * half;
        if (half < 128 && deep * 8 > least * 7) continue;
        least = deep;
        g.half = half;
        g.tiles_n = across;
    }
    // The last turn's tiles, if they leave pairs idle, in halves or quarters (a gated
    // tile's parts are 32 columns at least, and whole blocks of 32).
    const int64_t tiles = g.tiles_n * g.tiles_m, left = tiles % (sms / 2);
    g.cut = 1;
    for (int cut = 2; cut <= 4; cut *= 2)
        if (left * cut <= sms / 2 && g.half % (cut * (gated ? 32 : 16)) == 0) g.cut = cut;
    g.whole = g.cut > 1 ? tiles - left : tiles;
    g.steps = g.whole + (tiles - g.whole) * g.cut;
    return g;
}

}  // namespace product
}  // namespace zgb
