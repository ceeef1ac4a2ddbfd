// Host side that the bf16 and the 8-bit products share: which tiles a product
// takes, and the workspace of those whose contraction is split.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "epl.h"
#include "epl_product_kernels.h"

namespace epl_product_host {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int launch_status() { return hipGetLastError() == hipSuccess ? EPL_OK : EPL_EHIP; }

inline bool is_grad(int act)
{
    return act == EPL_ACT_SILU_GRAD || act == EPL_ACT_GELU_GRAD || act == EPL_ACT_SWIGLU_GRAD;
}

// Offsets within one expert's weight and within a tile are 32-bit.
constexpr int32_t kMaxCols = 1 << 20;

// The kernels step through an expert's rows in 32-bit counts, by up to a tile
// and the four rows read ahead of it.
constexpr int64_t kMaxRows = INT32_MAX - 1023;

// CUs that a launch counts on, at most (and those of an MI355X).
constexpr int kCus = 256;

inline int num_cus()
{
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1) {
        (void)hipGetLastError();
        return kCus;
    }
    return std::min(n, kCus);
}

// The kernel that a product takes: straight from memory for a few rows, or
// tiles of 256 x 256 or 128 x 128. The counts are on the GPU, so the choice
// goes by the rows that the caller expects an expert to have on average, however
// unevenly they fall.
enum Kind { kFew, kLarge, kSmall };

inline int side_of(Kind k) { return k == kSmall ? 128 : 256; }

// Parts that a contraction of `depth` is split into at most: of four stages of
// `deep` each at least.
inline int max_parts(int64_t depth, int deep)
{
    return (int)std::min<int64_t>(epl_product::kMaxParts, depth / (4 * deep));
}

inline int stages_of(int64_t depth, int deep) { return (int)((depth + deep - 1) / deep); }

// What a round of tiles costs (us): its start and epilogue, and a stage.
struct Cost {
    double start, stage;
};

// About how long (us) `experts` products of m x n outputs, `depth` deep, take
// with tiles of one kind, of which the GPU holds one round (256 large, or 512
// small ones) at a time.
inline double tiles_time(Kind k, int64_t m, int64_t n, int64_t experts, int64_t depth, int deep, Cost c)
{
    const int side = side_of(k), round = kCus * epl_product::tile_groups(side), stages = stages_of(depth, deep);
    const int64_t tiles = experts * ((m + side - 1) / side) * ((n + side - 1) / side);
    const int left = (int)(tiles % round);
    const int parts = epl_product::parts_of(left, round, max_parts(depth, deep), stages, side);
    double t = (double)(tiles / round) * (c.start + c.stage * stages);
    if (left > 0)
        t += c.start + c.stage * stages / parts +
             (parts > 1 ? left * parts * c.stage / (k == kLarge ? 17 : 42) : 0.0);
    return t;
}

// A workspace: what tile_kernel tells join_kernel, then the partial tiles.
constexpr size_t kHeaderBytes = 256;

inline size_t tile_workspace(Kind k, int64_t tiles, int parts)
{
    if (k == kFew || parts < 2)
        return 0;
    const int64_t slots = std::min<int64_t>(kCus * epl_product::tile_groups(side_of(k)), tiles * parts);
    return kHeaderBytes + (size_t)slots * side_of(k) * side_of(k) * sizeof(float);
}

inline void use_workspace(epl_product::Args &a, void *workspace)
{
    a.header = static_cast<int *>(workspace);
    a.ws = workspace ? reinterpret_cast<epl_product::f32x4 *>(static_cast<char *>(workspace) + kHeaderBytes)
                     : nullptr;
}

// Tiles of a product's outputs, at most: experts' last tiles are their own.
inline int64_t product_tiles(int64_t rows, int64_t experts, int64_t cols, Kind k)
{
    return (rows / side_of(k) + experts) * ((cols + side_of(k) - 1) / side_of(k));
}

// Workgroups of a tile kernel: every one that the CUs hold at once, striding
// over the tiles; also with fewer tiles where their contraction can be split.
// `tiles`: how many there are, or at most are.
inline int tile_grid(const epl_product::Args &a, int64_t tiles, int side, bool split)
{
    const int most = num_cus() * epl_product::tile_groups(side);
    return (int)std::min<int64_t>(split ? tiles * a.max_parts : tiles, most);
}

// Workgroups of the join behind it, for each of its pieces.
inline unsigned join_grid(int64_t tiles, int grid)
{
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(tiles, grid / 2));
}

}  // namespace epl_product_host
