// linear_plan.hpp -- which kernels a product with FP4 weights runs (linear.hip),
// from its types and sizes alone.  Host code.
#pragma once

#include <algorithm>

#include "linear_device.hpp"

namespace fp4q_dev {

// What a call runs, from its types and sizes alone.
enum class Kind { kSkinny, kTile32, kTile64, kTile128, kTile256 };

struct LinearPlan {
    Kind kind;
    int np;                    // bf16 planes of an activation
    bool copy;                 // activations go through k_linear_planes
    int64_t pitch;             // of a plane
    size_t plane_bytes;        // room for all planes of R rows
    int64_t tiles_m, tiles_o;
    int splits, split_steps;
    int64_t ld_part;
    size_t part_bytes;
};

constexpr int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

constexpr size_t round256(int64_t n) { return (size_t)(n + 255) / 256 * 256; }

// Rows of this many bytes or more together are beyond the tiles' 32-bit offsets.
constexpr int64_t kMaxGatherBytes = ((int64_t)1 << 32) - 65536;

// Whether 16-bit rows of this pitch are.
inline bool far_rows(int64_t rows, int64_t pitch) { return rows * pitch * 2 >= kMaxGatherBytes; }

// How the weights go to the matrix cores.
inline int weight_format(int sf, int x_dt) {
    return sf == SF_E8M0 ? WF_E8M0 : x_dt == DT_F16 ? WF_E4M3_F16 : WF_E4M3;
}

// Weight-row tiles of a few-row workgroup: the widest that still fills the
// device.  x is read once per workgroup (16 rows at 14336 x 4096: 14.7 us with
// 64 weight rows a workgroup, 24 with 16), but 4096 rows of weights keep only
// 64 workgroups of 64 busy (20 against 14 us at 4096 x 14336, NVFP4).
inline int few_rows_tiles(bool grouped, int64_t R, int64_t N, int E) {
    const int64_t n16 = (grouped ? std::min<int64_t>(E, R) : (R + 15) / 16) * ((N + 15) / 16);
    return n16 >= 4 * 224 ? 4 : n16 >= 2 * 224 ? 2 : 1;
}

// Which kernel runs.  Measured on bf16 (us a call at 4096 x 4096 / 14336 x
// 4096 weights, rows in front): the few-row kernel is ahead of the 32-row tile
// up to 16 rows (1: 11 / 12.5 against 16 / 16, 16: 11 / 14.7 against 16.5 /
// 16.2), from where its x reads cost more than the weights'.  Small tiles
// fill the device and need fewer parts to join: 64 rows a tile is ahead of
// 128 until there are about 448 of them (256 rows: 21 / 35.5 against 22 /
// 35.5, 512: 24 / 66 against 29 / 59), and 256 x 256 tiles are ahead once
// every compute unit has some 48 steps of them (1024 rows summed over 14336:
// 110 against 141; over 4096, 16 steps: 58 against 44).  Several planes go
// through the 64-row tile together (fp32, 512 rows: 196 against 220 by
// turns), until the largest tile takes over (179).  The gradient's 64-row
// tile decodes its weights for half as many rows as the 128-row one, which is
// ahead above 64 rows (128 rows: 29 against 35) unless the sum is short (1000
// x 2048, 1024 rows: 17 against 25).  Experts end in partial tiles, so theirs
// are smaller (128 experts of 256 rows, 768 x 2048: forward 147 with 64 rows,
// 165 with 128, 197 with 256; gradient 244, 192, 220).
inline LinearPlan plan_linear(bool grad, int sf, int x_dt, bool grouped, int64_t R, int64_t N, int64_t K, int E) {
    LinearPlan q{};
    const int64_t C = grad ? N : K, O = grad ? K : N;
    const bool as_is = x_dt == DT_BF16 || (x_dt == DT_F16 && sf == SF_E4M3);     // one 16-bit plane
    q.np = as_is ? 1 : x_dt == DT_F16 ? 2 : 3;
    q.pitch = up(C, 256);
    q.splits = 1;
    const int64_t groups = grouped ? std::min<int64_t>(E, R) : 1, per_group = (R + groups - 1) / groups;
    // (the tiles' scale reads need 8 bytes of scales)
    if (!grad && (per_group <= 16 || E * N * K < 8 * 32)) {
        q.kind = Kind::kSkinny;
        q.copy = !as_is;             // (K is whole 16-byte pieces)
        if (q.copy) q.plane_bytes = round256(q.np * R * q.pitch * 2);
        return q;
    }
    // tiles of a size that run: every group ends in a partial one, half of it empty
    const auto tiles = [&](int64_t bm, int64_t bo) {
        return (R / bm + (grouped ? groups / 2 : R % bm > 0)) * ((O + bo - 1) / bo);
    };
    const int64_t steps = (C + 63) / 64;
    const bool loaded = tiles(256, 256) * steps * q.np >= 256 * 48;
    if (per_group >= (!grouped ? 256 : grad ? 2048 : 768) && loaded) q.kind = Kind::kTile256;
    else if (!grad && per_group <= 32) q.kind = Kind::kTile32;
    else if (per_group <= 64 || q.np > 1) q.kind = Kind::kTile64;
    else if (grad) q.kind = steps <= 16 && tiles(64, 128) <= 512 ? Kind::kTile64 : Kind::kTile128;
    else q.kind = (grouped ? per_group <= 512 : tiles(64, 128) <= 448) ? Kind::kTile64 : Kind::kTile128;
    // the small tiles keep all planes of their rows in a stage, with 32-bit offsets over the planes
    if (q.kind != Kind::kTile256 && q.np > 1 && q.np * R * q.pitch * 2 >= kMaxGatherBytes) q.kind = Kind::kTile128;
    const int bo = q.kind == Kind::kTile256 ? 256 : 128;
    const int bm = q.kind == Kind::kTile32 ? 32 : q.kind == Kind::kTile64 ? 64 : bo;
    const bool turns = q.np > 1 && bm >= 128;      // planes one after the other, in whole groups of 4 steps
    // the tiles take x in whole steps of 64
    q.copy = !as_is || C % 64 != 0;
    if (q.copy) q.plane_bytes = round256(q.np * R * q.pitch * 2);
    q.tiles_m = row_tiles(grouped, R, E, bm);
    q.tiles_o = (O + bo - 1) / bo;
    // Parts of the sum, by a model of the time in ns: the steps of the busiest
    // compute unit (a step of a tile takes about 200, 300, 550 and 1200 ns) and
    // the join (4 us, and its bytes at 4 TB/s).  It was fitted to one plane, one
    // workgroup of a unit at a time.  Planes in one stage make a step longer than it
    // says (17 rows fp32 at 14336 x 4096: 6.4 us predicted for a kernel of 21), and
    // tiles of which two and more share a unit hide each other's latency, so for
    // short products with several planes its choice is not always the best.
    const double step_ns = bm == 32 ? 200 : bm == 64 ? 300 : bm == 128 ? 550 : 1200;
    const int64_t unit = turns ? 4 : 1;
    double best = 0;
    for (int64_t s = 1; s <= 16; ++s) {
        const int64_t part = up((steps + s - 1) / s, unit), n = part ? (steps + part - 1) / part : 1;
        if (n != s || (s > 1 && part < 2)) continue;
        const double ns = (double)((tiles(bm, bo) * s + 255) / 256) * (double)part * (turns ? q.np : 1) * step_ns +
                          (s > 1 ? 4000.0 + (double)s * R * O * 8 / 4000.0 : 0.0);
        if (s == 1 || ns < best) {
            best = ns;
            q.splits = (int)s;
            q.split_steps = (int)part;
        }
    }
    if (q.splits > 1) {
        q.ld_part = up(O, 4);
        q.part_bytes = (size_t)q.splits * R * q.ld_part * 4;
    }
    return q;
}

}  // namespace fp4q_dev
