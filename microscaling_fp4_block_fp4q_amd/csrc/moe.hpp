// moe.hpp -- arguments and launchers of moe.hip.
#pragma once

#include "linear_device.hpp"

namespace fp4q_dev {

constexpr int kSortMaxExperts = 1024;
constexpr int kSortThreads = 256;
constexpr int64_t kSortSmall = 8192;         // entries that one workgroup sorts by itself

struct SortArgs {
    const int32_t* ids;        // [R] expert of entry i = t k + j
    int64_t R;
    int E;
    int32_t* offsets;          // [E + 1]
    int32_t* rows;             // [R]
    int32_t* slots;            // [R]
    uint32_t* counts;          // [E + 1][chunks], then the totals [E + 1]
    int64_t chunk;             // entries of a chunk
    int chunks;
    int id_bits;
};

struct CombineArgs {
    const void* h;             // [R, N]
    int64_t ld_h, R;
    const void* dy;            // [T, N] (gradient)
    int64_t ld_dy;
    const int32_t* slots;      // [T, k]
    const int32_t* offsets;    // [E + 1] (gradient)
    const float* weights;      // [T, k] or null (1)
    int64_t T, N;
    int top_k, E;
    void* y;                   // [T, N]
    int y_dt;
    int64_t ld_y;
    void* dh;                  // [R, N]
    int dh_dt;
    int64_t ld_dh;
    float* dweights;           // [T, k] or null
    int64_t first;             // workgroup that this launch begins with
};

// Columns c .. c + 7 of a row as fp32, those at or past N zero.
template <int DT>
__device__ __forceinline__ void load_row8(const void* base, int64_t row, int64_t ld, int64_t c, int64_t N,
                                          float (&v)[8]) {
    const RawX<DT> r = load_x8<DT>((const char*)base + row * ld * (DT == DT_F32 ? 4 : 2), c, N);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DT_F32) {
            v[2 * i] = as_f(r.w[i / 2][2 * (i % 2)]);
            v[2 * i + 1] = as_f(r.w[i / 2][2 * (i % 2) + 1]);
        } else if constexpr (DT == DT_F16) {
            v[2 * i] = f16_bits_to_f32(r.w[0][i] & 0xFFFFu);
            v[2 * i + 1] = f16_bits_to_f32(r.w[0][i] >> 16);
        } else {
            v[2 * i] = as_f(r.w[0][i] << 16);
            v[2 * i + 1] = as_f(r.w[0][i] & 0xFFFF0000u);
        }
    }
}

size_t sort_workspace(int64_t R, int E);
hipError_t launch_sort(const SortArgs& a, hipStream_t s);
hipError_t launch_combine(const CombineArgs& p, int dt, hipStream_t s);
hipError_t launch_combine_grad(const CombineArgs& p, int dt, hipStream_t s);

}  // namespace fp4q_dev
