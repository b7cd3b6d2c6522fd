// linear_device.hpp -- building blocks of the products of FP4 weights with
// 16- and 32-bit activations (linear.hip).
//
// Number formats on the matrix cores.  A weight without its per-tensor
// scale, grid * dec(scale), has at most 2 + 4 significant bits, and its
// exponent is inside bf16's range unless it reaches 2^128: 4 and 6 at E8M0
// code 253 (2^126), 2, 3, 4 and 6 at code 254 (2^127), which are infinities,
// as in fp32.  bf16 holds every other one exactly (the scaled convert and the
// matrix cores keep bf16 subnormals; both were checked for every code and
// scale).
//
// Activations go in as bf16 planes whose sum is the activation: bf16 is one
// plane, fp16 (11 significant bits) two, fp32 (24) three, each plane the next
// 8 bits, truncated.  Every product of a plane and a weight is then exact in
// fp32, and the fp32 accumulation is the only rounding before the result's.
// (With several planes an infinite weight also meets planes that are zero: the
// sum is then NaN where the definition has an infinity.)  An E4M3-scaled
// weight (2^-10 .. 2688) is exact in fp16 too, so fp16 activations with it run
// on the fp16 matrix cores as they are (WF_E4M3_F16): half the products of two
// planes.  E8M0 scales leave fp16's range.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "fp4q_device.hpp"

namespace fp4q_dev {

// Scale format and operand type of the weights.
enum : int { WF_E8M0 = 0, WF_E4M3 = 1, WF_E4M3_F16 = 2 };

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));      // also holds fp16 operands, as bits
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Rows of codes start on 8 bytes when K is an odd multiple of 16; the
// 16-byte global loads of gfx950 need only dword alignment.
typedef uint32_t u32x4_a8 __attribute__((ext_vector_type(4), aligned(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));
typedef uint64_t u64_a1 __attribute__((aligned(1)));

// (HIP's min and max on 64-bit integers go through doubles.)
__device__ __forceinline__ int64_t imin(int64_t a, int64_t b) { return a < b ? a : b; }
__device__ __forceinline__ int64_t imax(int64_t a, int64_t b) { return a > b ? a : b; }

// A load from global memory through a pointer whose address space the
// compiler cannot prove (a selected address): a generic load would count as
// an LDS access too.
template <class T>
__device__ __forceinline__ T load_global(const void* p) {
    return *(const __attribute__((address_space(1))) T*)p;
}

// Work of any number of workgroups, launched in pieces: launch(first, n)
// starts workgroups first .. first + n - 1.  HIP counts the threads of a launch
// in 32 bits, so grids of 2^24 workgroups of 256 have to be cut.  A piece here
// has 2^28 threads at most, which run for a millisecond and more, next to
// which one more launch is nothing.
template <class Launch>
hipError_t launch_pieces(int64_t workgroups, int threads, Launch launch) {
    const int64_t most = ((int64_t)1 << 28) / threads;
    for (int64_t first = 0; first < workgroups; first += most) {
        launch(first, (unsigned)std::min(most, workgroups - first));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// One product: rows of x in groups (experts), each group with its own
// weights.  Dense calls have one group and no offsets.
struct LinearArgs {
    const void* x;             // [*, C] activations or output gradients, C the summed dimension
    int64_t ld_x;
    int64_t x_rows;            // rows of x (bounds of the gather)
    const int32_t* rows;       // sorted row r reads x row rows[r] / top_k; null: row r
    int top_k;
    const uint8_t* codes;      // [E, N, K / 2]
    const uint8_t* scales;     // [E, N, K / B]
    const float* g;            // [E] or null
    const float* bias;         // [E, N] or null
    const int32_t* offsets;    // [E + 1] or null (dense)
    int E;
    int64_t R;                 // rows of y
    int64_t N, K;
    void* y;
    int y_dt;
    int64_t ld_y;
};

// A row tile: rows row0 .. row0 + rows - 1 of group e; e < 0: rows that
// belong to no group and are written as zeros; rows <= 0: nothing to do.
struct RowTile {
    int e;
    int rows;
    int64_t row0;
};

// Row tile t of a launch, BM rows each: the groups' tiles in order, then
// those of the rows past the last group.  Offsets are clamped to [0, R], so
// no table makes a kernel leave its buffers.  Every lane of every wave calls
// it; the result is uniform.
template <int BM>
__device__ __forceinline__ RowTile row_tile(const LinearArgs& p, int64_t t) {
    RowTile o;
    if (!p.offsets) {
        o.e = 0;
        o.row0 = t * BM;
        o.rows = (int)imin(BM, p.R - o.row0);
        return o;
    }
    const int lane = threadIdx.x & 63;
    const int R = (int)p.R;
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < p.E) {
            lo = min(max(p.offsets[e], 0), R);
            hi = min(max(p.offsets[e + 1], lo), R);
        }
        const int n = (int)(((uint32_t)(hi - lo) + (BM - 1)) / BM);     // hi - lo may be 2^31 - 1
        int incl = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(incl, d);
            incl += lane >= d ? v : 0;
        }
        const int before = base + incl - n;
        const uint64_t hit = __ballot(t >= before && t < before + n);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int flo = __builtin_amdgcn_readlane(lo, src), fhi = __builtin_amdgcn_readlane(hi, src);
            const int first = flo + ((int)t - __builtin_amdgcn_readlane(before, src)) * BM;
            o.e = e0 + src;
            o.row0 = first;
            o.rows = min(BM, fhi - first);
            return o;
        }
        base += __builtin_amdgcn_readlane(incl, 63);
    }
    o.e = -1;
    o.row0 = (int64_t)min(max(p.offsets[p.E], 0), R) + (t - base) * BM;
    o.rows = (int)imax(imin(BM, R - o.row0), 0);
    return o;
}

// Row tiles that a launch needs at most: every group may end in a partial
// tile, and so may the rows past them.
inline int64_t row_tiles(bool grouped, int64_t R, int E, int BM) {
    if (!grouped) return (R + BM - 1) / BM;
    return R / BM + (E < R ? E : R) + 1;
}

// x row that row r of y is computed from.
__device__ __forceinline__ int64_t source_row(const LinearArgs& p, int64_t r) {
    if (!p.rows) return r;
    const int64_t t = (uint32_t)max(p.rows[r], 0) / (uint32_t)p.top_k;
    return imin(t, p.x_rows - 1);
}

// ---------------------------------------------------------------------------
// weights
// ---------------------------------------------------------------------------

// Block scale as the factor of decode8: for E8M0 the power of two itself
// (code 0 is 2^-127, an fp32 subnormal; 0xFF NaN), for E4M3 its value.
template <int SF>
__device__ __forceinline__ float weight_scale(uint32_t code) {
    if constexpr (SF == WF_E8M0) {
        const uint32_t b = code == 0u ? 0x00400000u : code << 23;
        return as_f(code == kE8M0NaN ? kQNaN : b);
    } else {
        return __builtin_amdgcn_cvt_f32_fp8((int)(code & 0x7Fu), 0);   // OCP E4M3; 0x7F is NaN
    }
}

// Two codes (byte B of w) times the scale, as a pair of operands.  E8M0: the
// scaled convert is exact.  E4M3: the convert applies only a scale's
// exponent, so the grid values are multiplied in fp32; the product has at
// most 6 significant bits, so its upper 16 bits are the bf16 value, and its
// conversion to fp16 is exact.
template <int SF, int B>
__device__ __forceinline__ uint32_t decode2(uint32_t w, float s) {
    if constexpr (SF == WF_E8M0) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, B));
    } else {
        const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, B);
        if constexpr (SF == WF_E4M3_F16)
            return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(v[0] * s, v[1] * s));
        return __builtin_amdgcn_perm(as_u(v[1] * s), as_u(v[0] * s), 0x07060302u);
    }
}

// Eight codes (one dword) as an operand.
template <int SF>
__device__ __forceinline__ u32x4 decode8(uint32_t w, float s) {
    return u32x4{decode2<SF, 0>(w, s), decode2<SF, 1>(w, s), decode2<SF, 2>(w, s), decode2<SF, 3>(w, s)};
}

template <int SF>
constexpr int kScaleBlock = SF == WF_E8M0 ? 32 : 16;

// acc += weights (first operand) times activations.
template <int SF>
__device__ __forceinline__ f32x16 mfma32(bf16x8 w, bf16x8 x, f32x16 acc) {
    if constexpr (SF == WF_E4M3_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), acc,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, x, acc, 0, 0, 0);
}
template <int SF>
__device__ __forceinline__ f32x4 mfma16(bf16x8 w, bf16x8 x, f32x4 acc) {
    if constexpr (SF == WF_E4M3_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), acc,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, acc, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------

template <int DT>
constexpr int kPlanes = DT == DT_BF16 ? 1 : DT == DT_F16 ? 2 : 3;

__device__ __forceinline__ uint32_t pack_hi16(float lo, float hi) {
    return __builtin_amdgcn_perm(as_u(hi), as_u(lo), 0x07060302u);
}

// The next plane of v (its upper 16 bits) and what is left of v.  A value
// that is not finite is one plane (NaN made quiet, so truncation keeps it).
__device__ __forceinline__ float next_plane(float& v) {
    const bool finite = __builtin_fabsf(v) < __builtin_inff();
    const float hi = v != v ? as_f(kQNaN) : as_f(as_u(v) & 0xFFFF0000u);
    v = finite ? v - hi : 0.0f;
    return hi;
}

// Eight consecutive activations from 16-byte-aligned memory as raw words:
// 4 (bf16, fp16) or 8 (fp32).
template <int DT>
struct RawX {
    u32x4 w[DT == DT_F32 ? 2 : 1];
};

// Values c .. c + 7 of a row of C values; those at or past C are zeros and
// are not read.  c is a multiple of 8.
template <int DT>
__device__ __forceinline__ RawX<DT> load_x8(const void* row, int64_t c, int64_t C) {
    constexpr int es = DT == DT_F32 ? 4 : 2;
    RawX<DT> r;
    const char* p = (const char*)row + c * es;
    if (c + 8 <= C) {
        r.w[0] = *(const u32x4*)p;
        if constexpr (DT == DT_F32) r.w[1] = *(const u32x4*)(p + 16);
    } else {
        uint32_t v[8] = {};
        for (int i = 0; i < 8; ++i)
            if (c + i < C) v[i] = DT == DT_F32 ? ((const uint32_t*)p)[i] : ((const uint16_t*)p)[i];
        if constexpr (DT == DT_F32) {
            r.w[0] = u32x4{v[0], v[1], v[2], v[3]};
            r.w[1] = u32x4{v[4], v[5], v[6], v[7]};
        } else {
            r.w[0] = u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
        }
    }
    return r;
}

// The bf16 planes of eight activations.
template <int DT>
__device__ __forceinline__ void planes_of(const RawX<DT>& r, u32x4 (&out)[kPlanes<DT>]) {
    if constexpr (DT == DT_BF16) {
        out[0] = r.w[0];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            if constexpr (DT == DT_F16) {
                a = f16_bits_to_f32(r.w[0][i] & 0xFFFFu);
                b = f16_bits_to_f32(r.w[0][i] >> 16);
            } else {
                a = as_f(r.w[i / 2][2 * (i % 2)]);
                b = as_f(r.w[i / 2][2 * (i % 2) + 1]);
            }
#pragma unroll
            for (int q = 0; q < kPlanes<DT>; ++q) {
                const float ha = next_plane(a), hb = next_plane(b);
                out[q][i] = pack_hi16(ha, hb);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// results
// ---------------------------------------------------------------------------

// Four consecutive results y[row][c .. c + 3] (c a multiple of 4, row
// starts on 16 bytes), those at or past C left out.
__device__ __forceinline__ void store_y4(void* y, int dt, int64_t row, int64_t ld, int64_t c, int64_t C, f32x4 v) {
    const int64_t at = row * ld + c;
    if (c + 4 <= C) {
        if (dt == DT_F32) {
            *(f32x4*)((float*)y + at) = v;
        } else {
            u32x2 w;
            w[0] = dt == DT_BF16 ? pack_bf16x2(v[0], v[1]) : pack_f16x2(v[0], v[1]);
            w[1] = dt == DT_BF16 ? pack_bf16x2(v[2], v[3]) : pack_f16x2(v[2], v[3]);
            *(u32x2*)((uint16_t*)y + at) = w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (c + i >= C) break;
        if (dt == DT_F32) ((float*)y)[at + i] = v[i];
        else ((uint16_t*)y)[at + i] = (uint16_t)(dt == DT_BF16 ? pack_bf16x2(v[i], 0.0f) : pack_f16x2(v[i], 0.0f));
    }
}

__device__ __forceinline__ f32x4 bias4(const float* bias, int64_t c, int64_t C) {
    f32x4 b = {0.0f, 0.0f, 0.0f, 0.0f};
    if (bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < C) b[i] = bias[c + i];
    }
    return b;
}

}  // namespace fp4q_dev
