// linear.hip -- products of FP4 weights with 16- and 32-bit activations:
//   forward   y[m][n]  = g_e sum_k x[m][k] w_e[n][k] + bias_e[n]
//   gradient  dx[m][k] = g_e sum_n dy[m][n] w_e[n][k]
// with w = grid * dec(scale) of packed E2M1 codes, E8M0 scales per 32 or
// E4M3 scales per 16 values along K, one weight matrix or one per expert
// (the W4A16 form of the FP4 products of the MR-GPTQ page, section 2.3, and
// the straight-through use of frozen FP4 weights in training).
#include "linear.hpp"

#include "linear_plan.hpp"
#include "linear_tile.hpp"

namespace fp4q_dev {

// ---------------------------------------------------------------------------
// Few rows: 16 rows of x against 16 NT rows of weights per workgroup, the
// summed dimension K split over its waves.  Bound by the weights' bytes
// (and for one token by latency), so weights go from memory to registers,
// 16 bytes a lane, and are decoded there.
//
// The order of K inside a sum is free, so it is chosen for the loads: of a
// 128-value chunk lane l takes the 32 consecutive values 32 (l / 16) .. + 31
// of weight row l % 16 -- 16 code bytes, one E8M0 or two E4M3 scales -- and
// its four dwords are its parts of four 16 x 16 x 32 products, for which the
// x operand of lane l holds the same values of x row l % 16.  Wave w of W
// takes the chunks w, w + W, ...; the waves' sums meet in LDS and are added in
// wave order.  Dense calls run 8 waves, experts 4: their workgroups begin with
// a chain of dependent reads (offsets, rows, x), which more and smaller ones
// hide better (16 rows of 64 experts at 1536 x 4096 NVFP4: 35 against 41 us;
// dense, one row at 14336 x 4096: 13.4 against 12.7).  Measured, MXFP4 bf16: one
// row at 4096 x 4096 5.9 us in the kernel (8.9 MB at 1.5 TB/s: launch and one
// memory latency), 16 entries of 32 experts at 2048 x 2048 about 13 us (35 MB
// of weights at most, 2.7 TB/s).  Activations that go in as several planes pay
// k_linear_planes' launch before and their products (one row at 4096 x 4096:
// fp16 9.3 us, fp32 10.2; 16 rows 14.7 and 18.8 where one plane takes 8.8).
// ---------------------------------------------------------------------------

// A lane's part of one 128-value chunk: codes, scale codes, activations.
template <int NP, int NT>
struct SkinnyChunk {
    u32x4 w[NT];
    uint32_t s[NT];
    u32x4 x[NP][4];
};

template <int SF, int NP, int NT>
struct Skinny {
    const uint8_t* w[NT];      // this lane's weight rows, at its 32 values of chunk 0
    const uint8_t* s[NT];
    const uint8_t* x;          // its x row, likewise
    int64_t plane_bytes;
    bool live;

    // Chunk c, all 128 values inside K.
    __device__ __forceinline__ void load(int64_t c, SkinnyChunk<NP, NT>& o) const {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            o.w[j] = *(const u32x4_a8*)(w[j] + c * 64);
            if constexpr (SF == WF_E8M0) {
                o.s[j] = s[j][c * 4];
            } else {
                const uint8_t* p = s[j] + c * 8;
                o.s[j] = p[0] | (uint32_t)p[1] << 8;
            }
        }
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                o.x[q][h] = u32x4{0u, 0u, 0u, 0u};
                if (live) o.x[q][h] = *(const u32x4*)(x + q * plane_bytes + c * 256 + 16 * h);
            }
    }

    // The last, partial chunk: left of the lane's 32 values are inside K (a
    // multiple of 16, or none).
    __device__ __forceinline__ void load_tail(int64_t c, int64_t left, SkinnyChunk<NP, NT>& o) const {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            o.w[j] = u32x4{0u, 0u, 0u, 0u};
            o.s[j] = 0u;
            if (left >= 16) {
                const u32x2 lo = *(const u32x2*)(w[j] + c * 64);
                o.w[j][0] = lo[0];
                o.w[j][1] = lo[1];
                o.s[j] = s[j][c * (SF == WF_E8M0 ? 4 : 8)];
            }
            if (left >= 32) {
                const u32x2 hi = *(const u32x2*)(w[j] + c * 64 + 8);
                o.w[j][2] = hi[0];
                o.w[j][3] = hi[1];
                if constexpr (SF != WF_E8M0) o.s[j] |= (uint32_t)s[j][c * 8 + 1] << 8;
            }
        }
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                o.x[q][h] = u32x4{0u, 0u, 0u, 0u};
                if (live && 8 * h < left) o.x[q][h] = *(const u32x4*)(x + q * plane_bytes + c * 256 + 16 * h);
            }
    }

    static __device__ __forceinline__ void multiply(const SkinnyChunk<NP, NT>& o, f32x4 (&acc)[NT]) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            bf16x8 a[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t code = SF == WF_E8M0 ? o.s[j] : (o.s[j] >> (h < 2 ? 0 : 8)) & 0xFFu;
                a[j] = __builtin_bit_cast(bf16x8, decode8<SF>(o.w[j][h], weight_scale<SF>(code)));
            }
#pragma unroll
            for (int q = NP - 1; q >= 0; --q)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[j] = mfma16<SF>(a[j], __builtin_bit_cast(bf16x8, o.x[q][h]), acc[j]);
        }
    }
};

template <int SF, int NP, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES == 4 ? 3 : 2) void k_linear_skinny(LinearArgs p, int64_t plane_bytes,
                                                                                int tiles_n, int first) {
    constexpr int B = kScaleBlock<SF>;
    constexpr int U = NP + NT <= 2 ? 4 : NP + NT <= 5 ? 2 : 1;      // chunks in flight
    __shared__ f32x4 red[WAVES][NT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const unsigned wg = (unsigned)first + blockIdx.x;
    const RowTile rt = row_tile<16>(p, wg / tiles_n);
    if (rt.rows <= 0) return;
    const int64_t n0 = (int64_t)(wg % tiles_n) * (16 * NT);
    const int r = lane & 15, q = lane >> 4;
    f32x4 acc[NT] = {};
    if (rt.e >= 0) {
        const int64_t K = p.K;
        const uint8_t* codes = p.codes + (int64_t)rt.e * p.N * (K / 2);
        const uint8_t* scales = p.scales + (int64_t)rt.e * p.N * (K / B);
        Skinny<SF, NP, NT> sk;
        sk.plane_bytes = plane_bytes;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int64_t n = imin(n0 + 16 * j + r, p.N - 1);
            sk.w[j] = codes + n * (K / 2) + 16 * q;
            sk.s[j] = scales + n * (K / B) + (32 / B) * q;
        }
        sk.live = r < rt.rows;
        sk.x = (const uint8_t*)p.x + (source_row(p, rt.row0 + (sk.live ? r : 0)) * p.ld_x + 32 * q) * 2;
        const int64_t full = K / 128;
        int64_t c = wave;
        for (; c + (U - 1) * WAVES < full; c += U * WAVES) {
            SkinnyChunk<NP, NT> ch[U];
#pragma unroll
            for (int u = 0; u < U; ++u) sk.load(c + u * WAVES, ch[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) sk.multiply(ch[u], acc);
        }
        for (; c < full; c += WAVES) {
            SkinnyChunk<NP, NT> ch;
            sk.load(c, ch);
            sk.multiply(ch, acc);
        }
        if (c == full && full * 128 < K) {
            SkinnyChunk<NP, NT> ch;
            sk.load_tail(full, K - full * 128 - 32 * q, ch);
            sk.multiply(ch, acc);
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) red[wave][j][lane] = acc[j];
    __syncthreads();
    const float g = rt.e >= 0 && p.g ? p.g[rt.e] : 1.0f;
    const float* bias = rt.e >= 0 && p.bias ? p.bias + rt.e * p.N : nullptr;
    for (int f = wave; f < NT; f += WAVES) {
        f32x4 v = red[0][f][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += red[w][f][lane];
        const int64_t n = n0 + 16 * f + 4 * q;
        if (r < rt.rows && n < p.N) store_y4(p.y, p.y_dt, rt.row0 + r, p.ld_y, n, p.N, v * g + bias4(bias, n, p.N));
    }
}

// ---------------------------------------------------------------------------
// Activations as dense 16-bit planes [NP][rows][pitch], zeros from C to the
// pitch: fp16 and fp32 activations as bf16 planes, and 16-bit rows of a length
// that the kernels do not take, copied (DT_BF16; plan_linear).  Gathers where p.rows is set.  One
// lane per 8 values.
// ---------------------------------------------------------------------------
template <int DT>
__global__ __launch_bounds__(256) void k_linear_planes(LinearArgs p, int64_t rows, int64_t C, int64_t pitch,
                                                       uint16_t* out, int64_t first) {
    constexpr int NP = kPlanes<DT>;
    const int64_t per = pitch / 8, i = (first + blockIdx.x) * 256 + threadIdx.x;
    if (i >= rows * per) return;
    const int64_t r = i / per, c = (i - r * per) * 8;
    u32x4 pl[NP];
    planes_of<DT>(load_x8<DT>((const char*)p.x + source_row(p, r) * p.ld_x * (DT == DT_F32 ? 4 : 2), c, C), pl);
#pragma unroll
    for (int q = 0; q < NP; ++q) *(u32x4*)(out + ((int64_t)q * rows + r) * pitch + c) = pl[q];
}

// Sum of the parts of a split product, in their order.  One lane per 4 values.
__global__ __launch_bounds__(256) void k_linear_join(const float* part, int splits, int64_t R, int64_t O,
                                                     int64_t ld_part, void* y, int y_dt, int64_t ld_y,
                                                     int64_t first) {
    const int64_t per = ld_part / 4, i = (first + blockIdx.x) * 256 + threadIdx.x;
    if (i >= R * per) return;
    const int64_t r = i / per, c = (i - r * per) * 4;
    f32x4 v = *(const f32x4*)(part + r * ld_part + c);
    for (int q = 1; q < splits; ++q) v += *(const f32x4*)(part + (q * R + r) * ld_part + c);
    store_y4(y, y_dt, r, ld_y, c, O, v);
}

namespace {

template <int SF, int NP, int NT, int WAVES>
hipError_t launch_skinny_waves(const LinearArgs& p, int64_t plane_bytes, hipStream_t s) {
    const int64_t tn = (p.N + 16 * NT - 1) / (16 * NT);
    const int64_t grid = row_tiles(p.offsets != nullptr, p.R, p.E, 16) * tn;
    if (grid > INT32_MAX) return hipErrorInvalidConfiguration;
    return launch_pieces(grid, 64 * WAVES, [&](int64_t first, unsigned n) {
        hipLaunchKernelGGL((k_linear_skinny<SF, NP, NT, WAVES>), dim3(n), dim3(64 * WAVES), 0, s, p, plane_bytes,
                           (int)tn, (int)first);
    });
}

template <int SF, int NP, int NT>
hipError_t launch_skinny(const LinearArgs& p, int64_t plane_bytes, hipStream_t s) {
    return p.offsets ? launch_skinny_waves<SF, NP, NT, 4>(p, plane_bytes, s)
                     : launch_skinny_waves<SF, NP, NT, 8>(p, plane_bytes, s);
}

template <int SF, int NP>
hipError_t launch_few_rows(const LinearArgs& p, int64_t plane_bytes, hipStream_t s) {
    switch (few_rows_tiles(p.offsets != nullptr, p.R, p.N, p.E)) {
        case 4: return launch_skinny<SF, NP, 4>(p, plane_bytes, s);
        case 2: return launch_skinny<SF, NP, 2>(p, plane_bytes, s);
        default: return launch_skinny<SF, NP, 1>(p, plane_bytes, s);
    }
}

// BIG: x gathered by 64-bit addresses.
template <bool GRAD, int SF, int NP, bool BIG>
hipError_t launch_tiles(const LinearPlan& q, const TileArgs& a, hipStream_t s) {
    const int64_t grid = q.tiles_m * q.tiles_o * q.splits;
    if (grid > INT32_MAX) return hipErrorInvalidConfiguration;
    return launch_pieces(grid, q.kind == Kind::kTile256 ? 512 : 256, [&](int64_t first, unsigned n) {
        TileArgs t = a;
        t.first = (int)first;
        const dim3 g(n);
        // the small tiles take all planes of their rows together; the last argument:
        // workgroups that a compute unit's LDS and registers hold
        constexpr bool PI = NP > 1;
        constexpr int TWO = NP == 3 ? 1 : 2;
        if constexpr (GRAD) {
            if (q.kind == Kind::kTile256)
                hipLaunchKernelGGL((k_linear_grad_tile<SF, NP, false, 4, 2, 2, 4, 1>), g, dim3(512), 0, s, t);
            else if (q.kind == Kind::kTile128)
                hipLaunchKernelGGL((k_linear_grad_tile<SF, NP, false, 2, 2, 2, 2, 2>), g, dim3(256), 0, s, t);
            else
                hipLaunchKernelGGL((k_linear_grad_tile<SF, NP, PI, 2, 1, 1, 4, TWO>), g, dim3(256), 0, s, t);
        } else {
            if (q.kind == Kind::kTile256)
                hipLaunchKernelGGL((k_linear_tile<SF, NP, false, BIG, 4, 2, 2, 4, 1>), g, dim3(512), 0, s, t);
            else if (q.kind == Kind::kTile128)
                hipLaunchKernelGGL((k_linear_tile<SF, NP, false, BIG, 2, 2, 2, 2, 2>), g, dim3(256), 0, s, t);
            else if (q.kind == Kind::kTile64)
                hipLaunchKernelGGL((k_linear_tile<SF, NP, PI, BIG, 2, 1, 1, 4, TWO>), g, dim3(256), 0, s, t);
            else
                hipLaunchKernelGGL((k_linear_tile<SF, NP, PI, BIG, 1, 1, 1, 4, 5 - NP>), g, dim3(256), 0, s, t);
        }
    });
}

template <bool GRAD, int SF, int NP>
hipError_t run_product(const LinearPlan& q, const LinearArgs& p, int64_t plane_bytes, void* workspace,
                       hipStream_t s) {
    if constexpr (!GRAD)
        if (q.kind == Kind::kSkinny) return launch_few_rows<SF, NP>(p, plane_bytes, s);
    TileArgs t{};
    t.a = p;
    t.plane_bytes = plane_bytes;
    t.tiles_m = (int)q.tiles_m;
    t.tiles_o = (int)q.tiles_o;
    t.splits = q.splits;
    t.split_steps = q.split_steps;
    t.part = (float*)((char*)workspace + q.plane_bytes);
    t.ld_part = q.ld_part;
    hipError_t e;
    const bool big = p.rows && far_rows(p.x_rows, p.ld_x);     // x as given (one plane)
    if constexpr (!GRAD && NP == 1) e = big ? launch_tiles<GRAD, SF, NP, true>(q, t, s)
                                            : launch_tiles<GRAD, SF, NP, false>(q, t, s);
    else e = launch_tiles<GRAD, SF, NP, false>(q, t, s);
    if (e != hipSuccess || q.splits == 1) return e;
    return launch_pieces((p.R * (q.ld_part / 4) + 255) / 256, 256, [&](int64_t first, unsigned n) {
        hipLaunchKernelGGL(k_linear_join, dim3(n), dim3(256), 0, s, t.part, q.splits, p.R, GRAD ? p.K : p.N, q.ld_part,
                           p.y, p.y_dt, p.ld_y, first);
    });
}

template <bool GRAD, int SF>
hipError_t run_planes(const LinearPlan& q, const LinearArgs& p, int64_t plane_bytes, void* ws, hipStream_t s) {
    if constexpr (SF == WF_E4M3_F16) {
        return run_product<GRAD, SF, 1>(q, p, plane_bytes, ws, s);
    } else {
        if (q.np == 1) return run_product<GRAD, SF, 1>(q, p, plane_bytes, ws, s);
        if constexpr (SF == WF_E8M0)
            if (q.np == 2) return run_product<GRAD, SF, 2>(q, p, plane_bytes, ws, s);
        return run_product<GRAD, SF, 3>(q, p, plane_bytes, ws, s);
    }
}

}  // namespace

size_t linear_workspace(bool grad, int sf, int x_dt, bool grouped, int64_t R, int64_t N, int64_t K, int E) {
    if (R == 0 || (grad ? K : N) == 0) return 0;
    const LinearPlan q = plan_linear(grad, sf, x_dt, grouped, R, N, K, E);
    return q.plane_bytes + q.part_bytes;
}

hipError_t launch_linear(const LinearArgs& a, bool grad, int sf, int x_dt, void* workspace, hipStream_t s) {
    const LinearPlan q = plan_linear(grad, sf, x_dt, a.offsets != nullptr, a.R, a.N, a.K, a.E);
    LinearArgs p = a;
    int64_t plane_bytes = 0;
    const int64_t C = grad ? a.N : a.K;
    if (q.copy && C > 0) {
        // a copy that the tiles could not gather from is gathered on the way
        const bool gather = a.rows && far_rows(a.x_rows, q.pitch);
        LinearArgs from = a;
        if (!gather) from.rows = nullptr;
        const int64_t rows = gather ? a.R : a.x_rows;
        uint16_t* out = (uint16_t*)workspace;
        const hipError_t e = launch_pieces((rows * (q.pitch / 8) + 255) / 256, 256, [&](int64_t first, unsigned n) {
            const dim3 g(n), b(256);
            if (q.np == 1)
                hipLaunchKernelGGL(k_linear_planes<DT_BF16>, g, b, 0, s, from, rows, C, q.pitch, out, first);
            else if (x_dt == DT_F16)
                hipLaunchKernelGGL(k_linear_planes<DT_F16>, g, b, 0, s, from, rows, C, q.pitch, out, first);
            else
                hipLaunchKernelGGL(k_linear_planes<DT_F32>, g, b, 0, s, from, rows, C, q.pitch, out, first);
        });
        if (e != hipSuccess) return e;
        p.x = out;
        p.ld_x = q.pitch;
        p.x_rows = rows;
        if (gather) p.rows = nullptr;
        plane_bytes = rows * q.pitch * 2;
    }
    const int wf = weight_format(sf, x_dt);
    if (grad) return wf == WF_E8M0   ? run_planes<true, WF_E8M0>(q, p, plane_bytes, workspace, s)
                     : wf == WF_E4M3 ? run_planes<true, WF_E4M3>(q, p, plane_bytes, workspace, s)
                                     : run_planes<true, WF_E4M3_F16>(q, p, plane_bytes, workspace, s);
    return wf == WF_E8M0   ? run_planes<false, WF_E8M0>(q, p, plane_bytes, workspace, s)
           : wf == WF_E4M3 ? run_planes<false, WF_E4M3>(q, p, plane_bytes, workspace, s)
                           : run_planes<false, WF_E4M3_F16>(q, p, plane_bytes, workspace, s);
}

}  // namespace fp4q_dev
