// linear_tile.hpp -- matrix-core tiles of the products with FP4 weights, for
// many rows (forward) and for the gradient.
//
// One workgroup computes BM rows by BO outputs; its WM x WO waves hold
// 32 MF x 32 OF pieces of it as 32 x 32 x 16 bf16 products.  The weight
// fragment is the first operand, so a lane ends up with one row of y and
// groups of four consecutive outputs.  The summed dimension advances 64 per
// step.
//
// Activations: a step's BM x 64 bf16 (128 bytes a row) go from memory
// straight into LDS, 8 rows per load of a wave, gathered rows included (the
// addresses are per lane).  Row r's eight 16-byte chunks sit at slot
// c ^ (r / 2 % 8), which makes the fragment reads conflict-free (16 lanes at
// a time, two rows per 64 banks).
//
// Forward weights stay 4-bit codes until a wave uses them: the order inside
// the sum is free, so lane l takes the 32 consecutive values 32 (l / 32) ..
// + 31 of its row's step -- 16 code bytes and one E8M0 or two E4M3 scales --
// and its four dwords are decoded into its parts of four products, for which
// the x fragments are read in the same order.
//
// Gradient weights are summed over rows of the code matrix, which are
// contiguous along the outputs, so they are transposed: each thread decodes
// 32 consecutive values of one row into LDS (row-major bf16), and the
// transposing LDS read (ds_read_b64_tr_b16: 4 rows x 16 columns per 16
// lanes) returns the fragments.  A thread's four 16-byte pieces go to four
// separate column blocks, so the lanes of a row write contiguously; columns
// are thereby permuted in groups of 8, which the epilogue undoes.  Rows are
// stored with their 16-byte chunks XOR-permuted by the row (tile_w_swizzle),
// which spreads the four rows of a transposing read, and the lanes of a
// write, over all banks.
//
// Schedule.  A step is four substeps of 16 summed values; the fragments of a
// substep are read (and weights decoded) while the products of the one
// before run.  The barrier stands before the last substep: there every wave
// has read its fragments of this step, so the step's stage can be refilled,
// and the next step's stage is complete, so its first fragments are read
// while the last products run.  Loads run ahead by three (forward) or two
// (gradient) steps of activations.
//
// Measured (a call, with its launches, over several runs): forward, 8192 x
// 14336 x 4096, MXFP4 bf16, 256 x 256 tiles 0.70-0.74 ms, 1.30-1.37 PFLOP/s;
// matrix cores busy 0.71 of the cycles at 1.65 GHz, which is the card's power
// limit (a library bf16 product of that shape, busy 0.89, falls to 1.48 GHz
// and takes 0.72-0.75 ms in the same run).  NVFP4 over 8 experts 0.98-1.04 ms
// for 8192 rows: one tile in nine is padding, and decoding costs 4
// instructions a pair of weights against one, done by both wave rows (matrix
// cores busy 0.64, VALU 0.46).  Gradient, 4096 x 4096 x 14336 NVFP4, 0.44-0.47
// ms, 1.03-1.10 PFLOP/s: 896 tiles are 3.5 rounds of the 256 compute units and
// take the time of four; inside a tile nothing is full (matrix cores busy
// 0.55, VALU 0.23, LDS 0.29, of it conflicts 0.01): its waves stand in line to
// issue for half of their time and wait at barriers and for loads for a
// quarter.
#pragma once

#include "linear_device.hpp"

namespace fp4q_dev {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;
typedef const __attribute__((address_space(1))) void* global_ptr;

// What weight loads past the matrix read.
static __device__ __attribute__((aligned(64))) const uint32_t kZeros[16] = {};

// Wait until at most N of this wave's vector-memory loads are outstanding and
// its LDS accesses are done, then a workgroup barrier; the empty asm
// statements keep the compiler from moving memory accesses across it.
template <int N>
__device__ __forceinline__ void tile_wait_barrier() {
    static_assert(N < 64, "vmcnt field");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0x0 << 8));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A uniform value in a scalar register.  The builtin is folded away where the
// compiler sees that the value is uniform, which leaves it in a vector
// register and puts a loop around every buffer load that uses it.  The first
// nop is the wait of a lane read on a vector register that the VALU wrote, the
// last that of a vector memory access on a scalar that the VALU wrote (the
// compiler sees neither inside the asm).
__device__ __forceinline__ uint32_t to_scalar(uint32_t v) {
    uint32_t s;
    asm("s_nop 3\n\tv_readfirstlane_b32 %0, %1\n\ts_nop 4" : "=s"(s) : "v"(v));
    return s;
}

struct TileArgs {
    LinearArgs a;              // a.x: bf16 [T, ld_x] per plane
    int64_t plane_bytes;       // distance of the planes
    int tiles_m, tiles_o;
    int splits;                // parts of the summed dimension
    int split_steps;           // steps of a part
    float* part;               // [splits][R][ld_part] partial sums (splits > 1)
    int64_t ld_part;
    int first;                 // workgroup that this launch begins with
};

// The tile of workgroup id b (one part of the sum): consecutive ids go
// round-robin to the 8 XCDs, so XCD x gets a run of consecutive tiles;
// tiles are numbered in groups of 8 row tiles, so the workgroups of one XCD
// share x rows and weights in its L2.
__device__ __forceinline__ void tile_of(const TileArgs& p, int b, int& tm, int& to) {
    const int n = p.tiles_m * p.tiles_o, x = b % 8, q = n / 8, r = n % 8;
    const int t = x * q + min(x, r) + b / 8;
    constexpr int G = 8;
    const int in_group = G * p.tiles_o, first = t / in_group * G, size = min(G, p.tiles_m - first);
    tm = first + t % in_group % size;
    to = t % in_group / size;
}

// Rows of the activations as this lane's direct loads take them: load q of
// wave w fills rows 8 (L w + q) .. + 7 of the stage.  Buffer loads: the
// compiler counts them like the weights' loads (a global load to LDS it takes
// for an access that may go either way, and waits for everything).  Offsets
// are 32 bits: from the tile's first row (its 256 rows of at most 2^22 values
// are below 2 GiB), or for gathered rows from x.  BIG: x gathered from 4 GiB
// and more, by 64-bit addresses and global loads.  The summed dimension of x
// is a multiple of 64 here (copied with zeros at the end otherwise), so no
// load needs a check.  PI: a stage holds all planes of the tile's BM rows, one
// plane after the other (small tiles: the weights are then decoded once for
// all planes); otherwise the planes take turns.
template <int NP, bool PI, int BM, int W, bool BIG>
struct TileX {
    static constexpr int ROWS = PI ? BM * NP : BM;      // of a stage
    static constexpr int LOADS = ROWS / 8 / W;
    uint64_t base;             // uniform: where the offsets count from, and the bytes behind it
    uint32_t bytes;
    int64_t plane_bytes;
    uint32_t at[LOADS];
    const uint8_t* row[BIG ? LOADS : 1];

    __device__ __forceinline__ void init(const TileArgs& p, const RowTile& rt, int wave, int lane) {
        const int64_t first = p.a.rows ? 0 : rt.row0, pitch = p.a.ld_x * 2;
        const uint8_t* from = (const uint8_t*)p.a.x + first * pitch;
        const uint64_t u = (uint64_t)from;
        base = (uint64_t)to_scalar((uint32_t)(u >> 32)) << 32 | to_scalar((uint32_t)u);
        const int64_t behind = (p.a.x_rows - first) * pitch + (PI ? (NP - 1) * p.plane_bytes : 0);
        bytes = to_scalar((uint32_t)imin(behind, 0xFFFFFFF0ll));
        plane_bytes = p.plane_bytes;
#pragma unroll
        for (int q = 0; q < LOADS; ++q) {
            const int r = 8 * (LOADS * wave + q) + (lane >> 3);
            const int64_t off = (source_row(p.a, rt.row0 + min(r % BM, rt.rows - 1)) - first) * pitch +
                                r / BM * p.plane_bytes + 16 * ((lane & 7) ^ ((r >> 1) & 7));
            if constexpr (BIG) row[q] = from + off;
            else at[q] = (uint32_t)off;
        }
    }

    __device__ __forceinline__ void load(uint8_t* stage, int step, int plane, int wave) const {
#ifdef __HIP_DEVICE_COMPILE__      // the host pass cannot check these builtins in a template
        const uint32_t k = (uint32_t)step * 128u;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(base + (NP == 1 || PI ? 0 : plane * plane_bytes)), (short)0, (int)bytes, 0x00020000);
#pragma unroll
        for (int q = 0; q < LOADS; ++q) {
            uint8_t* to = stage + (LOADS * wave + q) * 1024;
            if constexpr (BIG) __builtin_amdgcn_global_load_lds((global_ptr)(row[q] + k), (lds_ptr)to, 16, 0, 0);
            else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)to, 16, at[q], k, 0, 0);
        }
        asm volatile("" ::: "memory");     // groups of loads stay in their order: the waits count them
#endif
    }
};

// Fragment of rows r0 + l % 32, chunk c, of an activation stage.
__device__ __forceinline__ bf16x8 tile_x_frag(const uint8_t* stage, int r0, int c, int lane) {
    const int r = lane & 31;
    return *(const bf16x8*)(stage + (r0 + r) * 128 + 16 * (c ^ ((r >> 1) & 7)));
}

// Column of y at LDS column c of a gradient tile of BO columns (see above).
template <int BO>
__device__ __forceinline__ int tile_out_column(int c) {
    constexpr int NB = BO / 32;
    const int group = c >> 3;
    return 32 * (group % NB) + 8 * (group / NB) + (c & 7);
}

// Store a wave's 32 MF x 32 OF piece (rows m0.. of the tile, columns c0..)
// through its own LDS region, 32 rows at a time, as 16-byte pieces of rows.
template <class T, bool GRAD, int MF, int OF, int BO>
__device__ __forceinline__ void tile_store(const f32x16 (&acc)[MF][OF], uint8_t* buf, T* y, int dt, int64_t ld,
                                           int64_t row0, int rows, int m0, int64_t o0, int c0, int64_t O,
                                           const float* bias, float g, int lane) {
    constexpr int kVals = 16 / sizeof(T), kChunks = 32 * OF / kVals, kRowBytes = 32 * OF * sizeof(T);
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
#pragma unroll
        for (int j = 0; j < OF; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = 32 * j + 8 * q + 4 * h, chunk = col / kVals;
                f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                v = v * g;
                if constexpr (!GRAD) v = v + bias4(bias, o0 + c0 + col, O);
                uint8_t* at = buf + r * kRowBytes + 16 * (chunk ^ (r % kChunks)) + col % kVals * (int)sizeof(T);
                if constexpr (sizeof(T) == 4) {
                    *(f32x4*)at = v;
                } else {
                    *(u32x2*)at = dt == DT_BF16 ? u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}
                                                : u32x2{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
                }
            }
        asm volatile("" ::: "memory");
        constexpr int kRows = 64 / kChunks;            // rows of one pass
#pragma unroll
        for (int pass = 0; pass < 32 / kRows; ++pass) {
            const int row = kRows * pass + lane / kChunks, chunk = lane % kChunks;
            const u32x4 v = *(const u32x4*)(buf + row * kRowBytes + 16 * (chunk ^ (row % kChunks)));
            const int m = m0 + 32 * i + row, c = c0 + chunk * kVals;
            const int64_t col = o0 + (GRAD ? tile_out_column<BO>(c) : c);
            if (m < rows) {
                T* at = y + (row0 + m) * ld + col;
                if (col + kVals <= O) {
                    *(u32x4*)at = v;
                } else {
#pragma unroll
                    for (int e = 0; e < kVals; ++e) {
                        if (col + e < O)
                            at[e] = sizeof(T) == 4 ? (T)v[e] : (T)(v[e / 2 % 4] >> (16 * (e % 2)));
                    }
                }
            }
        }
        asm volatile("" ::: "memory");
    }
}

template <bool GRAD, int MF, int OF, int BO>
__device__ __forceinline__ void tile_finish(const TileArgs& p, const RowTile& rt, const f32x16 (&acc)[MF][OF],
                                            uint8_t* buf, int m0, int64_t o0, int c0, int split, int lane) {
    const int64_t O = GRAD ? p.a.K : p.a.N;
    const float g = rt.e >= 0 && p.a.g ? p.a.g[rt.e] : 1.0f;
    const float* bias = rt.e >= 0 && p.a.bias && split == 0 ? p.a.bias + rt.e * p.a.N : nullptr;
    if (p.splits > 1)
        tile_store<uint32_t, GRAD, MF, OF, BO>(acc, buf, (uint32_t*)p.part + split * p.a.R * p.ld_part, DT_F32,
                                               p.ld_part, rt.row0, rt.rows, m0, o0, c0, O, bias, g, lane);
    else if (p.a.y_dt == DT_F32)
        tile_store<uint32_t, GRAD, MF, OF, BO>(acc, buf, (uint32_t*)p.a.y, DT_F32, p.a.ld_y, rt.row0, rt.rows, m0, o0,
                                               c0, O, bias, g, lane);
    else
        tile_store<uint16_t, GRAD, MF, OF, BO>(acc, buf, (uint16_t*)p.a.y, p.a.y_dt, p.a.ld_y, rt.row0, rt.rows, m0,
                                               o0, c0, O, bias, g, lane);
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// Weights of a tile: codes of two steps at a time (64 bytes a row) by direct
// loads into LDS, 16 rows per load of a wave, row r's four 16-byte chunks at
// slot c ^ (r / 4 % 4) (conflict-free reads); scales of four steps at a time
// (8 or 16 bytes a row) into registers.  Loaded by the step straight into
// registers, codes and scales touch a cache line per row and step for 32 and
// 2 bytes of it, and the L2's request rate bounds the kernel.
//
// Past K: x is zero there, so the codes need only be finite (any code is) and
// the scales are set to code 0.  Codes past the array's end are not read: the
// buffer's bound holds them back, for steps that begin inside K (the bound is
// compared with the offset less the step's, which has to stay below it); the
// last scale reads of the array are moved back inside it and shifted.
template <int SF, int OF, int BO, int W>
struct TileWeights {
    static constexpr int B = kScaleBlock<SF>;
    static constexpr int LOADS = BO / 16 / W;
    static constexpr int Q = SF == WF_E8M0 ? 1 : 2;     // 8-byte pieces of four steps' scales
    uint64_t base;             // uniform: codes of the tile's first row, and the bytes behind it
    uint32_t bytes;
    uint32_t at[LOADS];
    const uint8_t* s[OF];      // scales of this lane's rows
    int64_t room[OF];          // bytes from there to the end of the array
    int K, h;                  // h: lane / 32

    __device__ __forceinline__ void init(const LinearArgs& a, int e, int64_t o0, int c0, int wave, int lane) {
        K = (int)a.K;
        h = lane >> 5;
        const int64_t pitch = a.K / 2, first = (int64_t)e * a.N + o0, end = (int64_t)a.E * a.N;
        const uint64_t u = (uint64_t)(a.codes + first * pitch);
        base = (uint64_t)to_scalar((uint32_t)(u >> 32)) << 32 | to_scalar((uint32_t)u);
        bytes = to_scalar((uint32_t)imin((end - first) * pitch, 0xFFFFFFF0ll));
        const int last = (int)imin(a.N - 1 - o0, BO - 1);        // rows past N read the last one
#pragma unroll
        for (int q = 0; q < LOADS; ++q) {
            const int r = 16 * (LOADS * wave + q) + (lane >> 2);
            at[q] = (uint32_t)(min(r, last) * pitch + 16 * ((lane & 3) ^ ((r >> 2) & 3)));
        }
#pragma unroll
        for (int j = 0; j < OF; ++j) {
            const int64_t row = first + min(c0 + 32 * j + (lane & 31), last);
            s[j] = a.scales + row * (a.K / B);
            room[j] = (end - row) * (a.K / B);
        }
    }

    // Codes of steps k and k + 1.
    __device__ __forceinline__ void load(uint8_t* stage, int k, int wave) const {
#ifdef __HIP_DEVICE_COMPILE__
        const __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)bytes, 0x00020000);
#pragma unroll
        for (int q = 0; q < LOADS; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(stage + (LOADS * wave + q) * 1024), 16, at[q],
                                                     (uint32_t)k * 32u, 0, 0);
        asm volatile("" ::: "memory");     // as above
#endif
    }

    // Scales of steps k .. k + 3, as loaded and as they are.
    __device__ __forceinline__ void load_scales(int k, uint64_t (&v)[OF][Q]) const {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int j = 0; j < OF; ++j)
#pragma unroll
            for (int q = 0; q < Q; ++q)
                v[j][q] = load_global<u64_a1>(s[j] + imin((int64_t)k * (64 / B) + 8 * q, room[j] - 8));
        asm volatile("" ::: "memory");
    }
    __device__ __forceinline__ void settle_scales(int k, uint64_t (&v)[OF][Q]) const {
#pragma unroll
        for (int j = 0; j < OF; ++j)
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                // the compiler may not work on them any earlier: it would wait for their loads
                asm volatile("" : "+v"(v[j][q]));
                const int64_t over = (int64_t)k * (64 / B) + 8 * q - (room[j] - 8);
                if (over > 0) v[j][q] = over < 8 ? v[j][q] >> (8 * over) : 0ull;
            }
    }

    // Scale codes of step k = 4 n + i for the lane's two 16-value halves.
    __device__ __forceinline__ void codes_of(const uint64_t (&v)[Q], int i, int k, uint32_t& s0, uint32_t& s1) const {
        if constexpr (SF == WF_E8M0) {
            s0 = s1 = (uint32_t)(v[0] >> (16 * i)) >> (8 * h) & 0xFFu;
        } else {
            const uint32_t w = (uint32_t)(v[i / 2] >> (32 * (i % 2))) >> (16 * h);
            s0 = w & 0x7Fu;
            s1 = w >> 8 & 0x7Fu;
        }
        if (k * 64 + 64 > K) {
            const int left = K - k * 64 - 32 * h;
            if (left <= 0) s0 = 0u;
            if (left <= 16) s1 = 0u;
        }
    }
};

template <int OF>
struct TileW {
    u32x4 c[OF];               // a lane's 32 codes of a step, per fragment
    float s[OF][2];            // scales of their halves
};

// Codes of a step: parity p of the two of the stage.
template <int OF>
__device__ __forceinline__ void tile_codes(TileW<OF>& w, const uint8_t* stage, int p, int c0, int lane) {
#pragma unroll
    for (int j = 0; j < OF; ++j) {
        const int r = c0 + 32 * j + (lane & 31);
        w.c[j] = *(const u32x4*)(stage + r * 64 + 16 * ((2 * p + (lane >> 5)) ^ ((r >> 2) & 3)));
    }
}

// Operands of one substep; P planes.
template <int P, int MF, int OF>
struct TileOps {
    bf16x8 x[P][MF], w[OF];
};

template <int SF, int P, int MF, int OF>
__device__ __forceinline__ void tile_products(const TileOps<P, MF, OF>& o, f32x16 (&acc)[MF][OF]) {
#pragma unroll
    for (int q = P - 1; q >= 0; --q)
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < OF; ++j)
                acc[i][j] = mfma32<SF>(o.w[j], o.x[q][i], acc[i][j]);
}

// The x operands of a substep: chunk c of the tile's rows from m0 on.
template <int BM, int P, int MF, int OF>
__device__ __forceinline__ void tile_x_operands(TileOps<P, MF, OF>& o, const uint8_t* stage, int c, int m0,
                                                int lane) {
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int i = 0; i < MF; ++i) o.x[q][i] = tile_x_frag(stage, q * BM + m0 + 32 * i, c, lane);
}

// Issue order of a substep: after each product an LDS read (of READS) and
// VALU decode instructions.
template <int PRODUCTS, int READS, int VALU>
__device__ __forceinline__ void tile_interleave() {
#pragma unroll
    for (int k = 0; k < PRODUCTS; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                  // MFMA
        if (k < READS) __builtin_amdgcn_sched_group_barrier(0x100, (READS + PRODUCTS - 1) / PRODUCTS, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    }
}

// Operands of substep q: x from the stage, w decoded from the lane's codes.
template <int SF, int BM, int P, int MF, int OF>
__device__ __forceinline__ void tile_operands(TileOps<P, MF, OF>& o, const uint8_t* stage, const TileW<OF>& w, int q,
                                              int m0, int lane) {
    tile_x_operands<BM>(o, stage, (lane >> 5) * 4 + q, m0, lane);
#pragma unroll
    for (int j = 0; j < OF; ++j)
        o.w[j] = __builtin_bit_cast(bf16x8, decode8<SF>(w.c[j][q], w.s[j][q / 2]));
}

template <int SF, int NP, bool PI, bool BIG, int MF, int OF, int WM, int WO, int PER_CU>
__global__ __launch_bounds__(64 * WM * WO, PER_CU * WM * WO / 4) void k_linear_tile(TileArgs p) {
    constexpr int BM = 32 * MF * WM, BO = 32 * OF * WO, W = WM * WO, P = PI ? NP : 1, TURNS = NP / P;
    using TX = TileX<NP, PI, BM, W, BIG>;
    constexpr int LOADS = TX::LOADS, READS = P * MF;
    using WT = TileWeights<SF, OF, BO, W>;
    __shared__ __attribute__((aligned(1024))) uint8_t st0[TX::ROWS * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[TX::ROWS * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t st2[TX::ROWS * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t st3[TX::ROWS * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t wa[BO * 64];
    __shared__ __attribute__((aligned(1024))) uint8_t wb[BO * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = 32 * MF * (wave / WO), c0 = 32 * OF * (wave % WO);
    const uint32_t wg = (uint32_t)p.first + blockIdx.x;
    const int tiles = p.tiles_m * p.tiles_o, split = wg / tiles;
    int tm, to;
    tile_of(p, wg % tiles, tm, to);
    const RowTile rt = row_tile<BM>(p.a, tm);
    if (rt.rows <= 0) return;
    const int64_t o0 = (int64_t)to * BO;
    f32x16 acc[MF][OF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < OF; ++j) acc[i][j] = f32x16{};
    // Steps k0 .. k0 + len - 1 of each plane in turn (with several turns len is
    // a multiple of 4, so that the weights' stages and scales start afresh).
    const int k0 = split * p.split_steps;
    const int len = min(TURNS == 1 ? (int)((p.a.K + 63) / 64) : (int)((p.a.K + 255) / 256 * 4), k0 + p.split_steps) - k0;
    const int ns = len * TURNS;
    if (rt.e >= 0 && ns > 0) {
        TX x;
        x.init(p, rt, wave, lane);
        WT wt;
        wt.init(p.a, rt.e, o0, c0, wave, lane);
        // After its barrier, step t issues (odd t) the codes of steps t + 3 and t + 4
        // into the buffer that step t was the last to use, then x(t + 4).  At step
        // t's barrier x(t + 1) and the codes of step t + 1 have to be there.  Younger
        // than them are, for odd t, x(t + 2) and x(t + 3), for even t also the codes
        // issued with x(t + 3).  Loads past the end reload the last stage, so the
        // counts always hold.
        constexpr int kYounger = 2 * LOADS;
        TileW<OF> w;
        uint64_t sc[OF][WT::Q], sn[OF][WT::Q];
        TileOps<P, MF, OF> oa, ob;
        const auto plane_of = [&](int s) { return TURNS == 1 ? 0 : s / len; };
        const auto step_of = [&](int s) { return k0 + (TURNS == 1 ? s : s % len); };
        const auto fetch_x = [&](uint8_t* st, int s) {
            const int c = min(s, ns - 1);
            x.load(st, step_of(c), plane_of(c), wave);
        };
        // Planes by turns go on past K to a whole group of four steps.  There x is zero
        // and any code will do: the last step's are read, since a step's offset past the
        // last rows of the codes is no longer one that the buffer's bound can hold back.
        const auto fetch_w = [&](uint8_t* st, int s) {
            const int k = step_of(min(s, ns - 1));
            wt.load(st, TURNS == 1 ? k : min(k, (int)(p.a.K - 1) / 64), wave);
        };
        const auto fetch_s = [&](uint64_t(&v)[OF][WT::Q], int s) { wt.load_scales(step_of(min(s, ns - 1)), v); };
        constexpr int kValu = SF == WF_E8M0 ? 2 : 6;
        // Step s = 4 n + I.  On entry oa holds substep 0 and w the step's codes; on
        // return those of the next step, whose codes have parity (I + 1) % 2 in wnext.
        const auto step = [&]<int I>(uint8_t* cur, const uint8_t* next, uint8_t* wfill, const uint8_t* wnext,
                                     int s) {
            tile_operands<SF, BM>(ob, cur, w, 1, m0, lane);
            tile_products<SF>(oa, acc);
            tile_interleave<P * MF * OF, READS, kValu>();
            __builtin_amdgcn_sched_barrier(0);
            tile_operands<SF, BM>(oa, cur, w, 2, m0, lane);
            tile_products<SF>(ob, acc);
            tile_interleave<P * MF * OF, READS, kValu>();
            __builtin_amdgcn_sched_barrier(0);
            tile_operands<SF, BM>(ob, cur, w, 3, m0, lane);
            tile_products<SF>(oa, acc);
            tile_interleave<P * MF * OF, READS, kValu>();
            __builtin_amdgcn_sched_barrier(0);
            tile_wait_barrier<kYounger>();
            if constexpr (I % 2 == 1) fetch_w(wfill, s + 3);
            fetch_x(cur, s + 4);
            if constexpr (I == 1) fetch_s(sn, s + 3);
            __builtin_amdgcn_sched_barrier(0);
            tile_codes(w, wnext, (I + 1) % 2, c0, lane);
            if constexpr (I == 3) {
                wt.settle_scales(step_of(min(s + 1, ns - 1)), sn);
#pragma unroll
                for (int j = 0; j < OF; ++j)
#pragma unroll
                    for (int q = 0; q < WT::Q; ++q) sc[j][q] = sn[j][q];
            }
#pragma unroll
            for (int j = 0; j < OF; ++j) {
                uint32_t s0, s1;
                wt.codes_of(sc[j], (I + 1) % 4, step_of(min(s + 1, ns - 1)), s0, s1);
                w.s[j][0] = weight_scale<SF>(s0);
                w.s[j][1] = SF == WF_E8M0 ? w.s[j][0] : weight_scale<SF>(s1);
            }
            tile_operands<SF, BM>(oa, next, w, 0, m0, lane);
            tile_products<SF>(ob, acc);
            tile_interleave<P * MF * OF, READS + OF, kValu>();
            __builtin_amdgcn_sched_barrier(0);
        };
        fetch_s(sc, 0);
        fetch_w(wa, 0);
        fetch_x(st0, 0);
        fetch_x(st1, 1);
        fetch_w(wb, 2);
        fetch_x(st2, 2);
        fetch_x(st3, 3);
        tile_wait_barrier<3 * LOADS + WT::LOADS>();
        wt.settle_scales(k0, sc);
        tile_codes(w, wa, 0, c0, lane);
#pragma unroll
        for (int j = 0; j < OF; ++j) {
            uint32_t s0, s1;
            wt.codes_of(sc[j], 0, k0, s0, s1);
            w.s[j][0] = weight_scale<SF>(s0);
            w.s[j][1] = SF == WF_E8M0 ? w.s[j][0] : weight_scale<SF>(s1);
        }
        tile_operands<SF, BM>(oa, st0, w, 0, m0, lane);
        // The loop has no exit inside, so the compiler's waits see only its own order
        // of loads; the steps left over follow.
        int s = 0;
        for (; s + 4 <= ns; s += 4) {
            step.template operator()<0>(st0, st1, nullptr, wa, s);
            step.template operator()<1>(st1, st2, wa, wb, s + 1);
            step.template operator()<2>(st2, st3, nullptr, wb, s + 2);
            step.template operator()<3>(st3, st0, wb, wa, s + 3);
        }
        if (s < ns) step.template operator()<0>(st0, st1, nullptr, wa, s);
        if (s + 1 < ns) step.template operator()<1>(st1, st2, wa, wb, s + 1);
        if (s + 2 < ns) step.template operator()<2>(st2, st3, nullptr, wb, s + 2);
        tile_wait_barrier<0>();          // the loads past the end land before st0 is reused
    }
    // each wave's region of the epilogue: the four stages hold a quarter of the waves each
    constexpr int kRegion = 32 * 32 * OF * 4;
    static_assert(TX::ROWS * 128 >= W / 4 * kRegion, "epilogue region");
    constexpr int QW = W / 4;
    uint8_t* buf = (wave < QW ? st0 : wave < 2 * QW ? st1 : wave < 3 * QW ? st2 : st3) + wave % QW * kRegion;
    tile_finish<false, MF, OF, BO>(p, rt, acc, buf, m0, o0, c0, split, lane);
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------

// The 16-byte chunks of decoded row n are stored XOR this.
__device__ __forceinline__ int tile_w_swizzle(int n) { return (n & 1) << 3 | (n & 2) << 1; }

// One thread's weights of a step: 32 consecutive values (half of them past K
// in the last block of an odd multiple of 16) of row n.
struct GradW {
    u32x4 c;
    uint32_t s;
};

template <int SF, int BO>
struct GradWeights {
    static constexpr int B = kScaleBlock<SF>;
    static constexpr int NB = BO / 32;
    static constexpr int kPitch = BO * 2;              // bytes of a decoded row
    const uint8_t* c;          // codes at row `row` of step 0
    const uint8_t* s;
    int64_t N, K;
    int row, blk;
    int left;                  // of the 32 values, those inside K

    __device__ __forceinline__ void init(const LinearArgs& a, int e, int64_t o0, int tid) {
        row = tid / NB;
        blk = tid % NB;
        N = a.N;
        K = a.K;
        const int64_t k = o0 + 32 * blk;
        left = (int)imax(imin(K - k, 32), 0);
        c = a.codes + ((int64_t)e * N + row) * (K / 2) + k / 2;
        s = a.scales + ((int64_t)e * N + row) * (K / B) + k / B;
    }

    // Two loads, whatever the shape.  Rows past N and blocks past K load zeros.
    // Half a block (K an odd multiple of 16) is loaded with the 16 values before
    // it; a row of 16 values has none and is loaded by itself.
    __device__ __forceinline__ void load(int k, GradW& w) const {
        const int64_t n = (int64_t)k * 64 + row;
        const uint8_t* cp = c + (int64_t)k * 64 * (K / 2);
        const uint8_t* sp = s + (int64_t)k * 64 * (K / B);
        const bool zero = n >= N || left <= 0;
        if (SF != WF_E8M0 && K == 16) {
            if (zero) cp = sp = (const uint8_t*)kZeros;
            const u32x2 lo = load_global<u32x2>(cp);
            w.c = u32x4{lo[0], lo[1], 0u, 0u};
            w.s = load_global<uint8_t>(sp);
            return;
        }
        if (SF != WF_E8M0 && left == 16) {
            cp -= 8;
            sp -= 1;
        }
        if (zero) cp = sp = (const uint8_t*)kZeros;
        w.c = load_global<u32x4_a8>(cp);
        if constexpr (SF == WF_E8M0) w.s = load_global<uint8_t>(sp);
        else w.s = load_global<u16_a1>(sp);
    }

    __device__ __forceinline__ void store(uint8_t* buf, GradW w) const {
        asm volatile("" : "+v"(w.s));        // not any earlier: that would wait for its load
        if (SF != WF_E8M0 && left == 16 && K > 16) {
            w.c = u32x4{w.c[2], w.c[3], 0u, 0u};
            w.s >>= 8;
        }
        const float s0 = weight_scale<SF>(w.s & 0xFFu);
        const float s1 = SF == WF_E8M0 ? s0 : weight_scale<SF>(w.s >> 8);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *(u32x4*)(buf + row * kPitch + ((q * NB + blk) ^ tile_w_swizzle(row)) * 16) =
                decode8<SF>(w.c[q], q < 2 ? s0 : s1);
    }
};

// Fragment of columns c0 + l % 32, rows 16 q + 8 (l / 32) .. + 7, of a
// decoded weight stage.
template <int PITCH>
__device__ __forceinline__ bf16x8 grad_w_frag(const uint8_t* buf, int c0, int q, int lane) {
    const int g = lane >> 4, i = lane & 15;
    const int row = 16 * q + 8 * (g >> 1) + (i >> 2), col = c0 + 16 * (g & 1) + 4 * (i & 3);
    const uint8_t* at = buf + row * PITCH + (((col >> 3) ^ tile_w_swizzle(i >> 2)) << 4) + (col & 4) * 2;
    union {
        s16x4 h[2];
        bf16x8 v;
    } f;
    f.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)at);
    f.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(at + 4 * PITCH));
    return f.v;
}

template <int PITCH, int BM, int P, int MF, int OF>
__device__ __forceinline__ void grad_operands(TileOps<P, MF, OF>& o, const uint8_t* xs, const uint8_t* ws, int q,
                                              int m0, int c0, int lane) {
    tile_x_operands<BM>(o, xs, 2 * q + (lane >> 5), m0, lane);
#pragma unroll
    for (int j = 0; j < OF; ++j) o.w[j] = grad_w_frag<PITCH>(ws, c0 + 32 * j, q, lane);
}

template <int SF, int NP, bool PI, int MF, int OF, int WM, int WO, int PER_CU>
__global__ __launch_bounds__(64 * WM * WO, PER_CU * WM * WO / 4) void k_linear_grad_tile(TileArgs p) {
    constexpr int BM = 32 * MF * WM, BO = 32 * OF * WO, W = WM * WO, P = PI ? NP : 1, TURNS = NP / P;
    using TX = TileX<NP, PI, BM, W, false>;
    constexpr int LOADS = TX::LOADS;
    static_assert(64 * BO / 32 == 64 * W, "one 32-value piece of weights per thread and step");
    using GW = GradWeights<SF, BO>;
    __shared__ __attribute__((aligned(1024))) uint8_t xs0[TX::ROWS * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t xs1[TX::ROWS * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t xs2[TX::ROWS * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t ws0[64 * GW::kPitch];
    __shared__ __attribute__((aligned(1024))) uint8_t ws1[64 * GW::kPitch];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = 32 * MF * (wave / WO), c0 = 32 * OF * (wave % WO);
    const uint32_t wg = (uint32_t)p.first + blockIdx.x;
    const int tiles = p.tiles_m * p.tiles_o, split = wg / tiles;
    int tm, to;
    tile_of(p, wg % tiles, tm, to);
    const RowTile rt = row_tile<BM>(p.a, tm);
    if (rt.rows <= 0) return;
    const int64_t o0 = (int64_t)to * BO;
    f32x16 acc[MF][OF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < OF; ++j) acc[i][j] = f32x16{};
    const int k0 = split * p.split_steps, k1 = min((int)((p.a.N + 63) / 64), k0 + p.split_steps);
    const int ns = (k1 - k0) * TURNS;
    if (rt.e >= 0 && ns > 0) {
        TX x;
        x.init(p, rt, wave, lane);
        GW wt;
        wt.init(p.a, rt.e, o0, threadIdx.x);
        // Step t decodes W(t + 1) (loaded two steps before) into its buffer ahead of
        // its barrier, then issues W(t + 3) and x(t + 3).  At step s's barrier
        // x(s + 1) has to be there; younger than it are W(s + 2) and x(s + 2).  In the
        // steps after the loop the compiler drops weight loads that no step uses, so
        // there only x(s + 2) is counted on.
        GradW wa, wb;
        TileOps<P, MF, OF> oa, ob;
        const auto fetch_x = [&](uint8_t* st, int s) {
            const int c = min(s, ns - 1);
            x.load(st, k0 + c / TURNS, c % TURNS, wave);
        };
        const auto fetch_w = [&](GradW& w, int s) {
            asm volatile("" ::: "memory");
            wt.load(k0 + min(s, ns - 1) / TURNS, w);
            asm volatile("" ::: "memory");
        };
        constexpr int kReads = P * MF + 2 * OF;
        const auto step = [&]<bool LAST>(uint8_t* xc, const uint8_t* xn, const uint8_t* wc, uint8_t* wn, GradW& w,
                                         int s) {
            grad_operands<GW::kPitch, BM>(ob, xc, wc, 1, m0, c0, lane);
            tile_products<SF>(oa, acc);
            tile_interleave<P * MF * OF, kReads, 2>();
            __builtin_amdgcn_sched_barrier(0);
            wt.store(wn, w);
            grad_operands<GW::kPitch, BM>(oa, xc, wc, 2, m0, c0, lane);
            tile_products<SF>(ob, acc);
            __builtin_amdgcn_sched_barrier(0);
            grad_operands<GW::kPitch, BM>(ob, xc, wc, 3, m0, c0, lane);
            tile_products<SF>(oa, acc);
            tile_interleave<P * MF * OF, kReads, 2>();
            __builtin_amdgcn_sched_barrier(0);
            tile_wait_barrier<LAST ? LOADS : LOADS + 2>();
            fetch_w(w, s + 3);
            fetch_x(xc, s + 3);
            __builtin_amdgcn_sched_barrier(0);
            grad_operands<GW::kPitch, BM>(oa, xn, wn, 0, m0, c0, lane);
            tile_products<SF>(ob, acc);
            tile_interleave<P * MF * OF, kReads, 2>();
            __builtin_amdgcn_sched_barrier(0);
        };
        fetch_w(wa, 0);
        fetch_w(wb, 1);
        fetch_x(xs0, 0);
        fetch_x(xs1, 1);
        wt.store(ws0, wa);
        fetch_w(wa, 2);
        fetch_x(xs2, 2);
        tile_wait_barrier<2 * LOADS>();
        grad_operands<GW::kPitch, BM>(oa, xs0, ws0, 0, m0, c0, lane);
        int s = 0;
        for (; s + 6 <= ns; s += 6) {
            step.template operator()<false>(xs0, xs1, ws0, ws1, wb, s);
            step.template operator()<false>(xs1, xs2, ws1, ws0, wa, s + 1);
            step.template operator()<false>(xs2, xs0, ws0, ws1, wb, s + 2);
            step.template operator()<false>(xs0, xs1, ws1, ws0, wa, s + 3);
            step.template operator()<false>(xs1, xs2, ws0, ws1, wb, s + 4);
            step.template operator()<false>(xs2, xs0, ws1, ws0, wa, s + 5);
        }
        if (s < ns) step.template operator()<true>(xs0, xs1, ws0, ws1, wb, s);
        if (s + 1 < ns) step.template operator()<true>(xs1, xs2, ws1, ws0, wa, s + 1);
        if (s + 2 < ns) step.template operator()<true>(xs2, xs0, ws0, ws1, wb, s + 2);
        if (s + 3 < ns) step.template operator()<true>(xs0, xs1, ws1, ws0, wa, s + 3);
        if (s + 4 < ns) step.template operator()<true>(xs1, xs2, ws0, ws1, wb, s + 4);
        tile_wait_barrier<0>();
    }
    constexpr int kRegion = 32 * 32 * OF * 4;
    uint8_t* buf = wave < W / 2 ? xs0 + wave * kRegion : xs1 + (wave - W / 2) * kRegion;
    static_assert(TX::ROWS * 128 >= W / 2 * kRegion, "epilogue region");
    tile_finish<true, MF, OF, BO>(p, rt, acc, buf, m0, o0, c0, split, lane);
}

}  // namespace fp4q_dev
