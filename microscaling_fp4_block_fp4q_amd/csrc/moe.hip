// moe.hip -- the routing table of a mixture of experts and the combination
// of its experts' rows: tokens sorted by expert, their weighted sum back,
// and the gradients of that sum.
#include "moe.hpp"

namespace fp4q_dev {

// ---------------------------------------------------------------------------
// Stable counting sort of the R = T k routed entries by expert.  Entries
// that belong to no expert here count as expert E and go last.
//
// A workgroup's entries are cut into one run per wave.  Each wave counts its
// run's experts, the counts of the waves before it (and of the workgroups
// before this one) give the first place of each expert in its run, and then
// the wave places its run 64 entries at a time, in order: the lanes with the
// same id are found with ballots, one bit of the id at a time, and an entry's
// place is its expert's next one plus the lower lanes with the same id.
// Atomics only count, so the table is the same on every run.
//
// Up to kSortSmall entries one workgroup does it all (512 entries of 64
// experts: 3.2-3.4 us, where the three kernels took 8): launches cost more than
// the work.  Above, three kernels (524288 entries of 256 experts: 4.4-4.6,
// 3.0-3.3 and 9.3 us, where the 6.3 MB would take 1.3; the last one's waves wait
// 0.73 of their time for memory and LDS: strided counts, and a chain of
// dependent accesses per 64 entries):
//   k_sort_count  counts[e][c] = entries of expert e in chunk c
//   k_sort_scan   per expert, exclusive sums over the chunks and their total
//   k_sort_place  sums over the experts' totals, then the places
// ---------------------------------------------------------------------------

// Lanes of the wave whose id equals this lane's (ids below 2^bits).
__device__ __forceinline__ uint64_t same_id(uint32_t id, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const bool on = (id >> b) & 1u;
        const uint64_t v = __ballot(on);
        m &= on ? v : ~v;
    }
    return m;
}

// The id of entry i, E for one that belongs to no expert here.
__device__ __forceinline__ uint32_t sort_id(const SortArgs& p, int64_t i) {
    const uint32_t id = (uint32_t)p.ids[i];
    return id < (uint32_t)p.E ? id : (uint32_t)p.E;
}

__device__ __forceinline__ void sort_clear(uint32_t* n, int count) {
    for (int i = threadIdx.x; i < count; i += blockDim.x) n[i] = 0u;
    __syncthreads();
}

__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t u = __shfl_up(v, d);
        v += lane >= d ? u : 0u;
    }
    return v;
}

// Exclusive sums of n[0 .. E - 1] (E at most 1024) over the workgroup, in
// place; the sum of all goes to n[E].  part: one word per wave.
template <int WAVES>
__device__ __forceinline__ void sort_scan_experts(uint32_t* n, uint32_t* part, int E) {
    constexpr int PER = kSortMaxExperts / (64 * WAVES);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t v[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = PER * tid + i < E ? n[PER * tid + i] : 0u;
        sum += v[i];
    }
    const uint32_t incl = wave_scan(sum, lane);
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    uint32_t at = incl - sum, all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        at += w < wave ? part[w] : 0u;
        all += part[w];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (PER * tid + i < E) n[PER * tid + i] = at;
        at += v[i];
    }
    if (tid == 0) n[E] = all;
    __syncthreads();
}

// Count this wave's run i0 .. i1 - 1 into n.
__device__ __forceinline__ void sort_count_run(const SortArgs& p, uint32_t* n, int64_t i0, int64_t i1, int lane) {
    for (int64_t i = i0 + lane; i < i1; i += 64) atomicAdd(&n[sort_id(p, i)], 1u);
}

// A point that the lanes of a wave pass together, with the LDS accesses of each
// before it ahead of those of all behind it.  The LDS carries out a wave's
// accesses in order, so this costs nothing: it keeps the compiler to it.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Place this wave's run; next[e]: places taken by earlier entries of the
// workgroup, base[e]: first place of its expert for the workgroup.
__device__ __forceinline__ void sort_place_run(const SortArgs& p, uint32_t* next, const uint32_t* base, int64_t i0,
                                               int64_t i1, int lane) {
    const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
    for (int64_t b = i0; b < i1; b += 64) {
        const int64_t i = b + lane;
        const bool in = i < i1;
        const uint32_t id = in ? sort_id(p, i) : 0u;
        const uint64_t same = same_id(id, p.id_bits) & __ballot(in);
        wave_sync();                 // the leaders of the 64 entries before have written
        const uint32_t taken = next[id];
        wave_sync();                 // every lane has read before a leader overwrites
        if (!in) continue;
        if ((same & below) == 0ull) next[id] = taken + (uint32_t)__popcll(same);
        const uint32_t place = base[id] + taken + (uint32_t)__popcll(same & below);
        const bool routed = id < (uint32_t)p.E;
        p.rows[place] = routed ? (int32_t)i : -1;
        p.slots[i] = routed ? (int32_t)place : -1;
    }
}

// next[w][e]: exclusive sums of the waves' counts; their total to all[e].
template <int WAVES>
__device__ __forceinline__ void sort_sum_waves(uint32_t* next, uint32_t* all, int E) {
    for (int e = threadIdx.x; e <= E; e += 64 * WAVES) {
        uint32_t sum = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const uint32_t c = next[w * (kSortMaxExperts + 1) + e];
            next[w * (kSortMaxExperts + 1) + e] = sum;
            sum += c;
        }
        if (all) all[e] = sum;
    }
    __syncthreads();
}

__global__ __launch_bounds__(1024) void k_sort_small(SortArgs p) {
    constexpr int WAVES = 16;
    __shared__ uint32_t next[WAVES * (kSortMaxExperts + 1)], base[kSortMaxExperts + 1], part[WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t* mine = next + wave * (kSortMaxExperts + 1);
    const int64_t run = ((p.R + 64 * WAVES - 1) / (64 * WAVES)) * 64;
    const int64_t i0 = imin(wave * run, p.R), i1 = imin(i0 + run, p.R);
    for (int e = lane; e <= p.E; e += 64) mine[e] = 0u;
    __syncthreads();
    sort_count_run(p, mine, i0, i1, lane);
    __syncthreads();
    sort_sum_waves<WAVES>(next, base, p.E);
    sort_scan_experts<WAVES>(base, part, p.E);
    for (int e = threadIdx.x; e <= p.E; e += 1024) p.offsets[e] = (int32_t)base[e];
    sort_place_run(p, mine, base, i0, i1, lane);
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs p) {
    __shared__ uint32_t n[kSortMaxExperts + 1];
    sort_clear(n, p.E + 1);
    const int64_t i0 = blockIdx.x * p.chunk, i1 = imin(i0 + p.chunk, p.R);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) atomicAdd(&n[sort_id(p, i)], 1u);
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += kSortThreads) p.counts[(int64_t)e * p.chunks + blockIdx.x] = n[e];
}

// One workgroup per expert: exclusive sums over its chunks in place, the
// total to totals[e].
__global__ __launch_bounds__(kSortThreads) void k_sort_scan(SortArgs p) {
    __shared__ uint32_t part[kSortThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t* n = p.counts + (int64_t)blockIdx.x * p.chunks;
    uint32_t carry = 0;
    for (int c0 = 0; c0 < p.chunks; c0 += kSortThreads) {
        const int c = c0 + tid;
        const uint32_t v = c < p.chunks ? n[c] : 0u, incl = wave_scan(v, lane);
        if (lane == 63) part[wave] = incl;
        __syncthreads();
        uint32_t at = carry + incl - v;
#pragma unroll
        for (int w = 0; w < kSortThreads / 64; ++w) {
            at += w < wave ? part[w] : 0u;
            carry += part[w];
        }
        if (c < p.chunks) n[c] = at;
        __syncthreads();
    }
    if (tid == 0) p.counts[(int64_t)(p.E + 1) * p.chunks + blockIdx.x] = carry;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortArgs p) {
    constexpr int WAVES = kSortThreads / 64;
    __shared__ uint32_t next[WAVES * (kSortMaxExperts + 1)], base[kSortMaxExperts + 1], part[WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t* mine = next + wave * (kSortMaxExperts + 1);
    const int64_t c0 = blockIdx.x * p.chunk, c1 = imin(c0 + p.chunk, p.R);
    const int64_t run = p.chunk / WAVES, i0 = imin(c0 + wave * run, c1), i1 = imin(i0 + run, c1);
    const uint32_t* totals = p.counts + (int64_t)(p.E + 1) * p.chunks;
    for (int e = lane; e <= p.E; e += 64) mine[e] = 0u;
    for (int e = tid; e < p.E; e += kSortThreads) base[e] = totals[e];
    __syncthreads();
    sort_count_run(p, mine, i0, i1, lane);
    sort_scan_experts<WAVES>(base, part, p.E);
    if (blockIdx.x == 0)
        for (int e = tid; e <= p.E; e += kSortThreads) p.offsets[e] = (int32_t)base[e];
    __syncthreads();
    for (int e = tid; e <= p.E; e += kSortThreads) base[e] += p.counts[(int64_t)e * p.chunks + blockIdx.x];
    sort_sum_waves<WAVES>(next, nullptr, p.E);
    sort_place_run(p, mine, base, i0, i1, lane);
}

namespace {

// Entries of a chunk: a multiple of the workgroup's size, and no more than
// about 4096 chunks.
int64_t sort_chunk(int64_t R) {
    int64_t c = 1024;
    while ((R + c - 1) / c > 4096) c *= 2;
    return c;
}

}  // namespace

size_t sort_workspace(int64_t R, int E) {
    if (R <= kSortSmall) return 0;
    const int64_t chunks = (R + sort_chunk(R) - 1) / sort_chunk(R);
    return (size_t)((E + 1) * (chunks + 1) * 4 + 255) / 256 * 256;
}

hipError_t launch_sort(const SortArgs& a, hipStream_t s) {
    SortArgs p = a;
    p.id_bits = 1;
    while ((1 << p.id_bits) <= p.E) ++p.id_bits;      // ids 0 .. E
    if (p.R <= kSortSmall) {
        hipLaunchKernelGGL(k_sort_small, dim3(1), dim3(1024), 0, s, p);
        return hipGetLastError();
    }
    p.chunk = sort_chunk(p.R);
    p.chunks = (int)((p.R + p.chunk - 1) / p.chunk);
    hipLaunchKernelGGL(k_sort_count, dim3(p.chunks), dim3(kSortThreads), 0, s, p);
    hipLaunchKernelGGL(k_sort_scan, dim3(p.E + 1), dim3(kSortThreads), 0, s, p);
    hipLaunchKernelGGL(k_sort_place, dim3(p.chunks), dim3(kSortThreads), 0, s, p);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Combination: y[t] = sum_j weights[t][j] h[slots[t][j]], in the order of j,
// fp32 throughout and rounded once.  One lane per 8 columns of a token.  Bound
// by the rows' bytes: 4096 tokens of 8 entries, 4096 columns, bf16, 63-65 us,
// 4.7 TB/s, what a large copy reaches.
// ---------------------------------------------------------------------------

__device__ __forceinline__ int combine_slot(const CombineArgs& p, int64_t i) {
    const int s = p.slots[i];
    return s < (int)p.R ? s : -1;
}

template <int DT>
__global__ __launch_bounds__(256) void k_combine(CombineArgs p) {
    const int64_t per = (p.N + 7) / 8;
    const int64_t i = (p.first + blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.T * per) return;
    const int64_t t = i / per, c = (i - t * per) * 8;
    float sum[8] = {};
    for (int j = 0; j < p.top_k; ++j) {
        const int slot = combine_slot(p, t * p.top_k + j);
        if (slot < 0) continue;
        const float w = p.weights ? p.weights[t * p.top_k + j] : 1.0f;
        float v[8];
        load_row8<DT>(p.h, slot, p.ld_h, c, p.N, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += w * v[q];
    }
    store_y4(p.y, p.y_dt, t, p.ld_y, c, p.N, f32x4{sum[0], sum[1], sum[2], sum[3]});
    if (c + 4 < p.N) store_y4(p.y, p.y_dt, t, p.ld_y, c + 4, p.N, f32x4{sum[4], sum[5], sum[6], sum[7]});
}

// Its gradients: dh[slots[t][j]] = weights[t][j] dy[t] and
// dweights[t][j] = <h[slots[t][j]], dy[t]>; rows of dh that no entry holds
// (from offsets[E] on) are zeros.  One workgroup per token, then per row past
// the entries; dy[t] is read again from the cache for each of its entries.
// Bound by bytes on wide rows: 2047 tokens of 4 entries, 2056 columns, bf16,
// 18.6 us, 4.1 TB/s; 8192 tokens of 8, 4096 columns, 248 us, 4.6 TB/s.  256
// lanes take 2048 columns at a time and the entries one after the other, so
// narrow rows leave lanes idle: 1024 columns 104 us (2.8 TB/s), 512 85 (1.7), 256
// 65 (1.1).
template <int DT>
__global__ __launch_bounds__(256) void k_combine_grad(CombineArgs p) {
    __shared__ float part[4];
    const int tid = threadIdx.x;
    const int64_t t = p.first + blockIdx.x;
    if (t >= p.T) {
        const int64_t r = (int64_t)min(max(p.offsets[p.E], 0), (int)p.R) + t - p.T;
        if (r < p.R)
            for (int64_t c = 4 * tid; c < p.N; c += 1024)
                store_y4(p.dh, p.dh_dt, r, p.ld_dh, c, p.N, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
        return;
    }
    for (int j = 0; j < p.top_k; ++j) {
        const int slot = combine_slot(p, t * p.top_k + j);
        const float w = p.weights ? p.weights[t * p.top_k + j] : 1.0f;
        float dot = 0.0f;
        if (slot >= 0) {
            for (int64_t c = 8 * tid; c < p.N; c += 2048) {
                float g[8];
                load_row8<DT>(p.dy, t, p.ld_dy, c, p.N, g);
                if (p.dweights) {
                    float v[8];
                    load_row8<DT>(p.h, slot, p.ld_h, c, p.N, v);
#pragma unroll
                    for (int q = 0; q < 8; ++q) dot += g[q] * v[q];
                }
                store_y4(p.dh, p.dh_dt, slot, p.ld_dh, c, p.N, f32x4{w * g[0], w * g[1], w * g[2], w * g[3]});
                if (c + 4 < p.N)
                    store_y4(p.dh, p.dh_dt, slot, p.ld_dh, c + 4, p.N,
                             f32x4{w * g[4], w * g[5], w * g[6], w * g[7]});
            }
        }
        if (p.dweights) {
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d);
            if ((tid & 63) == 0) part[tid >> 6] = dot;
            __syncthreads();
            if (tid == 0) p.dweights[t * p.top_k + j] = (part[0] + part[1]) + (part[2] + part[3]);
            __syncthreads();
        }
    }
}

hipError_t launch_combine(const CombineArgs& a, int dt, hipStream_t s) {
    return launch_pieces((a.T * ((a.N + 7) / 8) + 255) / 256, 256, [&](int64_t first, unsigned n) {
        CombineArgs p = a;
        p.first = first;
        const dim3 g(n), b(256);
        if (dt == DT_BF16) hipLaunchKernelGGL(k_combine<DT_BF16>, g, b, 0, s, p);
        else if (dt == DT_F16) hipLaunchKernelGGL(k_combine<DT_F16>, g, b, 0, s, p);
        else hipLaunchKernelGGL(k_combine<DT_F32>, g, b, 0, s, p);
    });
}

hipError_t launch_combine_grad(const CombineArgs& a, int dt, hipStream_t s) {
    return launch_pieces(a.T + a.R, 256, [&](int64_t first, unsigned n) {
        CombineArgs p = a;
        p.first = first;
        const dim3 g(n), b(256);
        if (dt == DT_BF16) hipLaunchKernelGGL(k_combine_grad<DT_BF16>, g, b, 0, s, p);
        else if (dt == DT_F16) hipLaunchKernelGGL(k_combine_grad<DT_F16>, g, b, 0, s, p);
        else hipLaunchKernelGGL(k_combine_grad<DT_F32>, g, b, 0, s, p);
    });
}

}  // namespace fp4q_dev
