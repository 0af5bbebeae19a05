// grouped_few_kernel.cuh -- the products of grouped_kernel.cuh for calls of few tiles
// (single tokens, small batches), and low-rank adapters of requests of a few rows.
//
// One CTA of 6 warps per tile of 128 x TN and slice of the sum; KS CTAs of a cluster
// share a tile's sum, and their fp32 parts meet through distributed shared memory,
// added in slice order and rounded once.  Two CTAs an SM.  What bounds such a call is
// the matrix's bytes on few SMs, and a start and end of its own; hence the split.
//
// LORA: all rows are one group, the shared product's, and each row's own adapter is
// added in fp32 as the parts meet, after h = scale_a * x * down_a^T from a launch before
// (lora_down_kernel, fp32):
//
//     D[j][i] = round(sum_r W[i][r] * x[j][r] + sum_c up_a(j)[i][c] * h[j][c])
//
// As one more stretch of the MMA's sum, with zeros for the rows of other adapters, that
// would be 0 * up for those rows, NaN where an adapter holds an infinity.
#pragma once

#include "grouped_kernel.cuh"

namespace linear_ops {

template <int TN>
struct FewShape {
    static constexpr int P_BYTES = 128 * 128, Q_BYTES = TN * 128, STAGE = P_BYTES + Q_BYTES;
    static constexpr int LISTS = 2 * 4 * (GROUPED_MAX_GROUPS + 4);  // the groups' first rows and first tiles
    // two CTAs an SM: half of 228 KiB, less 1 KiB that each takes beside its own
    static constexpr int BUDGET = 113 * 1024;
    static constexpr int REST = LISTS + TN * 4 + 256 + 896;
    static constexpr int STAGES = (BUDGET - REST) / STAGE;
    // the CTA's fp32 sums, in the ring once it is idle: row j at j * LD floats, 16 bytes
    // off a multiple of 128 bytes
    static constexpr int LD = 128 + 4;
    static constexpr int OFF_P = 0, OFF_Q = STAGES * P_BYTES;
    static constexpr int OFF_START = STAGES * STAGE;
    static constexpr int OFF_TILES = OFF_START + 4 * (GROUPED_MAX_GROUPS + 4);
    static constexpr int OFF_ROWS = OFF_TILES + 4 * (GROUPED_MAX_GROUPS + 4);  // int32 [TN]: the rows' adapters
    static constexpr int OFF_BAR = OFF_ROWS + TN * 4;
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 1) * 8;
    static constexpr int SMEM_ALLOC = OFF_MISC + 16 + 896;
    static constexpr int THREADS = 192;
    static constexpr int TMEM_COLS = TN < 32 ? 32 : TN;
    static_assert(TN == 16 || TN == 32 || TN == 64 || TN == 128, "tile");
    static_assert(STAGES >= 3 && STAGES * STAGE >= 4 * TN * LD && SMEM_ALLOC <= BUDGET, "two CTAs an SM");
};

// What LORA's rows take beside the shared product.
struct LoraParams {
    const float *h;          // [rows][rank]
    const uint16_t *up;      // [adapters][N][rank]
    int64_t up_row, up_matrix;
};

__device__ __forceinline__ float2 widen16(bool bf16, uint32_t w) {
    return bf16 ? Pair<__nv_bfloat16>::widen(&w) : Pair<__half>::widen(&w);
}

// Four sums of a CTA of the cluster (of this CTA without a split).
template <int KS>
__device__ __forceinline__ float4 few_sums(uint32_t addr) {
    float4 v;
    if constexpr (KS > 1) {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(addr)
                     : "memory");
    } else {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(addr)
                     : "memory");
    }
    return v;
}

template <int TN, int KS, int MODE>
__global__ void __launch_bounds__(192, 2)
    grouped_few_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ, const GroupParams p,
                       const LoraParams l) {
    using C = FewShape<TN>;
    static_assert(MODE == kGroupNT || MODE == kGroupNN || MODE == kGroupLora, "the rows are the N side");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const int rank = KS > 1 ? static_cast<int>(blockIdx.x) % KS : 0;
    const int tile = static_cast<int>(blockIdx.x) / KS;

    const uint32_t bar_full = base + C::OFF_BAR, bar_empty = bar_full + 8 * C::STAGES, bar_done = bar_empty + 8 * C::STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    int32_t *start = reinterpret_cast<int32_t *>(smem + C::OFF_START), *tiles = reinterpret_cast<int32_t *>(smem + C::OFF_TILES);
    int32_t *chosen = reinterpret_cast<int32_t *>(smem + C::OFF_ROWS);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_done, 1);
        *abort_flag = 0;
        ptx::fence_mbarrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc<1>(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
        ptx::tmem_relinquish<1>();
    }
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    // LORA follows lora_down_kernel, which lets it start only once the kernels before both
    // have completed: it waits for h alone, below
    if (MODE != kGroupLora || !p.follows) ptx::griddep_wait();
    const int groups = group_starts(p, start, false, nullptr, static_cast<int>(threadIdx.x), C::THREADS);
    __syncthreads();
    GroupTile w;
    if constexpr (MODE == kGroupLora) {
        if (warp == 2) group_tiles<TN, kGroupNT>(p, groups, start, tiles, nullptr, lane);  // the first rows in order
        const int32_t j_tiles = (p.rows + TN - 1) / TN;
        w.group = 0;
        w.i0 = tile / j_tiles * 128;
        w.j0 = tile % j_tiles * TN;
        w.n = p.rows - w.j0 < TN ? p.rows - w.j0 : TN;
        w.r0 = 0;
        w.r = p.R;
        ptx::tcgen05_fence_before();
        __syncthreads();
        ptx::tcgen05_fence_after();
    } else {
        if (warp == 2) group_tiles<TN, MODE>(p, groups, start, tiles, nullptr, lane);
        ptx::tcgen05_fence_before();
        __syncthreads();
        ptx::tcgen05_fence_after();
        if (p.zero_rest) {  // rows without a group: 16-byte units, a warp a row
            const int32_t head = start[0], rest = head + p.rows - start[groups];
            uint16_t *out = static_cast<uint16_t *>(p.out);
            for (int32_t k = static_cast<int32_t>(blockIdx.x) * 6 + warp; k < rest; k += static_cast<int32_t>(gridDim.x) * 6) {
                uint16_t *row = out + static_cast<int64_t>(k < head ? k : start[groups] + (k - head)) * p.out_row;
                for (int32_t u = lane * 8; u < p.I; u += 256) *reinterpret_cast<uint4 *>(row + u) = make_uint4(0, 0, 0, 0);
            }
        }
        w.n = 0;
        if (tile < tiles[groups]) w = group_tile<1, TN, MODE>(p, groups, start, tiles, tile);
    }
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    const bool work = w.n > 0;  // all CTAs of a cluster alike
    const int k_tiles = work ? (w.r + 63) / 64 : 0;
    const int kt_begin = static_cast<int>(static_cast<int64_t>(k_tiles) * rank / KS);
    const int kt_end = static_cast<int>(static_cast<int64_t>(k_tiles) * (rank + 1) / KS);

    if (warp == 0) {
        if (work && ptx::elect_one()) {
            PipelineState ring(C::STAGES, (p.debug_flags & 1u) ? 0u : 1u);
            bool ok = true;
            for (int kt = kt_begin; kt < kt_end; ++kt) {
                if (!wait_bounded(bar_empty + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns, kWaitProducer, kt)) {
                    ok = false;
                    break;
                }
                const int s = ring.stage;
                const uint32_t sp = base + C::OFF_P + s * C::P_BYTES, full = bar_full + 8 * s;
                ptx::mbar_arrive_expect_tx(full, C::STAGE);
                if constexpr (MODE == kGroupNN) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) ptxg::tma_load_3d(sp + b * 8192, &tmP, full, w.i0 + 64 * b, kt * 64, w.group);
                } else {
                    ptxg::tma_load_3d(sp, &tmP, full, kt * 64, w.i0, w.group);
                }
                ptx::tma_load_2d(base + C::OFF_Q + s * C::Q_BYTES, &tmQ, full, kt * 64, w.j0);
                ring.advance();
            }
            if (!ok) {  // time for loads in flight to land before the shared memory goes
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 20000) ptx::nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (work && ptx::elect_one()) {
            PipelineState ring(C::STAGES, 0u);
            const uint32_t idesc = group_idesc<1, MODE>((w.n + 15) / 16 * 16, p.bf16);
            for (int kt = kt_begin; kt < kt_end; ++kt) {
                if (!wait_bounded(bar_full + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns, kWaitMma, kt)) break;
                ptx::tcgen05_fence_after();
                const int s = ring.stage;
                const uint32_t sp = base + C::OFF_P + s * C::P_BYTES, sq = base + C::OFF_Q + s * C::Q_BYTES;
                constexpr bool kMn = MODE == kGroupNN;
                const uint64_t pd = kMn ? ptxg::smem_desc_mn_sw128(sp, 8192) : ptx::smem_desc_k_sw128(sp);
                const uint64_t qd = ptx::smem_desc_k_sw128(sq);
                const int steps = w.r - kt * 64 >= 64 ? 4 : (w.r - kt * 64 + 15) / 16;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k < steps) {
                        ptx::mma_f16<1>(tmem_base, pd + k * (kMn ? 128 : 2), qd + k * 2, idesc, kt > kt_begin || k > 0 ? 1u : 0u);
                    }
                }
                ptx::mma_commit<1>(bar_empty + 8 * s, 0x1);
                ring.advance();
            }
            // every MMA issued so far (after an abort as well: TMEM is freed below)
            ptx::mma_commit<1>(bar_done, 0x1);
            wait_bounded(bar_done, 0, abort_flag, p.timeout_ns, kWaitMma, 0xFFFFFFFFu, false);
        }
        __syncwarp();
    } else if (work) {
        if constexpr (MODE == kGroupLora) {  // the rows' adapters: the last request that starts at or before a row
            for (int32_t j = static_cast<int32_t>(threadIdx.x) - 64; j < w.n; j += 128) {
                const int32_t row = w.j0 + j;
                int lo = -1, hi = groups;  // start[lo] <= row < start[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (start[mid] <= row) {
                        lo = mid;
                    } else {
                        hi = mid;
                    }
                }
                chosen[j] = lo >= 0 && row < start[groups] ? adapter_of(p, lo) : -1;
            }
        }
        // all MMAs done: the accumulator is complete and the ring idle
        bool ok = true;
        if (lane == 0) ok = wait_bounded(bar_done, 0, abort_flag, p.timeout_ns, kWaitEpilogue, 0);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (ok && *abort_flag == 0) {
            ptx::tcgen05_fence_after();
            const int i = (warp & 3) * 32 + lane;
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
            for (int c = 0; c < TN; c += 16) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(taddr + c, v);
                ptx::tmem_wait_ld();
                // without K tiles of its own a CTA adds nothing
#pragma unroll
                for (int j = 0; j < 16; ++j) sums[(c + j) * C::LD + i] = kt_begin < kt_end ? __uint_as_float(v[j]) : 0.f;
            }
        }
    }
    // ---- the cluster's sums of this CTA's share of the tile, added and stored
    ptx::tcgen05_fence_before();
    if constexpr (KS > 1) {
        ptx::cluster_sync();
    } else {
        __syncthreads();
    }
    if (MODE == kGroupLora) ptx::griddep_wait();  // all threads: no later kernel may start before lora_down_kernel has ended
    if (work && *abort_flag == 0) {
        // four columns i a thread and step, 32 threads a row j
        const int units = w.n * 32;
        const int first = units * rank / KS, last = units * (rank + 1) / KS;
        uint32_t peer[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) peer[s] = KS > 1 ? ptx::mapa(base, static_cast<uint32_t>(s)) : base;
        for (int u = first + static_cast<int>(threadIdx.x); u < last; u += C::THREADS) {
            const int j = u / 32, i = u % 32 * 4;
            const int32_t col = w.i0 + i;
            if (col >= p.I) continue;
            const uint32_t at = static_cast<uint32_t>(j * C::LD + i) * 4u;
            float4 part[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) part[s] = few_sums<KS>(peer[s] + at);
            float v[4] = {part[0].x, part[0].y, part[0].z, part[0].w};
#pragma unroll
            for (int s = 1; s < KS; ++s) v[0] += part[s].x, v[1] += part[s].y, v[2] += part[s].z, v[3] += part[s].w;
            const int64_t row = w.j0 + j;
            if constexpr (MODE == kGroupLora) {
                const int32_t a = chosen[j];
                if (a >= 0) {
                    const uint16_t *up = l.up + a * l.up_matrix + col * l.up_row;
                    const float *h = l.h + row * p.rank;
#pragma unroll 2
                    for (int c = 0; c < p.rank; c += 8) {
                        const float4 h0 = *reinterpret_cast<const float4 *>(h + c), h1 = *reinterpret_cast<const float4 *>(h + c + 4);
                        uint4 m[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) m[q] = *reinterpret_cast<const uint4 *>(up + q * l.up_row + c);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float2 t = widen16(p.bf16, m[q].x);
                            v[q] = fmaf(h0.x, t.x, v[q]), v[q] = fmaf(h0.y, t.y, v[q]);
                            t = widen16(p.bf16, m[q].y);
                            v[q] = fmaf(h0.z, t.x, v[q]), v[q] = fmaf(h0.w, t.y, v[q]);
                            t = widen16(p.bf16, m[q].z);
                            v[q] = fmaf(h1.x, t.x, v[q]), v[q] = fmaf(h1.y, t.y, v[q]);
                            t = widen16(p.bf16, m[q].w);
                            v[q] = fmaf(h1.z, t.x, v[q]), v[q] = fmaf(h1.w, t.y, v[q]);
                        }
                    }
                }
            }
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + row * p.out_row + col) =
                make_uint2(pack_pair(p.bf16, __float_as_uint(v[0]), __float_as_uint(v[1])),
                           pack_pair(p.bf16, __float_as_uint(v[2]), __float_as_uint(v[3])));
        }
    }
    if constexpr (KS > 1) {
        // no CTA leaves while another reads its sums (they are in registers by now)
        ptx::cluster_arrive_relaxed();
        ptx::cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        ptx::tcgen05_fence_after();
        ptx::tmem_dealloc<1>(tmem_base, C::TMEM_COLS);
    }
}

// h[row] = scale_a * x[row] * down_a^T in fp32 for the rows with an adapter: a warp a rank,
// of ROWS consecutive rows, of which those of one adapter share what is read of it.
struct DownParams {
    const uint16_t *x, *down;
    int64_t x_row, down_row, down_matrix;
    float *h;
};

__device__ __forceinline__ float dot_8(bool bf16, uint4 a, uint4 b, float sum) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 s = widen16(bf16, u[i]), t = widen16(bf16, v[i]);
        sum = fmaf(s.x, t.x, sum);
        sum = fmaf(s.y, t.y, sum);
    }
    return sum;
}

template <int ROWS>
__global__ void __launch_bounds__(256) lora_down_kernel(const GroupParams p, const DownParams d) {
    __shared__ int32_t past[ROWS];  // the first request that starts behind a row
    const int tid = static_cast<int>(threadIdx.x), lane = tid % 32;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS;
    if (tid < ROWS) past[tid] = p.groups + 1;
    ptx::griddep_wait();
    // what follows may start: all before this kernel has completed
    if (tid == 0) ptx::griddep_launch_dependents();
    __syncthreads();
    int32_t least[ROWS];
#pragma unroll
    for (int t = 0; t < ROWS; ++t) least[t] = p.groups + 1;
    for (int e = p.groups - tid; e >= 0; e -= 256) {
        const int64_t o = offset_of(p, e);
#pragma unroll
        for (int t = 0; t < ROWS; ++t) {
            if (o > first + t) least[t] = e;
        }
    }
#pragma unroll
    for (int t = 0; t < ROWS; ++t) {
        const int32_t v = __reduce_min_sync(0xffffffffu, least[t]);
        if (lane == 0) atomicMin(&past[t], v);
    }
    __syncthreads();
    const int j = static_cast<int>(blockIdx.y) * 8 + tid / 32;
    if (j >= p.rank) return;
    int32_t a[ROWS];
#pragma unroll
    for (int t = 0; t < ROWS; ++t) {
        const int e = past[t] - 1;
        a[t] = first + t < p.rows && e >= 0 && e < p.groups ? adapter_of(p, e) : -1;
    }
    const uint16_t *x = d.x + first * d.x_row, *down = d.down + j * d.down_row;
    float sum[ROWS];
#pragma unroll
    for (int t = 0; t < ROWS; ++t) sum[t] = 0.f;
    if constexpr (ROWS == 1) {
        if (a[0] < 0) return;
        down += a[0] * d.down_matrix;
        constexpr int U = 8;  // loads on their way at once
        for (int k = lane * 8; k < p.R; k += 256 * U) {
            uint4 u[U], v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                u[i] = v[i] = make_uint4(0, 0, 0, 0);
                if (k + i * 256 < p.R) {
                    u[i] = load_unit(down + k + i * 256);
                    v[i] = *reinterpret_cast<const uint4 *>(x + k + i * 256);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) sum[0] = dot_8(p.bf16, u[i], v[i], sum[0]);
        }
    } else {
        for (int k = lane * 8; k < p.R; k += 256) {
            uint4 m = make_uint4(0, 0, 0, 0), v[ROWS];
#pragma unroll
            for (int t = 0; t < ROWS; ++t) {
                v[t] = make_uint4(0, 0, 0, 0);
                if (a[t] >= 0) v[t] = *reinterpret_cast<const uint4 *>(x + t * d.x_row + k);
            }
#pragma unroll
            for (int t = 0; t < ROWS; ++t) {
                if (a[t] < 0) continue;
                if (t == 0 || a[t] != a[t - 1]) m = *reinterpret_cast<const uint4 *>(down + a[t] * d.down_matrix + k);
                sum[t] = dot_8(p.bf16, m, v[t], sum[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < ROWS; ++t) {
        float v = sum[t];
#pragma unroll
        for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0 && a[t] >= 0) d.h[(first + t) * p.rank + j] = v * (p.scales ? p.scales[a[t]] : 1.f);
    }
}

}  // namespace linear_ops
