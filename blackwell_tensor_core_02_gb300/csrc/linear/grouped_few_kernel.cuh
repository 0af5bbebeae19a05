// grouped_few_kernel.cuh -- the products of grouped_kernel.cuh for calls of few tiles
// (single tokens, small batches), and low-rank adapters of requests of a few rows.
//
// One CTA of 6 warps per tile of 128 x TN and slice of the sum; KS CTAs of a cluster
// share a tile's sum, and their fp32 parts meet through distributed shared memory,
// added in slice order and rounded once.  Two CTAs an SM.  What bounds such a call is
// the matrix's bytes on few SMs (of sums over rows, TN: the rows'), and a start and end of
// its own; hence the split.
//
// LORA: all rows are one group, the shared product's, and each row's own adapter is
// added before the parts meet, after h = scale_a * x * down_a^T from a launch before
// (lora_down_kernel, as two 16-bit numbers, see grouped_kernel.cuh):
//
//     D[j][i] = round(sum_r W[i][r] * x[j][r] + sum_c up_a(j)[i][c] * h[j][c])
//
// As one more stretch of the shared sum, with zeros for the rows of other adapters, that
// would be 0 * up for those rows, NaN where an adapter holds an infinity.  So consecutive
// rows of one adapter are a piece, with columns of TMEM of its own: the MMA multiplies
// up_a with the rows of h from the piece's first on, and the epilogue adds the columns
// that are the piece's to its sums.  The cluster's CTAs have the pieces of a share of the
// tile's rows each, as many at once as TMEM has columns for.
#pragma once

#include <type_traits>

#include "grouped_kernel.cuh"

namespace linear_ops {

template <int TN, bool LORA>
struct FewShape {
    static constexpr int P_BYTES = 128 * 128, Q_BYTES = (LORA && TN < 32 ? 32 : TN) * 128, STAGE = P_BYTES + Q_BYTES;
    static constexpr int LIST = 4 * (GROUPED_MAX_GROUPS + 4);  // the groups' first rows; their first tiles
    static constexpr int PIECE = TN < 64 ? 16 : TN / 2;        // rows of a piece, at most: h, twice, lies where a stage has Q
    static constexpr int PIECE_COLS = 512 - TN;                // columns of TMEM for pieces, each a multiple of 16
    // the CTA's fp32 sums, row j at j * LD floats, 16 bytes off a multiple of 128 bytes: in
    // the ring once it is idle, of LORA behind it
    static constexpr int LD = 128 + 4;
    static constexpr int SUMS = 4 * TN * LD;
    // the rest of the shared memory, behind the ring
    static constexpr int OFF_START = LORA ? SUMS : 0, OFF_TILES = OFF_START + LIST;
    static constexpr int OFF_ROWS = OFF_TILES + LIST;             // int32 [TN]: the rows' adapters
    static constexpr int OFF_BACK = OFF_ROWS + TN * 4;            // float [TN]: what brings the rows' h back
    static constexpr int OFF_PIECES = OFF_BACK + (LORA ? TN * 4 : 0);  // Piece [TN], behind it their number
    static constexpr int OFF_BAR = OFF_PIECES + (LORA ? TN * 16 : 0) + 16;
    static constexpr int MOST_STAGES = 12;
    // full, empty [stages]; done, list, pieces full, pieces free, drain
    static constexpr int OFF_MISC = OFF_BAR + (2 * MOST_STAGES + 5) * 8;
    static constexpr int REST = OFF_MISC + 16 + 896;
    // Stages of a CTA that shares its SM with another (half of 228 KiB, less 1 KiB that each
    // takes beside its own), and of one that has it alone, where that is more memory than
    // two could have.  64 x 4096 x 4096: 4 CTAs a tile with 4 stages 10.8 us, with 8 9.2.
    static constexpr int PAIRED = LORA ? 0 : (113 * 1024 - REST) / STAGE;
    static constexpr int MOST = LORA ? 220 * 1024 : 232448;  // LORA leaves room for the launch before it
    static constexpr int ALONE = (MOST - REST) / STAGE < MOST_STAGES ? (MOST - REST) / STAGE : MOST_STAGES;
    static constexpr int smem(int stages) { return stages * STAGE + REST; }
    static constexpr int THREADS = 192;
    static constexpr int TMEM_COLS = LORA ? 512 : (TN < 32 ? 32 : TN);
    static_assert(TN == 16 || TN == 32 || TN == 64 || TN == 128, "tile");
    static_assert(OFF_BAR % 8 == 0 && ALONE >= 4 && ALONE * STAGE + REST > 114 * 1024, "an SM alone");
    static_assert(LORA || (PAIRED >= 3 && PAIRED * STAGE >= SUMS), "two CTAs an SM");
};

// A piece as the producer and the MMA issuer take it, ready for use (a thread by itself
// issues an instruction every few cycles: with these taken apart piece by piece, one cost
// it 600 cycles, the MMAs' four times).
struct alignas(16) Piece {
    uint32_t idesc;
    uint16_t column;  // of the TMEM columns for pieces: [column, column + rows in whole 16s)
    uint8_t first;    // row of the tile
    uint8_t rows;
    int32_t adapter;
    uint32_t turn;    // 1: the columns start again from 0, when the pieces before have been read
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
__global__ void __launch_bounds__(192, MODE == kGroupLora ? 1 : 2)
    grouped_few_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmH,
                       const __grid_constant__ GroupTails<MODE> tails, const GroupParams p, const int stages) {
    constexpr bool LORA = MODE == kGroupLora;
    using C = FewShape<TN, LORA>;
    static_assert(MODE != kGroupDown && (MODE != kGroupTN || TN % 64 == 0), "MN-major blocks of 64");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t ring_bytes = static_cast<uint32_t>(stages) * C::STAGE, off_q = static_cast<uint32_t>(stages) * C::P_BYTES;
    uint8_t *smem = smem_raw + (base - raw) + ring_bytes;  // what lies behind the ring
    const uint32_t sums_at = LORA ? base + ring_bytes : base;
    float *sums = reinterpret_cast<float *>(smem_raw + (sums_at - raw));
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const int rank = KS > 1 ? static_cast<int>(blockIdx.x) % KS : 0;
    const int tile = static_cast<int>(blockIdx.x) / KS;

    const uint32_t bar_full = base + ring_bytes + C::OFF_BAR, bar_empty = bar_full + 8 * stages;
    const uint32_t bar_done = bar_empty + 8 * stages;                               // the shared sum is complete
    const uint32_t bar_list = bar_done + 8, bar_pfull = bar_list + 8, bar_pfree = bar_pfull + 8, bar_drain = bar_pfree + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    int32_t *start = reinterpret_cast<int32_t *>(smem + C::OFF_START), *tiles = reinterpret_cast<int32_t *>(smem + C::OFF_TILES);
    int32_t *chosen = reinterpret_cast<int32_t *>(smem + C::OFF_ROWS), *piece_count = reinterpret_cast<int32_t *>(smem + C::OFF_BAR) - 4;
    float *back = reinterpret_cast<float *>(smem + C::OFF_BACK);
    Piece *pieces = reinterpret_cast<Piece *>(smem + C::OFF_PIECES);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < stages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_done, 1);
        ptx::mbar_init(bar_list, 1);
        ptx::mbar_init(bar_pfull, 1);
        ptx::mbar_init(bar_pfree, 4);
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0;
        ptx::fence_mbarrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc<1>(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
        ptx::tmem_relinquish<1>();
    }
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    // LORA follows lora_down_kernel, which lets it start only once the kernels before both
    // have completed: it waits for h alone, in the producer
    if (!LORA || !p.follows) ptx::griddep_wait();
    const int groups = p.groups;
    if constexpr (!LORA) {  // LORA's epilogue lists the requests, beside the shared sum
        group_starts(p, start, false, nullptr, static_cast<int>(threadIdx.x), C::THREADS);
        __syncthreads();
        if (warp == 2) group_tiles<TN, MODE>(p, groups, start, tiles, nullptr, lane);
    }
    ptx::tcgen05_fence_before();
    __syncthreads();
    ptx::tcgen05_fence_after();
    GroupTile w;
    w.n = 0;
    if constexpr (LORA) {
        const int32_t j_tiles = (p.rows + TN - 1) / TN;
        w.group = 0;
        w.i0 = tile / j_tiles * 128;
        w.j0 = tile % j_tiles * TN;
        w.n = p.rows - w.j0 < TN ? p.rows - w.j0 : TN;
        w.r0 = 0;
        w.r = p.R;
    } else {
        if (p.zero_rest) {  // rows without a group: 16-byte units, a warp a row
            const int32_t head = start[0], rest = head + p.rows - start[groups];
            uint16_t *out = static_cast<uint16_t *>(p.out);
            for (int32_t k = static_cast<int32_t>(blockIdx.x) * 6 + warp; k < rest; k += static_cast<int32_t>(gridDim.x) * 6) {
                uint16_t *row = out + static_cast<int64_t>(k < head ? k : start[groups] + (k - head)) * p.out_row;
                for (int32_t u = lane * 8; u < p.I; u += 256) *reinterpret_cast<uint4 *>(row + u) = make_uint4(0, 0, 0, 0);
            }
        }
        if (tile < tiles[groups]) {
            int lo = 0, hi = groups;  // tiles[lo] <= tile < tiles[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (tiles[mid] <= tile) {
                    lo = mid;
                } else {
                    hi = mid;
                }
            }
            w = group_tile<1, TN, MODE>(p, start, tiles, tile, lo);
        }
    }
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    const bool work = w.n > 0;  // all CTAs of a cluster alike
    const int k_tiles = work ? (w.r + 63) / 64 : 0;
    const int kt_begin = static_cast<int>(static_cast<int64_t>(k_tiles) * rank / KS);
    const int kt_end = static_cast<int>(static_cast<int64_t>(k_tiles) * (rank + 1) / KS);

    if (warp == 0) {
        if (work && ptx::elect_one()) {
            PipelineState ring(stages, (p.debug_flags & 1u) ? 0u : 1u);
            bool ok = true;
            for (int kt = kt_begin; kt < kt_end; ++kt) {
                if (!wait_bounded(bar_empty + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns, kWaitProducer, kt)) {
                    ok = false;
                    break;
                }
                const int s = ring.stage;
                const uint32_t sp = base + s * C::P_BYTES, full = bar_full + 8 * s;
                if constexpr (MODE == kGroupTN) {
                    load_sum_rows<1>(p, tmP, tmQ, tails, w, kt * 64, w.i0, w.j0, (w.n + 63) / 64, true, sp, base + off_q + s * C::Q_BYTES, full);
                    ring.advance();
                    continue;
                }
                ptx::mbar_arrive_expect_tx(full, C::P_BYTES + TN * 128);
                if constexpr (MODE == kGroupNN) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) ptxg::tma_load_3d(sp + b * 8192, &tmP, full, w.i0 + 64 * b, kt * 64, w.group);
                } else {
                    ptxg::tma_load_3d(sp, &tmP, full, kt * 64, w.i0, w.group);
                }
                ptx::tma_load_2d(base + off_q + s * C::Q_BYTES, &tmQ, full, kt * 64, w.j0);
                ring.advance();
            }
            if constexpr (LORA) {
                ok = ok && wait_bounded(bar_list, 0, abort_flag, p.timeout_ns, kWaitProducer, 0);
                const int count = ok ? *piece_count : 0;
                if (count > 0) ptx::griddep_wait();
                Piece piece = pieces[0];
                for (int q = 0, c = 0; ok && q < count;) {
                    const int32_t row = w.j0 + piece.first, a = piece.adapter;
                    const int boxes = (piece.rows + 15) / 16;  // of 16 rows of h
                    if (!wait_bounded(bar_empty + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns, kWaitProducer, q)) {
                        ok = false;
                        break;
                    }
                    const int s = ring.stage;
                    const uint32_t sq = base + off_q + s * C::Q_BYTES, full = bar_full + 8 * s;
                    ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(C::P_BYTES + 2 * boxes * 2048));
                    ptxg::tma_load_3d(base + s * C::P_BYTES, &tmU, full, c, w.i0, a);
                    for (int b = 0; b < boxes; ++b) {
                        ptx::tma_load_2d(sq + b * 2048, &tmH, full, c, row + 16 * b);
                        ptx::tma_load_2d(sq + C::PIECE * 128 + b * 2048, &tmH, full, p.rank_pad + c, row + 16 * b);
                    }
                    ring.advance();
                    c += 64;
                    if (c >= p.rank) c = 0, piece = pieces[++q];
                }
            }
            if (!ok) {  // time for loads in flight to land before the shared memory goes
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 20000) ptx::nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (work && ptx::elect_one()) {
            PipelineState ring(stages, 0u);
            const uint32_t idesc = group_idesc<1, MODE>((w.n + 15) / 16 * 16, p.bf16);
            constexpr bool kMnP = MODE == kGroupNN || MODE == kGroupTN, kMnQ = MODE == kGroupTN;
            const uint32_t p_low = kMnP ? ptxg::desc_mn_low(base) : ptxg::desc_k_low(base);
            const uint32_t q_low = kMnQ ? ptxg::desc_mn_low(base + off_q) : ptxg::desc_k_low(base + off_q);
            bool ok = true;
            for (int kt = kt_begin; kt < kt_end; ++kt) {
                if (!wait_bounded(bar_full + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns, kWaitMma, kt)) {
                    ok = false;
                    break;
                }
                ptx::tcgen05_fence_after();
                const int s = ring.stage;
                const int left = w.r - kt * 64;
                ptxg::mma_stage<1, kMnP ? 128 : 2, kMnQ ? 128 : 2>(
                    tmem_base, p_low + static_cast<uint32_t>(s * (C::P_BYTES >> 4)), q_low + static_cast<uint32_t>(s * (C::Q_BYTES >> 4)),
                    idesc, left >= 64 ? 4 : (left + 15) / 16, kt == kt_begin);
                ptx::mma_commit<1>(bar_empty + 8 * s, 0x1);
                ring.advance();
            }
            if (ok) ptx::mma_commit<1>(bar_done, 0x1);
            if constexpr (LORA) {
                ok = ok && wait_bounded(bar_list, 0, abort_flag, p.timeout_ns, kWaitMma, 0);
                const int count = ok ? *piece_count : 0;
                uint32_t turn = 0;  // pieces that had their columns at once
                Piece piece = pieces[0];
                for (int q = 0; ok && q < count; ++q) {
                    const uint32_t d = tmem_base + TN + piece.column, piece_idesc = piece.idesc;
                    if (piece.turn) {  // the epilogue has read the pieces before
                        ptx::mma_commit<1>(bar_pfull, 0x1);
                        if (!wait_bounded(bar_pfree, turn & 1u, abort_flag, p.timeout_ns, kWaitMma, q)) {
                            ok = false;
                            break;
                        }
                        ++turn;
                        ptx::tcgen05_fence_after();
                    }
                    piece = pieces[q + 1];  // behind the last one: anything
                    // little code: a thread by itself waits for each line of it that is not at hand
                    uint32_t more = 0;
                    int left = p.rank;
#pragma unroll 1
                    do {
                        if (!wait_bounded(bar_full + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns, kWaitMma, q)) {
                            ok = false;
                            break;
                        }
                        ptx::tcgen05_fence_after();
                        uint32_t up = p_low + static_cast<uint32_t>(ring.stage * (C::P_BYTES >> 4));
                        uint32_t high = q_low + static_cast<uint32_t>(ring.stage * (C::Q_BYTES >> 4));
                        const int end = left > 64 ? left - 64 : 0;
#pragma unroll 1
                        for (; left > end; left -= 16, up += 2, high += 2, more = 1) {
                            ptxg::mma_f16<1>(d, up, high, piece_idesc, more);
                            ptxg::mma_f16<1>(d, up, high + (C::PIECE * 128 >> 4), piece_idesc, 1u);
                        }
                        left = end;
                        ptx::mma_commit<1>(bar_empty + 8 * ring.stage, 0x1);
                        ring.advance();
                    } while (left > 0);
                }
                if (ok && count > 0) ptx::mma_commit<1>(bar_pfull, 0x1);
            }
            // every MMA issued so far (after an abort as well: TMEM is freed below)
            ptx::mma_commit<1>(bar_drain, 0x1);
            wait_bounded(bar_drain, 0, abort_flag, p.timeout_ns, kWaitMma, 0xFFFFFFFFu, false);
        }
        __syncwarp();
    } else if (work) {
        if constexpr (LORA) {  // the rows' adapters: that of the last request that starts at or before a row
            group_starts(p, start, false, nullptr, static_cast<int>(threadIdx.x) - 64, 128);
            ptxg::sync_128(1);
            if (warp == 2) group_tiles<TN, kGroupNT>(p, groups, start, tiles, nullptr, lane);
            ptxg::sync_128(1);
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
            ptxg::sync_128(1);
            if (warp == 2 && lane == 0) {  // the pieces of this CTA's share of the rows
                const int first = w.n * rank / KS, last = w.n * (rank + 1) / KS;
                int count = 0, column = 0;
                int32_t next = first < last ? chosen[first] : -1;
                for (int j = first; j < last;) {
                    const int32_t a = next;
                    int n = 1;
                    while (j + n < last && (next = chosen[j + n]) == a && n < C::PIECE) ++n;
                    if (a >= 0) {
                        const int columns = (n + 15) / 16 * 16;
                        const bool turn = column + columns > C::PIECE_COLS;
                        if (turn) column = 0;
                        pieces[count++] = {group_idesc<1, MODE>(columns, p.bf16), static_cast<uint16_t>(column),
                                           static_cast<uint8_t>(j), static_cast<uint8_t>(n), a, turn ? 1u : 0u};
                        column += columns;
                    }
                    j += n;
                }
                *piece_count = count;
                ptx::mbar_arrive(bar_list);
            }
        }
        // the shared sum is complete (without LORA, the ring idle)
        bool ok = true;
        if (lane == 0) ok = wait_bounded(bar_done, 0, abort_flag, p.timeout_ns, kWaitEpilogue, 0);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        const int i = (warp & 3) * 32 + lane;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        if (ok && *abort_flag == 0) {
            ptx::tcgen05_fence_after();
#pragma unroll
            for (int c = 0; c < TN; c += 16) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(taddr + c, v);
                ptx::tmem_wait_ld();
                // without K tiles of its own a CTA adds nothing
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float own = kt_begin < kt_end ? __uint_as_float(v[j]) : 0.f;
                    sums[(c + j) * C::LD + i] = own;
                }
            }
        }
        if constexpr (LORA) {
            if (lane == 0) ok = ok && wait_bounded(bar_list, 0, abort_flag, p.timeout_ns, kWaitEpilogue, 0);
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            const int count = ok ? *piece_count : 0;
            uint32_t turn = 0;
            bool scaled = false;
            if (!p.bf16 && p.follows) {  // the powers of two that h has been divided by, while the first pieces are multiplied
                ptx::griddep_wait();
                for (int32_t j = static_cast<int32_t>(threadIdx.x) - 64; j < w.n; j += 128) {
                    back[j] = chosen[j] >= 0 ? p.row_scale[w.j0 + j] : 1.f;
                    scaled = scaled || back[j] != 1.f;
                }
                scaled = ptxg::any_of_128(1, scaled);
            }
            // What the columns v are of tile's rows j on, times those rows' powers (apart from the sums, whose
            // loads would wait for one another's stores; with the choice inside the loop 128 requests of 4 rows
            // took 50.7 us, so 49.8).
            auto bring_back = [&](uint32_t (&v)[16], int j) {
#pragma unroll
                for (int t = 0; t < 16; ++t) {
                    if (j + t < TN) v[t] = __float_as_uint(__uint_as_float(v[t]) * back[j + t]);
                }
            };
            auto add_pieces = [&](auto scaled_type) {
                constexpr bool SCALED = decltype(scaled_type)::value;
                for (int q = 0; q < count; ++turn) {
                    if (lane == 0) ok = wait_bounded(bar_pfull, turn & 1u, abort_flag, p.timeout_ns, kWaitEpilogue, q);
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (!ok) break;
                    ptx::tcgen05_fence_after();
                    do {
                        // pieces of one row, up to eight at once
                        constexpr int B = 8;
                        uint32_t v[16];
                        int some = 0;
#pragma unroll
                        for (int s = 0; s < B; ++s) {
                            if (s == some && q + s < count && pieces[q + s].rows == 1 && (s == 0 || !pieces[q + s].turn)) {
                                ptxg::tmem_ld_32x32b_x1(taddr + TN + pieces[q + s].column, v[s]);
                                ++some;
                            }
                        }
                        if (some > 0) {
                            ptx::tmem_wait_ld();
                            if constexpr (SCALED) {
#pragma unroll
                                for (int s = 0; s < B; ++s) {
                                    if (s < some) v[s] = __float_as_uint(__uint_as_float(v[s]) * back[pieces[q + s].first]);
                                }
                            }
#pragma unroll
                            for (int s = 0; s < B; ++s) {
                                if (s < some) sums[pieces[q + s].first * C::LD + i] += __uint_as_float(v[s]);
                            }
                            q += some;
                            continue;
                        }
                        // 16 columns of two pieces at once, or of one of more
                        const Piece piece = pieces[q];
                        const bool two = piece.rows <= 16 && q + 1 < count && !pieces[q + 1].turn && pieces[q + 1].rows <= 16;
                        const Piece next = pieces[two ? q + 1 : q];
                        uint32_t x[16];
                        for (int c = 0; c < piece.rows; c += 16) {
                            ptx::tmem_ld_32x32b_x16(taddr + TN + piece.column + c, v);
                            if (two) ptx::tmem_ld_32x32b_x16(taddr + TN + next.column, x);
                            ptx::tmem_wait_ld();
                            if constexpr (SCALED) bring_back(v, piece.first + c);
#pragma unroll
                            for (int t = 0; t < 16; ++t) {
                                if (c + t < piece.rows) sums[(piece.first + c + t) * C::LD + i] += __uint_as_float(v[t]);
                            }
                        }
                        if (two) {
                            if constexpr (SCALED) bring_back(x, next.first);
#pragma unroll
                            for (int t = 0; t < 16; ++t) {
                                if (t < next.rows) sums[(next.first + t) * C::LD + i] += __uint_as_float(x[t]);
                            }
                            ++q;
                        }
                        ++q;
                    } while (q < count && !pieces[q].turn);
                    ptx::tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar_pfree);
                }
            };
            if (scaled) {
                add_pieces(std::true_type{});
            } else {
                add_pieces(std::false_type{});
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
    if (LORA) ptx::griddep_wait();  // all threads: no later kernel may start before lora_down_kernel has ended
    if (work && *abort_flag == 0) {
        // four columns i a thread and step, 32 threads a row j
        const int units = w.n * 32;
        const int first = units * rank / KS, last = units * (rank + 1) / KS;
        uint32_t peer[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) peer[s] = KS > 1 ? ptx::mapa(sums_at, static_cast<uint32_t>(s)) : sums_at;
        for (int u = first + static_cast<int>(threadIdx.x); u < last; u += C::THREADS) {
            const int j = u / 32, i = u % 32 * 4;
            const int32_t col = w.i0 + i;
            if (col >= p.I) continue;
            const uint32_t at = static_cast<uint32_t>(j * C::LD + i) * 4u;
            float4 part[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) part[s] = few_sums<KS>(peer[s] + at);
            float4 v = part[0];
#pragma unroll
            for (int s = 1; s < KS; ++s) v.x += part[s].x, v.y += part[s].y, v.z += part[s].z, v.w += part[s].w;
            uint16_t *out = static_cast<uint16_t *>(p.out) + (MODE == kGroupTN ? w.group * p.out_group : 0);
            *reinterpret_cast<uint2 *>(out + static_cast<int64_t>(w.j0 + j) * p.out_row + col) =
                make_uint2(pack_pair(p.bf16, __float_as_uint(v.x), __float_as_uint(v.y)),
                           pack_pair(p.bf16, __float_as_uint(v.z), __float_as_uint(v.w)));
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

// h[row] = scale_a * x[row] * down_a^T for a row with an adapter, as two 16-bit numbers
// (split_16; zeros up to a whole 16 ranks), for few rows.  256 threads: two warps a rank and
// half of K each, RANKS ranks at a time and `each` times so many a CTA.  The chain of a single token is the launch, the
// offsets and adapters, what down holds, and the sums; x is on its way from the start.
// SCALED (fp16): the row's CTAs are a cluster, which agrees on the row's power of two (row_exponent()).  RANKS: those
// at a time, with 64 threads each.
struct DownParams {
    const uint16_t *x, *down;
    int64_t x_row, down_row, down_matrix;
    uint16_t *h;
    int32_t each;
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

template <bool SCALED, int RANKS>
__global__ void __launch_bounds__(64 * RANKS) lora_down_kernel(const GroupParams p, const DownParams d) {
    // the first request that starts behind the row, and its predecessor's adapter
    __shared__ unsigned long long past;
    __shared__ float halves[RANKS];
    __shared__ float held[2][SCALED ? 128 : 1];  // SCALED: both halves of this CTA's ranks of h
    __shared__ uint32_t top_here;
    const int tid = static_cast<int>(threadIdx.x), lane = tid % 32, warp = tid / 32;
    const int64_t row = blockIdx.x;
    if (tid == 0) past = ~0ull;
    ptx::griddep_wait();
    // what follows may start: all before this kernel has completed
    if (tid == 0) ptx::griddep_launch_dependents();
    const int half = warp / RANKS;
    const int k_half = (p.R / 8 + 1) / 2 * 8;  // whole units of eight
    const int k_begin = half * k_half, k_end = half ? p.R : k_half;
    const uint16_t *x = d.x + row * d.x_row;
    constexpr int U = RANKS == 16 ? 4 : 8;  // loads on their way at once
    uint4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int k = k_begin + lane * 8 + i * 256;
        v[i] = make_uint4(0, 0, 0, 0);
        if (k < k_end) v[i] = *reinterpret_cast<const uint4 *>(x + k);
    }
    __syncthreads();
    unsigned long long least = ~0ull;
    for (int e = p.groups - tid; e >= 0; e -= 64 * RANKS) {
        const int64_t o = offset_of(p, e);
        const uint32_t a = e > 0 ? static_cast<uint32_t>(adapter_of(p, e - 1)) : ~0u;
        if (o > row) least = static_cast<unsigned long long>(e) << 32 | a;
    }
    // few threads have found one; of them the lowest
    const uint32_t first = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(least >> 32));
    if (static_cast<uint32_t>(least >> 32) == first && first != ~0u) atomicMin(&past, least);
    __syncthreads();
    // none behind it: the row is behind the last request (all of a cluster return, or none)
    const int32_t a = past != ~0ull ? static_cast<int32_t>(past & 0xffffffffull) : -1;
    if (a < 0) return;
    const int padded = (p.rank + 15) / 16 * 16;
    for (int q = 0; q < d.each; ++q) {
        const int j = (static_cast<int>(blockIdx.y) * d.each + q) * RANKS + warp % RANKS;
        float sum = 0.f;
        if (j < p.rank) {
            const uint16_t *down = d.down + j * d.down_row + a * d.down_matrix;
            for (int k = k_begin + lane * 8; k < k_end; k += 256 * U) {
                uint4 u[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    u[i] = make_uint4(0, 0, 0, 0);
                    if (k + i * 256 < k_end) u[i] = load_unit(down + k + i * 256);
                }
                if (k_end - k_begin > 256 * U) {  // v holds all of x only where it is no longer
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (k + i * 256 < k_end) v[i] = *reinterpret_cast<const uint4 *>(x + k + i * 256);
                    }
                }
#pragma unroll
                for (int i = 0; i < U; ++i) sum = dot_8(p.bf16, u[i], v[i], sum);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if constexpr (SCALED) {
            if (lane == 0) held[half][q * RANKS + warp % RANKS] = sum;
        } else {
            if (half && lane == 0) halves[warp % RANKS] = sum;
            __syncthreads();
            if (!half && lane == 0 && j < padded) {
                const float h = j < p.rank ? (sum + halves[warp]) * (p.scales ? p.scales[a] : 1.f) : 0.f;
                uint16_t *to = d.h + row * (2 * p.rank_pad) + j;
                split_16(p.bf16, h, to, to + p.rank_pad);
            }
            __syncthreads();
        }
    }
    if constexpr (SCALED) {
        const int first = static_cast<int>(blockIdx.y) * d.each * RANKS;
        const int count = padded - first < d.each * RANKS ? padded - first : d.each * RANKS;  // none: below 1
        if (tid == 0) top_here = 0;
        __syncthreads();
        const float h = tid < count && first + tid < p.rank ? (held[0][tid] + held[1][tid]) * (p.scales ? p.scales[a] : 1.f) : 0.f;
        if (warp * 32 < count) {  // up to four warps
            const uint32_t t = __reduce_max_sync(0xffffffffu, finite_bits(h));
            if (lane == 0) atomicMax(&top_here, t);
            __syncwarp();
        }
        uint32_t top = 0;
        const bool alone = gridDim.y == 1;
        if (alone) {
            __syncthreads();
            top = top_here;
        } else {
            ptx::cluster_sync();
            for (uint32_t s = 0; s < gridDim.y; ++s) {
                uint32_t t;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(t) : "r"(ptx::mapa(ptx::smem_u32(&top_here), s)) : "memory");
                top = top > t ? top : t;
            }
            ptx::cluster_arrive();
        }
        const int e = row_exponent(top);
        if (tid < count) {
            uint16_t *to = d.h + row * (2 * p.rank_pad) + first + tid;
            split_16(false, h * power_of_two(-e), to, to + p.rank_pad);
        }
        if (blockIdx.y == 0 && tid == 0) p.row_scale[row] = power_of_two(e);
        __syncwarp();
        if (!alone) ptx::cluster_wait();  // no CTA leaves while another reads its largest
    }
}

}  // namespace linear_ops
