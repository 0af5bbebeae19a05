// grouped_kernel.cuh -- products grouped by rows on the tensor cores
// (tcgen05.mma kind::f16): each group of rows has a matrix of its own.
//
// All three directions are one sum, with the contiguous axis of the result, i,
// on the 128-row side of the MMA (P) and the other, j, on its N side (Q):
//
//     out[j][i] = sum_r P[i][r] * Q[j][r]
//
//          i               j               r            P             Q
//     NT   columns of B_e  rows (ragged)   K            B_e           A
//     NN   K               rows (ragged)   columns      B_e, MN-major dD
//     TN   K               columns of dD   rows (ragged) A, MN-major  dD, MN-major
//
//     LORA columns of W    rows (ragged)   K, ranks      W, up_a       x, x * down_a^T
//     DOWN ranks           rows (ragged)   K             down_a        x
//
// So the ragged axis of NT and NN is N of the MMA, which takes any multiple of 16:
// a group's last tile costs what its rows cost, and few rows (decoding) leave the
// matrices' bytes to stream through the 128-row side.  Results of other groups' rows
// that a tile loaded with its own are other columns of the accumulator and are not
// stored.
//
// The ragged axis of TN is summed over: rows of the next group must not count with a
// group's last ones, whatever they hold (zeros by mask times an infinity would be NaN).
// The MMAs go in steps of 16 rows, so a last K tile that is no whole number of steps is
// loaded in boxes of 16, 8, 4, 2 and 1 rows, and the rest of its last step, in such boxes
// too, from behind the matrix, where the copy engine fills zeros.  (Cleared by a warp in
// shared memory, between the load's arrival and the MMA, they came too late: 8 groups of
// 1025 rows, 4096 x 4096, took 189 us where those of 1024 took 153; so 152 and 146.)
//
// LORA and DOWN are the two launches of low-rank adapters beside a shared product, with
// the rows of a request as a group.  DOWN leaves h = scale_a * x * down_a^T as two
// 16-bit numbers, h rounded and what that rounding left, which hold 16 bits of it (bf16) or, in fp16,
// 22 of its row's largest: fp16 has few exponents, so there a row of h is held times a power of two of
// its own where its largest is not in their midst (row_exponent()).  LORA's sum goes on over the ranks,
// once for each, so the result is rounded once; where rows of a tile have such a power, the ranks' sum
// goes to the other accumulator, and the epilogue brings each row's back before it adds it (4100
// tokens of 11 requests, rank 64, 4096 x 4096 fp16: 115 us without such rows, 137 with all).
// Rows without a request are a group without an adapter, before the first and behind the
// last.  A request's tile holds its own rows only: what another request's adapter holds
// cannot reach them.
//
// Persistent CTAs (or pairs, cta_group::2, 256 x 256 tiles) walk one list of tiles
// over all groups; each CTA reads the offsets once and keeps the groups' first rows
// and first tiles in shared memory, so the host needs to know no offset.
//
// Warps: 0 TMA producer, 1 MMA issuer and TMEM allocator, 2 lists the groups, 4-7 and
// 8-11 epilogue: two teams that take turns at
// 32 columns of the accumulator, as a team's way from TMEM to the store is latency.
#pragma once

#include "../schedule.h"
#include "bounded_wait.cuh"
#include "common.cuh"
#include "grouped_choice.h"
#include "grouped_ops.h"

namespace linear_ops {

using gemm_f16::PipelineState;

namespace ptxg {

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x,
                                                 int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// An arrival, possibly on the peer's barrier, that publishes no memory writes.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// 16 TMEM lanes x 32 columns of 32 bits: thread t gets of lane t / 4 and columns 8 n + 2 (t % 4),
// + 1 registers 4 n and 4 n + 1, of lane t / 4 + 8 registers 4 n + 2 and 4 n + 3.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// The first 8 of such columns: registers 0 to 3.
__device__ __forceinline__ void tmem_ld_16x256b_x1(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
}

// 32 TMEM lanes x one column.
__device__ __forceinline__ void tmem_ld_32x32b_x1(uint32_t taddr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
}

// Four 8 x 8 matrices of 16-bit elements, transposed on the way: thread t holds of
// matrix m elements (t / 4, 2 (t % 4)) and (t / 4, 2 (t % 4) + 1) in a word; threads
// 8 m to 8 m + 7 give the addresses of the 16 bytes that its columns 0 to 7 become.
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

// Shared-memory descriptors of operands with the 128-byte swizzle, as words: the high one
// (atoms of 8 rows, 1024 bytes, apart along M/N of a K-major operand, along K of an
// MN-major one; fields as in ptx::smem_desc_k_sw128) is the same for both, the low one has
// the address and, of an MN-major operand (rows of 64 elements along M/N, one for each k),
// how far its blocks of 64 lie apart.  Addresses move by additions to the low word (14 bits
// of it hold any offset in a CTA's shared memory; above them an address has the CTA's
// number in its cluster).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k_low(uint32_t smem_addr) { return ((smem_addr >> 4) & 0x3FFFu) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn_low(uint32_t smem_addr) {
    return ((smem_addr >> 4) & 0x3FFFu) | ((8192u >> 4) << 16);
}

template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
#define GROUPED_MMA(GROUP)                                                                                         \
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"                           \
                 "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"                                              \
                 "tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),                   \
                 "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(kDescHigh)                                \
                 : "memory")
    if constexpr (CG == 2) {
        GROUPED_MMA("2");
    } else {
        GROUPED_MMA("1");
    }
#undef GROUPED_MMA
}

// The MMAs of a stage, 16 elements of the sum each: A and B move on by A_STEP and B_STEP (of
// their low words; 32 bytes of a K-major row, 16 rows of 128 bytes of an MN-major tile).
template <int CG, uint32_t A_STEP, uint32_t B_STEP>
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, int steps, bool first) {
    mma_f16<CG>(d, a_low, b_low, idesc, first ? 0u : 1u);
    if (steps == 4) {
        mma_f16<CG>(d, a_low + A_STEP, b_low + B_STEP, idesc, 1u);
        mma_f16<CG>(d, a_low + 2 * A_STEP, b_low + 2 * B_STEP, idesc, 1u);
        mma_f16<CG>(d, a_low + 3 * A_STEP, b_low + 3 * B_STEP, idesc, 1u);
    } else {
        for (int k = 1; k < steps; ++k) mma_f16<CG>(d, a_low + k * A_STEP, b_low + k * B_STEP, idesc, 1u);
    }
}

// True in every thread if it is true in any of the 128 that share the barrier.
__device__ __forceinline__ bool any_of_128(uint32_t barrier, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "r"(barrier)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_128(uint32_t barrier) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(barrier) : "memory");
}

}  // namespace ptxg

// CG: CTAs of a tile; TN: its columns j.  A CTA holds 128 rows of P and TN / CG of Q.
template <int CG, int TN, int MODE>
struct GroupShape {
    static constexpr int BLOCK_R = 64;  // 128 bytes of a K-major row, 64 rows of an MN-major tile
    static constexpr int Q_ROWS = TN / CG;
    static constexpr int P_BYTES = 128 * 128;
    static constexpr int Q_BYTES = Q_ROWS * 128;
    static constexpr int STAGE = P_BYTES + Q_BYTES;
    // Q comes in boxes of so many rows, as many as a tile's columns need
    static constexpr int Q_BOX = MODE == kGroupTN ? 64 : (Q_ROWS < 32 ? Q_ROWS : 32);
    static constexpr int TMEM_COLS = 2 * TN;
    // The epilogue's staging: of each team a buffer of 32 rows j of 128 elements, as two
    // boxes of 64 with the 128-byte swizzle.
    static constexpr int BOX = 32 * 128;
    static constexpr int BUF = 2 * BOX;
    static constexpr bool ADAPTERS = MODE == kGroupLora || MODE == kGroupDown;
    static constexpr int LIST = 4 * (GROUPED_MAX_GROUPS + 4);  // int32 of each group, and its end
    static constexpr int REST = 2 * BUF + (ADAPTERS ? 3 : 2) * LIST + 1024 + 512;
    static constexpr int STAGES = (232448 - REST) / STAGE < 9 ? (232448 - REST) / STAGE : 9;
    static constexpr int OFF_P = 0;
    static constexpr int OFF_Q = OFF_P + STAGES * P_BYTES;
    static constexpr int OFF_D = OFF_Q + STAGES * Q_BYTES;
    static constexpr int OFF_START = OFF_D + 2 * BUF;
    static constexpr int OFF_TILES = OFF_START + LIST;
    static constexpr int OFF_CHOSEN = OFF_TILES + LIST;  // the groups' adapters, -1 without
    static constexpr int OFF_BAR = OFF_CHOSEN + (ADAPTERS ? LIST : 0);
    // full, empty [STAGES]; accumulator full, empty [2]; drain
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 5) * 8;
    static constexpr int OFF_APART = OFF_MISC + 16;  // LORA: whether a stage's tile has its ranks apart, [STAGES]
    static constexpr int SMEM_ALLOC = OFF_APART + (MODE == kGroupLora ? 4 * STAGES : 0) + 896;  // from a multiple of 128 bytes to one of 1024
    static constexpr int THREADS = 384;
    static_assert(STAGES >= 4 && OFF_BAR % 8 == 0 && SMEM_ALLOC <= 232448, "227 KiB");
    static_assert((CG == 2 && TN == 256) || (CG == 1 && (TN == 32 || TN == 64 || TN == 128)), "tile");
    static_assert(MODE != kGroupTN || Q_ROWS % 64 == 0, "MN-major blocks of 64");
};

struct GroupParams {
    const void *offsets;
    void *out;
    int64_t out_row, out_group;  // elements between rows j of the result, and between groups' matrices (TN)
    int32_t offsets_64;
    int32_t groups, rows;
    int32_t I, J, R;             // sizes; the ragged one is `rows`
    int32_t i_tiles, j_tiles;    // of a group; j_tiles for TN
    uint32_t band_inverse;       // 2^32 / (kGroupBand * i_tiles), rounded up
    int32_t turn;                // places that a cluster moves on by with each turn (TileWalk)
    int32_t bf16;
    int32_t zero_rest;
    // adapters
    const int32_t *adapters;     // of each request
    const float *scales;         // of each adapter (NULL: 1)
    int32_t adapter_count, rank;
    int32_t rank_pad;            // rank in whole 64s: h has 2 * rank_pad elements a row
    int32_t follows;             // LORA: behind a launch that leaves h
    // fp16: what brings each row of h back, and at the first row of each 32 of a request that DOWN had at
    // once whether that is 1 for all of them
    float *row_scale;
    int32_t *some_scaled;
    uint32_t debug_flags;
    uint64_t timeout_ns;
};

// A tile: its group, first i and j (of the result's row 0, or of the group's matrix),
// the j that count, and the length of its sum from row r0 on.
struct GroupTile {
    int32_t group, i0, j0, n, r0, r;
};

// Tiles of a band of j tiles share their P tiles, one after the other; a group's P is
// read again for each band.
constexpr int kGroupBand = 8;

// A sum from which on results leave by the copy engine.
constexpr int kLongSum = 512;

// The tiles of a persistent cluster: one of each turn of `clusters`, `turn` places further on than in
// the turn before (see turn_of() in grouped_gemm.cu).
struct TileWalk {
    int base, place, clusters, turn;
    __device__ __forceinline__ TileWalk(int cluster, int clusters, int turn)
        : base(0), place(cluster), clusters(clusters), turn(turn) {}
    __device__ __forceinline__ int t() const { return base + place; }
    __device__ __forceinline__ void next() {
        base += clusters;
        place += turn;
        if (place >= clusters) place -= clusters;
    }
};

// n / d for d >= 1 by d's rounded-up 2^32 / d: one too many at most, which the product shows.
__device__ __forceinline__ int div_by(int n, int d, uint32_t inverse) {
    if (d == 1) return n;
    const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(n), inverse));
    return q * d > n ? q - 1 : q;
}

// Tile t, t not before the one asked for last; `group` is that one's group (0 at first).
// A role asks once a tile, and tiles of short sums take some 2000 cycles, so there is no
// division here (band: kGroupBand * i_tiles, and its inverse).
template <int CG, int TN, int MODE>
__device__ __forceinline__ GroupTile group_tile(const GroupParams &p, const int32_t *start, const int32_t *tiles, int t,
                                                int &group) {
    while (tiles[group + 1] <= t) ++group;
    const int32_t first = start[group], count = start[group + 1] - first;
    const int32_t J = MODE == kGroupTN ? p.J : count;
    const int j_tiles = (J + TN - 1) / TN;
    int l = t - tiles[group];
    const int band = div_by(l, kGroupBand * p.i_tiles, p.band_inverse);
    const int width = j_tiles - band * kGroupBand < kGroupBand ? j_tiles - band * kGroupBand : kGroupBand;
    l -= band * kGroupBand * p.i_tiles;
    constexpr uint32_t kInverse[kGroupBand + 1] = {0,          0,          0x80000000, 0x55555556, 0x40000000,
                                                   0x33333334, 0x2aaaaaab, 0x24924925, 0x20000000};
    uint32_t inverse = kInverse[kGroupBand];
#pragma unroll
    for (int d = 2; d < kGroupBand; ++d) inverse = width == d ? kInverse[d] : inverse;
    const int i = div_by(l, width, inverse);
    GroupTile w;
    w.group = group;
    w.i0 = i * (128 * CG);
    const int32_t j = (band * kGroupBand + l - i * width) * TN;
    w.n = J - j < TN ? J - j : TN;
    w.j0 = MODE == kGroupTN ? j : first + j;
    w.r0 = MODE == kGroupTN ? first : 0;
    w.r = MODE == kGroupTN ? count : p.R;
    return w;
}

// The adapter of request e, -1 if it has none.
__device__ __forceinline__ int32_t adapter_of(const GroupParams &p, int e) {
    const int32_t a = p.adapters[e];
    return a >= 0 && a < p.adapter_count ? a : -1;
}

__device__ __forceinline__ int64_t offset_of(const GroupParams &p, int e) {
    if (!p.offsets) return 0;  // no requests
    return p.offsets_64 ? static_cast<const int64_t *>(p.offsets)[e]
                        : static_cast<int64_t>(static_cast<const int32_t *>(p.offsets)[e]);
}

// The groups' first rows (all threads), then from them, by one warp, their first tiles.
// With `rest` the rows without a group are groups too, the first and the last; `chosen`
// gets the groups' adapters.  Returns the number of groups.
__device__ __forceinline__ int group_starts(const GroupParams &p, int32_t *start, bool rest, int32_t *chosen, int thread,
                                            int threads) {
    const int shift = rest ? 1 : 0, groups = p.groups + 2 * shift;
    for (int e = thread; e <= p.groups; e += threads) {
        const int64_t o = offset_of(p, e);
        start[e + shift] = static_cast<int32_t>(o < 0 ? 0 : (o > p.rows ? p.rows : o));
        if (chosen && e < p.groups) chosen[e + shift] = adapter_of(p, e);
    }
    if (rest && thread == 0) {
        start[0] = 0;
        start[groups] = p.rows;
        if (chosen) chosen[0] = chosen[groups - 1] = -1;
    }
    return groups;
}
template <int TN, int MODE>
__device__ __forceinline__ void group_tiles(const GroupParams &p, int groups, int32_t *start, int32_t *tiles,
                                            const int32_t *chosen, int lane) {
    int32_t most = 0, sum = 0;
    for (int base = 0; base <= groups; base += 32) {
        const int e = base + lane;
        int32_t v = e <= groups ? start[e] : 0;
        v = v > most ? v : most;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {  // none lies before its predecessor
            const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o && u > v) v = u;
        }
        int32_t before = __shfl_up_sync(0xffffffffu, v, 1);
        if (lane == 0) before = most;
        // the tiles of group e - 1
        int32_t n = e == 0 || e > groups ? 0 : (MODE == kGroupTN ? p.j_tiles : (v - before + TN - 1) / TN) * p.i_tiles;
        if (MODE == kGroupDown && n > 0 && chosen[e - 1] < 0) n = 0;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int32_t u = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += u;
        }
        if (e <= groups) {
            start[e] = v;
            tiles[e] = sum + n;
        }
        most = __shfl_sync(0xffffffffu, v, 31);
        sum += __shfl_sync(0xffffffffu, n, 31);
    }
}

// Instruction descriptor of tcgen05.mma kind::f16 (PTX ISA): D fp32 [4,6)=1, A and B
// fp16 [7,10)=[10,13)=0 or bf16 1, MN-major ones marked [15], [16], N>>3 at [17,23),
// M>>4 at [24,29).
template <int CG, int MODE>
__device__ __forceinline__ uint32_t group_idesc(int n, bool bf16) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 * CG >> 4) << 24) | (bf16 ? (1u << 7) | (1u << 10) : 0u) |
           (MODE == kGroupNN || MODE == kGroupTN ? 1u << 15 : 0u) | (MODE == kGroupTN ? 1u << 16 : 0u);
}

__device__ __forceinline__ uint32_t pack_pair(bool bf16, uint32_t lo, uint32_t hi) {
    const float2 v = make_float2(__uint_as_float(lo), __uint_as_float(hi));
    uint32_t w;
    if (bf16) {
        Pair<__nv_bfloat16>::narrow(v, &w);
    } else {
        Pair<__half>::narrow(v, &w);
    }
    return w;
}

// h as a 16-bit number and the rest of it as another (0 where h, or its rounding, is not
// finite: an infinity less itself would be NaN).
__device__ __forceinline__ void split_16(bool bf16, float h, uint16_t *high, uint16_t *low) {
    uint32_t a, b;
    if (bf16) {
        Pair<__nv_bfloat16>::narrow(make_float2(h, 0.f), &a);
        if ((a & 0x7fffu) == 0x7f80u && fabsf(h) < INFINITY) --a;  // past the largest bf16, whose rest the second one holds
        const float rest = h - Pair<__nv_bfloat16>::widen(&a).x;
        Pair<__nv_bfloat16>::narrow(make_float2(fabsf(rest) < INFINITY ? rest : 0.f, 0.f), &b);
    } else {
        Pair<__half>::narrow(make_float2(h, 0.f), &a);
        const float rest = h - Pair<__half>::widen(&a).x;
        Pair<__half>::narrow(make_float2(fabsf(rest) < INFINITY ? rest : 0.f, 0.f), &b);
    }
    *high = static_cast<uint16_t>(a);
    *low = static_cast<uint16_t>(b);
}

// h of fp16 rows: the bits of a magnitude, 0 of infinities and NaN (they stay what they are).
__device__ __forceinline__ uint32_t finite_bits(float h) {
    const uint32_t b = __float_as_uint(h) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}
// The exponent of the power of two that a row of h is divided by, from its largest finite magnitude: 0
// where that is from 2^-3 to 2^15 (then the second number's least step, 2^-24, is 2^-21 of it at most),
// else what brings it to 2^14 to 2^15; from -112 on, as 2^112 and 2^-112 are normal and what is
// smaller still adds nothing that fp16 shows.
__device__ __forceinline__ int row_exponent(uint32_t top) {
    const int e = static_cast<int>(top >> 23) - 127;
    return top == 0u || (e >= -3 && e <= 14) ? 0 : (e < -98 ? -112 : e - 14);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// TN: P's and Q's maps with boxes of 2^k rows.
template <int MODE>
struct GroupTails {};
template <>
struct GroupTails<kGroupTN> {
    CUtensorMap P[5], Q[5];
};

// A K tile of a sum over rows, from the sum's row r on: P's columns from i0 on and `boxes` blocks of
// Q's from j0 on.  A last tile that is no whole number of steps comes in boxes of 16 to 1 rows, and
// zeros from behind the matrix up to the step's end.
template <int CG>
__device__ __forceinline__ void load_sum_rows(const GroupParams &p, const CUtensorMap &tmP, const CUtensorMap &tmQ,
                                              const GroupTails<kGroupTN> &tails, const GroupTile &w, int r, int32_t i0, int32_t j0,
                                              int boxes, bool leader, uint32_t sp, uint32_t sq, uint32_t full) {
    const int rows = w.r - r;
    const bool tail = rows < 64 && rows % 16 != 0;
    const int steps = (rows + 15) / 16 * 16;
    if (leader) ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(CG * (tail ? steps : 64) * 128 * (2 + boxes)));
    if constexpr (CG == 2) full = ptx::mapa(full, 0);
    auto load = [&](const CUtensorMap &mapP, const CUtensorMap &mapQ, int row, int32_t y) {
        auto one = [&](uint32_t dst, const CUtensorMap &map, int32_t x) {
            if constexpr (CG == 2) {
                ptx::tma_load_2d_pair(dst + row * 128, &map, full, x, y);
            } else {
                ptx::tma_load_2d(dst + row * 128, &map, full, x, y);
            }
        };
#pragma unroll
        for (int b = 0; b < 2; ++b) one(sp + b * 8192, mapP, i0 + 64 * b);
        for (int b = 0; b < boxes; ++b) one(sq + b * 8192, mapQ, j0 + 64 * b);
    };
    if (!tail) {
        load(tmP, tmQ, 0, w.r0 + r);
        return;
    }
    int row = 0;
    for (; rows - row >= 16; row += 16) load(tails.P[4], tails.Q[4], row, w.r0 + r + row);
    for (int k = 3, left = rows - row; k >= 0; --k) {
        if (left >> k & 1) load(tails.P[k], tails.Q[k], row, w.r0 + r + row), row += 1 << k;
    }
    for (int k = 0, left = steps - row; k < 4; ++k) {
        if (left >> k & 1) load(tails.P[k], tails.Q[k], row, p.rows), row += 1 << k;
    }
}

// Sums of 16 TMEM lanes x 32 columns (as tmem_ld_16x256b_x4 has them), each column's times its row's
// scale, added to v; `rows` of the columns have one.
__device__ __forceinline__ void add_scaled(uint32_t taddr, const float *row_scale, int rows, int lane, uint32_t (&v)[16]) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {  // 8 columns at a time: few registers
        uint32_t more[4];
        ptxg::tmem_ld_16x256b_x1(taddr + n * 8, more);
        const int j = 8 * n + 2 * (lane % 4);
        const float s = j < rows ? row_scale[j] : 0.f, t = j + 1 < rows ? row_scale[j + 1] : 0.f;
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[4 * n + i] = __float_as_uint(fmaf(__uint_as_float(more[i]), i % 2 ? t : s, __uint_as_float(v[4 * n + i])));
        }
    }
}

// LORA in 80 registers, as for two CTAs an SM, to find room beside lora_down_kernel's: 300 rows of rank 24, 4096 x
// 4096, 25.3 us, else 35.3.
template <int CG, int TN, int MODE>
__global__ void __launch_bounds__(384, MODE == kGroupLora ? 2 : 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmU,
                   const __grid_constant__ CUtensorMap tmH, const __grid_constant__ GroupTails<MODE> tails, const GroupParams p) {
    using C = GroupShape<CG, TN, MODE>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const int rank = CG == 2 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
    const bool leader = rank == 0;
    const int cluster = static_cast<int>(blockIdx.x) / CG, clusters = static_cast<int>(gridDim.x) / CG;

    const uint32_t bar_full = base + C::OFF_BAR, bar_empty = bar_full + 8 * C::STAGES;
    const uint32_t bar_tfull = bar_empty + 8 * C::STAGES, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    volatile int32_t *stage_apart = reinterpret_cast<volatile int32_t *>(smem + C::OFF_APART);
    int32_t *start = reinterpret_cast<int32_t *>(smem + C::OFF_START);
    int32_t *tiles = reinterpret_cast<int32_t *>(smem + C::OFF_TILES);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(bar_tfull + 8 * a, 1);
            ptx::mbar_init(bar_tempty + 8 * a, 8 * CG);  // the epilogue warps of all the tile's CTAs
        }
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0;
        ptx::fence_mbarrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc<CG>(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
        ptx::tmem_relinquish<CG>();
    }
    // LORA follows DOWN, which lets it start only once the kernels before both have
    // completed: it waits for h alone, in the producer.
    if (MODE != kGroupDown && threadIdx.x == 0) ptx::griddep_launch_dependents();
    if (MODE != kGroupLora || !p.follows) ptx::griddep_wait();
    if (MODE == kGroupDown && threadIdx.x == 0) ptx::griddep_launch_dependents();
    int32_t *chosen = C::ADAPTERS ? reinterpret_cast<int32_t *>(smem + C::OFF_CHOSEN) : nullptr;
    const int groups = group_starts(p, start, MODE == kGroupLora, chosen, static_cast<int>(threadIdx.x), C::THREADS);
    __syncthreads();
    if (warp == 2) group_tiles<TN, MODE>(p, groups, start, tiles, chosen, lane);
    ptx::tcgen05_fence_before();
    if constexpr (CG == 2) {
        ptx::cluster_sync();
    } else {
        __syncthreads();
    }
    ptx::tcgen05_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    const int total = tiles[groups];
    int group = 0;  // of a role's last tile
    auto tile_of = [&](int t) { return group_tile<CG, TN, MODE>(p, start, tiles, t, group); };
    // K tiles over the ranks, two of each 64: with h rounded and with the rest of it
    auto rank_tiles = [&](const GroupTile &w) {
        return MODE == kGroupLora && chosen[w.group] >= 0 ? p.rank_pad / 64 * 2 : 0;
    };
    // what DOWN has left of a tile's rows, and whether its ranks have an accumulator of their own.  Asked for
    // at a tile's start and looked at near its end, the answer costs nothing (4100 tokens in fp16 115 us, else 117)
    constexpr int FLAGS = MODE == kGroupLora ? TN / 32 : 1;
    auto ask_scaled = [&](const GroupTile &w, int32_t (&some)[FLAGS]) {
#pragma unroll
        for (int j = 0; j < FLAGS; ++j) some[j] = j * 32 < w.n ? p.some_scaled[w.j0 + j * 32] : 0;
    };
    auto any_scaled = [](const int32_t (&some)[FLAGS]) {
        int32_t any = 0;
#pragma unroll
        for (int j = 0; j < FLAGS; ++j) any |= some[j];
        return any;
    };
    // N of a tile's MMAs; a pair's CTAs hold half of these rows of Q each
    auto columns_of = [](const GroupTile &w) { return (w.n + 16 * CG - 1) / (16 * CG) * (16 * CG); };

    if (warp == 0) {
        if (ptx::elect_one()) {
            PipelineState ring(C::STAGES, (p.debug_flags & 1u) ? 0u : 1u);
            bool ok = true, waited = false;
            uint32_t seq = 0;
            for (TileWalk walk(cluster, clusters, p.turn); ok && walk.t() < total; walk.next(), ++seq) {
                const GroupTile w = tile_of(walk.t());
                const int k_tiles = (w.r + 63) / 64, all_tiles = k_tiles + rank_tiles(w);
                const int32_t i0 = w.i0 + rank * 128, j0 = w.j0 + rank * (columns_of(w) / 2);
                const int boxes = (columns_of(w) / CG + C::Q_BOX - 1) / C::Q_BOX;  // of Q, in each CTA
                // of DOWN's P only the ranks that there are
                const uint32_t bytes = (MODE == kGroupDown ? p.rank * 128u : C::P_BYTES) + static_cast<uint32_t>(boxes * C::Q_BOX) * 128u;
                const bool ask = MODE == kGroupLora && !p.bf16 && leader && all_tiles > k_tiles, asked = ask && waited;
                int32_t some[FLAGS];
                if (asked) ask_scaled(w, some);
                for (int kt = 0; kt < all_tiles; ++kt) {
                    if (!wait_bounded(bar_empty + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns,
                                      kWaitProducer, seq)) {
                        ok = false;
                        break;
                    }
                    const int s = ring.stage, r = kt * 64;
                    const uint32_t sp = base + C::OFF_P + s * C::P_BYTES, sq = base + C::OFF_Q + s * C::Q_BYTES;
                    uint32_t full = bar_full + 8 * s;
                    if constexpr (MODE == kGroupTN) {
                        load_sum_rows<CG>(p, tmP, tmQ, tails, w, r, i0, j0, boxes, leader, sp, sq, full);
                        ring.advance();
                        continue;
                    }
                    if constexpr (MODE == kGroupLora) {
                        if (kt >= k_tiles) {
                            if (!waited) ptx::griddep_wait();
                            waited = true;
                            if (kt == k_tiles && ask && !asked) ask_scaled(w, some);
                            // the issuer reads it behind the stage's barrier
                            if (kt == k_tiles && leader) stage_apart[s] = ask ? any_scaled(some) : 0;
                        }
                    }
                    if (leader) ptx::mbar_arrive_expect_tx(full, CG * bytes);
                    if constexpr (CG == 2) full = ptx::mapa(full, 0);
                    auto load_2d = [&](uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y) {
                        if constexpr (CG == 2) {
                            ptx::tma_load_2d_pair(dst, map, full, x, y);
                        } else {
                            ptx::tma_load_2d(dst, map, full, x, y);
                        }
                    };
                    auto load_3d = [&](uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z) {
                        if constexpr (CG == 2) {
                            ptxg::tma_load_3d_pair(dst, map, full, x, y, z);
                        } else {
                            ptxg::tma_load_3d(dst, map, full, x, y, z);
                        }
                    };
                    if constexpr (MODE == kGroupLora) {
                        if (kt >= k_tiles) {
                            const int32_t c = (kt - k_tiles) / 2 * 64, rest = (kt - k_tiles) % 2 * p.rank_pad;
                            load_3d(sp, &tmU, c, i0, chosen[w.group]);
                            for (int b = 0; b < boxes; ++b) load_2d(sq + b * C::Q_BOX * 128, &tmH, rest + c, j0 + b * C::Q_BOX);
                            ring.advance();
                            continue;
                        }
                        load_3d(sp, &tmP, r, i0, 0);
                    } else if constexpr (MODE == kGroupDown) {
                        load_3d(sp, &tmP, r, 0, chosen[w.group]);
                    } else if constexpr (MODE == kGroupNT) {
                        load_3d(sp, &tmP, r, i0, w.group);
                    } else if constexpr (MODE == kGroupNN) {
#pragma unroll
                        for (int b = 0; b < 2; ++b) load_3d(sp + b * 8192, &tmP, i0 + 64 * b, r, w.group);
                    }
                    for (int b = 0; b < boxes; ++b) load_2d(sq + b * C::Q_BOX * 128, &tmQ, r, j0 + b * C::Q_BOX);
                    ring.advance();
                }
            }
            if (!ok) {  // time for loads in flight to land before the shared memory goes
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 20000) ptx::nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader && ptx::elect_one()) {
            PipelineState ring(C::STAGES, 0u);
            PipelineState acc(2, 1u);
            const uint32_t sp = base + C::OFF_P, sq = base + C::OFF_Q;
            const uint32_t p_low = MODE == kGroupNN || MODE == kGroupTN ? ptxg::desc_mn_low(sp) : ptxg::desc_k_low(sp);
            const uint32_t q_low = MODE == kGroupTN ? ptxg::desc_mn_low(sq) : ptxg::desc_k_low(sq);
            bool ok = true;
            uint32_t seq = 0;
            for (TileWalk walk(cluster, clusters, p.turn); ok && walk.t() < total; walk.next(), ++seq) {
                const GroupTile w = tile_of(walk.t());
                const int k_tiles = (w.r + 63) / 64, all_tiles = k_tiles + rank_tiles(w);
                if (all_tiles == 0) continue;
                const uint32_t idesc = group_idesc<CG, MODE>(columns_of(w), p.bf16);
                uint32_t d = tmem_base + static_cast<uint32_t>(acc.stage * TN);
                bool apart = false;
                if (!wait_bounded(bar_tempty + 8 * acc.stage, acc.phase, abort_flag, p.timeout_ns, kWaitMma,
                                  seq)) {
                    break;
                }
                ptx::tcgen05_fence_after();
                for (int kt = 0; kt < all_tiles; ++kt) {
                    if (!wait_bounded(bar_full + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns,
                                      kWaitMma, seq)) {
                        ok = false;
                        break;
                    }
                    ptx::tcgen05_fence_after();
                    const int s = ring.stage;
                    constexpr bool kMnP = MODE == kGroupNN || MODE == kGroupTN, kMnQ = MODE == kGroupTN;
                    const int left = kt < k_tiles ? w.r - kt * 64 : p.rank - (kt - k_tiles) / 2 * 64;
                    if constexpr (MODE == kGroupLora) {
                        if (kt == k_tiles && stage_apart[s]) {
                            apart = true;
                            PipelineState other = acc;
                            other.advance();
                            if (!wait_bounded(bar_tempty + 8 * other.stage, other.phase, abort_flag, p.timeout_ns, kWaitMma, seq)) {
                                ok = false;
                                break;
                            }
                            ptx::tcgen05_fence_after();
                            d = tmem_base + static_cast<uint32_t>(other.stage * TN);
                        }
                    }
                    ptxg::mma_stage<CG, kMnP ? 128 : 2, kMnQ ? 128 : 2>(
                        d, p_low + static_cast<uint32_t>(s * (C::P_BYTES >> 4)), q_low + static_cast<uint32_t>(s * (C::Q_BYTES >> 4)),
                        idesc, left >= 64 ? 4 : (left + 15) / 16, kt == 0 || (apart && kt == k_tiles));
                    ptx::mma_commit<CG>(bar_empty + 8 * s, 0x3);
                    ring.advance();
                }
                if (!ok) break;
                ptx::mma_commit<CG>(bar_tfull + 8 * acc.stage, 0x3);
                acc.advance();
                if (apart) {
                    ptx::mma_commit<CG>(bar_tfull + 8 * acc.stage, 0x3);
                    acc.advance();
                }
            }
            ptx::mma_commit<CG>(bar_drain, 0x1);
            wait_bounded(bar_drain, 0, abort_flag, p.timeout_ns, kWaitMma, 0xFFFFFFFFu, false);
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quarter = warp % 4, team = (warp - 4) / 4;
        const uint32_t tempty = CG == 2 ? ptx::mapa(bar_tempty, 0) : bar_tempty;
        const int tid = static_cast<int>(threadIdx.x) % 128;  // in the team
        const int x = tid % 16, y = tid / 16;
        const uint32_t barrier = 1u + static_cast<uint32_t>(team);
        uint16_t *out = static_cast<uint16_t *>(p.out);
        const uint4 none = make_uint4(0, 0, 0, 0);
        if ((MODE == kGroupNT || MODE == kGroupNN) && p.zero_rest) {  // rows without a group: 16-byte units, a warp a row
            const int32_t head = start[0], rest = head + p.rows - start[p.groups];
            for (int32_t k = static_cast<int32_t>(blockIdx.x) * 8 + (warp - 4); k < rest; k += static_cast<int32_t>(gridDim.x) * 8) {
                uint16_t *row = out + static_cast<int64_t>(k < head ? k : start[p.groups] + (k - head)) * p.out_row;
                for (int32_t u = lane * 8; u < p.I; u += 256) *reinterpret_cast<uint4 *>(row + u) = none;
            }
        }
        PipelineState acc(2, 0u);
        bool waited = false;
        uint32_t seq = 0;
        for (TileWalk walk(cluster, clusters, p.turn); walk.t() < total; walk.next(), ++seq) {
            const GroupTile w = tile_of(walk.t());
            const int32_t i0 = w.i0 + rank * 128;
            const int32_t width = p.I - i0 < 128 ? p.I - i0 : 128;  // of this CTA's columns
            uint16_t *at = out + (MODE == kGroupTN ? w.group * p.out_group : 0) + static_cast<int64_t>(w.j0) * p.out_row + i0;
            if (w.r == 0) {  // a sum of nothing
                for (int32_t j = team * 8 + y; j < w.n; j += 16) {
                    if (x * 8 < width) *reinterpret_cast<uint4 *>(at + j * p.out_row + x * 8) = none;
                }
                continue;
            }
            const bool ask = MODE == kGroupLora && !p.bf16 && rank_tiles(w) > 0, asked = ask && waited;
            bool apart = false;
            if (asked) {  // before the tile's wait, not behind it
                int32_t some[FLAGS];
                ask_scaled(w, some);
                apart = any_scaled(some) != 0;
            }
            bool failed = false;
            if (lane == 0) {
                failed = !wait_bounded(bar_tfull + 8 * acc.stage, acc.phase, abort_flag, p.timeout_ns,
                                       kWaitEpilogue, seq);
            }
            if (ptxg::any_of_128(barrier, failed)) break;  // all four warps or none
            ptx::tcgen05_fence_after();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc.stage * TN);
            const int chunks = (w.n + 31) / 32;
            PipelineState other = acc;  // LORA: the accumulator of ranks apart
            if constexpr (MODE == kGroupLora) {
                if (ask && !asked) {  // DOWN has ended, as the tile's sums have come
                    ptx::griddep_wait();
                    waited = true;
                    int32_t some[FLAGS];
                    ask_scaled(w, some);
                    apart = any_scaled(some) != 0;
                }
                if (apart) {
                    other.advance();
                    if (lane == 0) failed = !wait_bounded(bar_tfull + 8 * other.stage, other.phase, abort_flag, p.timeout_ns, kWaitEpilogue, seq);
                    if (ptxg::any_of_128(barrier, failed)) break;
                    ptx::tcgen05_fence_after();
                }
            }
            if constexpr (MODE == kGroupDown) {
                // a lane a rank: h and what its rounding left, zeros up to a whole 16
                const int32_t padded = (p.rank + 15) / 16 * 16, i = quarter * 32 + lane;
                const float scale = p.scales ? p.scales[chosen[w.group]] : 1.f;
                uint16_t *to = out + static_cast<int64_t>(w.j0) * p.out_row + i;
#pragma unroll 1
                for (int c = team; c < chunks; c += 2) {
                    uint32_t v[32];
                    const bool some = quarter * 32 < padded;
                    if (some) {
                        ptx::tmem_ld_32x32b_x32(taddr + c * 32, v);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * scale);
                    }
                    float by = 1.f;  // of fp16: what row c * 32 + lane is held times
                    uint32_t scaled = 0;  // rows for which that is not 1
                    if (!p.bf16) {
                        uint32_t top = 0;
                        if (some) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const uint32_t t = __reduce_max_sync(0xffffffffu, i < p.rank ? finite_bits(__uint_as_float(v[j])) : 0u);
                                if (lane == j) top = t;
                            }
                        }
                        // the warps have 32 ranks each; the team's staging buffer is not used else
                        volatile uint32_t *tops = reinterpret_cast<volatile uint32_t *>(smem + C::OFF_D + team * C::BUF);
                        tops[quarter * 32 + lane] = top;
                        ptxg::sync_128(barrier);
#pragma unroll
                        for (int q = 0; q < 4; ++q) top = top > tops[q * 32 + lane] ? top : tops[q * 32 + lane];
                        const bool there = c * 32 + lane < w.n;
                        const int e = row_exponent(top);
                        by = power_of_two(-e);
                        scaled = __ballot_sync(0xffffffffu, there && e != 0);
                        if (quarter == 0 && there) p.row_scale[w.j0 + c * 32 + lane] = power_of_two(e);
                        if (quarter == 0 && lane == 0) p.some_scaled[w.j0 + c * 32] = scaled != 0u;
                    }
                    if (!some) continue;
                    if (scaled != 0u) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * __shfl_sync(0xffffffffu, by, j));
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (c * 32 + j >= w.n || i >= padded) continue;
                        uint16_t high, low;
                        split_16(p.bf16, i < p.rank ? __uint_as_float(v[j]) : 0.f, &high, &low);
                        to[(c * 32 + j) * p.out_row] = high;
                        to[(c * 32 + j) * p.out_row + p.rank_pad] = low;
                    }
                }
                ptx::tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(tempty + 8 * acc.stage);
                acc.advance();
            } else {
                auto hand_over = [&] {  // the accumulator is read: the next tile but one may have it
                    ptx::tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 2) {
                            ptxg::mbar_arrive_cluster_relaxed(tempty + 8 * acc.stage);
                            if (apart) ptxg::mbar_arrive_cluster_relaxed(tempty + 8 * other.stage);
                        } else {
                            ptx::mbar_arrive(tempty + 8 * acc.stage);
                        }
                    }
                };
                if (chunks <= team) hand_over();
#pragma unroll 1
                for (int c = team; c < chunks; c += 2) {
                    uint32_t lo[16], hi[16];
                    ptxg::tmem_ld_16x256b_x4(taddr + c * 32, lo);
                    ptxg::tmem_ld_16x256b_x4(taddr + (16u << 16) + c * 32, hi);
                    ptx::tmem_wait_ld();
                    if constexpr (MODE == kGroupLora) {
                        if (apart) {
                            const uint32_t ranks = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(other.stage * TN + c * 32);
                            add_scaled(ranks, p.row_scale + w.j0 + c * 32, w.n - c * 32, lane, lo);
                            add_scaled(ranks + (16u << 16), p.row_scale + w.j0 + c * 32, w.n - c * 32, lane, hi);
                        }
                    }
                    if (c + 2 >= chunks) hand_over();
                    const uint32_t buf = base + C::OFF_D + team * C::BUF;
                    if (tid == 0) ptx::bulk_wait_group_read<0>();  // what was in the buffer has left it
                    ptxg::sync_128(barrier);
                    // lane l: row l % 8 of matrix l / 8 (columns 8 (n + l / 16) on, lanes 8 (l / 8 % 2) on);
                    // 16-byte unit u of row j lies at u ^ j % 8
                    const uint32_t own = buf + static_cast<uint32_t>(quarter >> 1) * C::BOX +
                                         static_cast<uint32_t>((lane & 7) + (lane >> 4) * 8) * 128u;
                    const uint32_t unit = static_cast<uint32_t>((quarter & 1) * 4 + (lane >> 3 & 1));
                    const uint32_t low = own + ((unit ^ (lane & 7u)) * 16u), high = own + (((unit + 2) ^ (lane & 7u)) * 16u);
#pragma unroll
                    for (int n = 0; n < 4; n += 2) {
                        ptxg::stmatrix_trans(low + n * 8 * 128, pack_pair(p.bf16, lo[4 * n], lo[4 * n + 1]),
                                             pack_pair(p.bf16, lo[4 * n + 2], lo[4 * n + 3]),
                                             pack_pair(p.bf16, lo[4 * n + 4], lo[4 * n + 5]),
                                             pack_pair(p.bf16, lo[4 * n + 6], lo[4 * n + 7]));
                        ptxg::stmatrix_trans(high + n * 8 * 128, pack_pair(p.bf16, hi[4 * n], hi[4 * n + 1]),
                                             pack_pair(p.bf16, hi[4 * n + 2], hi[4 * n + 3]),
                                             pack_pair(p.bf16, hi[4 * n + 4], hi[4 * n + 5]),
                                             pack_pair(p.bf16, hi[4 * n + 6], hi[4 * n + 7]));
                    }
                    // By the copy engine, which needs no thread, where a tile's MMAs take longer than
                    // its epilogue: weights of 8 groups of 1024 rows, 4096 x 4096, 146 us, by threads
                    // 152.  By threads, which need not wait for it, where the epilogue is what takes
                    // the time: 32 groups of 16 rows, 1416 x 2040, 41.9 us, by the copy engine 50.7.
                    if ((MODE == kGroupTN || w.n - c * 32 >= 32) && w.r >= kLongSum) {
                        ptx::fence_proxy_async_smem();
                        ptxg::sync_128(barrier);
                        if (tid == 0) {
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                if (width <= b * 64) continue;
                                if constexpr (MODE == kGroupTN) {
                                    ptx::tma_store_3d(&tmD, buf + b * C::BOX, i0 + b * 64, w.j0 + c * 32, w.group);
                                } else {
                                    ptx::tma_store_2d(&tmD, buf + b * C::BOX, i0 + b * 64, w.j0 + c * 32);
                                }
                            }
                            ptx::bulk_commit_group();
                        }
                        continue;
                    }
                    ptxg::sync_128(barrier);
                    // 16 threads a row, 16 bytes each; rows behind a group's end belong to the next
                    const uint32_t from = buf + static_cast<uint32_t>(x / 8) * C::BOX + static_cast<uint32_t>(y) * 128u +
                                          ((static_cast<uint32_t>(x & 7) ^ (y & 7u)) * 16u);
                    uint16_t *to = at + (c * 32 + y) * p.out_row + x * 8;
                    const int32_t rows = x * 8 < width ? w.n - c * 32 - y : 0;
                    uint4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = ptx::ld_shared_v4(from + k * 8 * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k, to += 8 * p.out_row) {
                        if (k * 8 >= rows) continue;
                        if constexpr (MODE == kGroupTN) {
                            // matrices that are far more than L2 holds leave it first: 32 groups of 16
                            // rows, 1416 x 2040, 41.9 us, else 42.2 (only zeros, of 16 matrices of 4096 x
                            // 4096: 82 to 84, 6.4 TB/s, which is what writes get)
                            __stcs(reinterpret_cast<uint4 *>(to), v[k]);
                        } else {
                            *reinterpret_cast<uint4 *>(to) = v[k];
                        }
                    }
                }
                acc.advance();
                if (apart) acc.advance();
            }
        }
        if (tid == 0) ptx::bulk_wait_group_read<0>();
        __syncwarp();
    }
    if (MODE == kGroupLora) ptx::griddep_wait();  // the next kernel waits for this one alone: not before DOWN has ended
    ptx::tcgen05_fence_before();
    if constexpr (CG == 2) {
        ptx::cluster_arrive_relaxed();
        ptx::cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        ptx::tcgen05_fence_after();
        ptx::tmem_dealloc<CG>(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace linear_ops
